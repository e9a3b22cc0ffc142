"""GPU: the short causal convolution (kda_conv_*) against the fp64 oracle.

Tolerance.  Every output is a sum of products computed in fp32 from the exact
input values, so its error is at most (number of roundings) * 2^-24 times the sum
of the terms' absolute values, which the oracle gives with absolute=True: W + 1
roundings for the sum, and about 8 more through the exponential (2 ulp), the
reciprocal (1 ulp) and the products of the activation, taken as 32 in all.  The
weight's gradient adds up to T tokens: T / 8 + 32 more.  A bf16 output adds one
rounding, half a step of 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle.mixer as om
import gated_delta_rule_133_b200 as kda
from tests._helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _inputs(lens, D, W, dtype, seed, bias=True, state=True):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    x = torch.randn(T, D, generator=g).to(dtype)
    w = torch.randn(D, W, generator=g) * 0.5
    b = torch.randn(D, generator=g) if bias else None
    s0 = torch.randn(N, W - 1, D, generator=g).to(dtype) if state else None
    gy, gsT = torch.randn(T, D, generator=g), torch.randn(N, W - 1, D, generator=g)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return x, w, b, s0, gy, gsT, cu


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _close(got, ref, mag, n, rounded=False):
    got, bound = f64(got), n * U * mag + (2.0 ** -8 * (np.abs(ref) + n * U * mag) if rounded else 0) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (bad.sum(), np.abs(got - ref).max(), np.argwhere(bad)[:3])


DENSE = [(2, 37, 24, 4), (1, 1, 8, 2), (3, 2, 64, 4), (1, 200, 1032, 3), (2, 64, 136, 2), (1, 129, 256, 4)]


@pytest.mark.parametrize("dtype,o_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                           (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("B,T,D,W", DENSE)
def test_conv_fwd(B, T, D, W, dtype, o_dtype):
    silu = T != 64
    x, w, b, s0, _, _, cu = _inputs([T] * B, D, W, dtype, 7 * T + W, bias=T > 1, state=B < 3)
    xd, wd, bd, sd = _dev(x, w, b, s0)
    y, sT = kda.kda_conv_fwd(xd.view(B, T, D), wd, bd, sd, silu=silu, o_dtype=o_dtype)
    kda.kda_check()
    args = (f64(x), f64(w), f64(b), cu, f64(s0), silu)
    ref, ref_s = om.conv(*args)
    mag, _ = om.conv(*args, absolute=True)
    _close(y.view(B * T, D), ref, mag, 32, o_dtype == torch.bfloat16)
    assert np.array_equal(f64(sT), ref_s)


LENS = [[5, 0, 1, 2, 70, 3], [1], [0, 0, 4], [64, 64, 1, 63], [1] * 40, [300]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("W", [2, 4])
def test_conv_varlen_fwd(lens, W, dtype):
    D = 40
    x, w, b, s0, _, _, cu = _inputs(lens, D, W, dtype, len(lens) + W)
    xd, wd, bd, sd = _dev(x, w, b, s0)
    y, sT = kda.kda_conv_varlen_fwd(xd, wd, bd, torch.from_numpy(cu).to(DEV), sd, o_dtype=torch.float32)
    kda.kda_check()
    ref, ref_s = om.conv(f64(x), f64(w), f64(b), cu, f64(s0))
    mag, _ = om.conv(f64(x), f64(w), f64(b), cu, f64(s0), absolute=True)
    _close(y, ref, mag, 32)
    assert np.array_equal(f64(sT), ref_s)


def test_conv_many_sequences():
    """More sequences than one probe of the boundary search covers, empty ones among them."""
    lens = [(7 * i) % 5 for i in range(3000)]
    D, W = 16, 4
    x, w, b, s0, gy, gsT, cu = _inputs(lens, D, W, torch.float32, 5)
    xd, wd, bd, sd, gyd, gsd = _dev(x, w, b, s0, gy, gsT)
    cud = torch.from_numpy(cu).to(DEV)
    y, sT = kda.kda_conv_varlen_fwd(xd, wd, bd, cud, sd)
    got = kda.kda_conv_varlen_bwd(xd, wd, bd, cud, sd, gyd, gsd)
    kda.kda_check()
    args = (f64(x), f64(w), f64(b), cu, f64(s0))
    ref, ref_s = om.conv(*args)
    _close(y, ref, om.conv(*args, absolute=True)[0], 32)
    assert np.array_equal(f64(sT), ref_s)
    grads = dict(gy=f64(gy), gsT=f64(gsT))
    for a, r, m in zip(got, om.conv(*args, **grads), om.conv(*args, **grads, absolute=True)):
        _close(a, r, m, 64 + sum(lens) / 8)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype,W,lens", [
    (torch.bfloat16, 4, [37, 37]), (torch.float32, 3, [129]), (torch.float32, 2, [1, 1, 1]), (torch.bfloat16, 4, [200])])
def test_conv_bwd(dtype, W, lens, silu):
    B, T, D = len(lens), lens[0], 136
    x, w, b, s0, gy, gsT, cu = _inputs(lens, D, W, dtype, 3 * T, bias=silu)
    xd, wd, bd, sd, gyd, gsd = _dev(x, w, b, s0, gy, gsT)
    got = kda.kda_conv_bwd(xd.view(B, T, D), wd, bd, sd, gyd.view(B, T, D), gsd, silu=silu)
    kda.kda_check()
    args = (f64(x), f64(w), f64(b), cu, f64(s0), silu, f64(gy), f64(gsT))
    for a, r, m in zip(got, om.conv(*args), om.conv(*args, absolute=True)):
        if a is not None:
            _close(a.reshape(r.shape), r, m, 64 + B * T / 8)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("W", [3, 4])
def test_conv_varlen_bwd(lens, W):
    D = 40
    x, w, b, s0, gy, gsT, cu = _inputs(lens, D, W, torch.float32, len(lens) + W)
    xd, wd, bd, sd, gyd, gsd = _dev(x, w, b, s0, gy, gsT)
    cud = torch.from_numpy(cu).to(DEV)
    got = kda.kda_conv_varlen_bwd(xd, wd, bd, cud, sd, gyd, gsd)
    kda.kda_check()
    args = (f64(x), f64(w), f64(b), cu, f64(s0), True, f64(gy), f64(gsT))
    for a, r, m in zip(got, om.conv(*args), om.conv(*args, absolute=True)):
        _close(a, r, m, 64 + sum(lens) / 8)
    none = kda.kda_conv_varlen_bwd(xd, wd, bd, cud, None, gyd, None, want_initial_state_grad=False)
    args = (f64(x), f64(w), f64(b), cu, None, True, f64(gy), None)
    assert none[3] is None
    for a, r, m in zip(none[:3], om.conv(*args), om.conv(*args, absolute=True)):
        _close(a, r, m, 64 + sum(lens) / 8)


def test_conv_gradient_against_differences():
    """The directional derivative of the forward (fp32 outputs, loss summed in fp64)
    agrees with the gradient: step h = 2^-5, third-order term h^2 and the outputs'
    rounding 2^-24 sqrt(T D) / h both below 1e-3 of the derivative's scale."""
    T, D, W, h = 90, 64, 4, 2.0 ** -5
    x, w, b, s0, gy, _, _ = _inputs([T], D, W, torch.float32, 77)
    xd, wd, bd, sd, gyd = _dev(x, w, b, s0, gy)
    g = torch.Generator().manual_seed(1)
    dx, dw = _dev(torch.randn(x.shape, generator=g), torch.randn(w.shape, generator=g) * 0.1)

    def loss(k):
        y, _ = kda.kda_conv_fwd((xd + k * h * dx)[None], wd + k * h * dw, bd, sd)
        return (y[0].double() * gyd.double()).sum().item()
    got = kda.kda_conv_bwd(xd[None], wd, bd, sd, gyd[None])
    want = (got[0][0].double() * dx).sum().item() + (got[1].double() * dw).sum().item()
    scale = (got[0][0].double() * dx).norm().item() + (got[1].double() * dw).norm().item()
    fd = (8 * (loss(1) - loss(-1)) - (loss(2) - loss(-2))) / (12 * h)   # fourth order
    assert abs(fd - want) <= 1e-3 * scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_prompt_then_steps(W, dtype):
    """Steps continue a prompt exactly as one longer prompt."""
    N, T, D = 5, 9, 72
    x, w, b, s0, _, _, _ = _inputs([T] * N, D, W, dtype, 11 + W)
    xd, wd, bd, sd = _dev(x.view(N, T, D), w, b, s0)
    y, sT = kda.kda_conv_fwd(xd, wd, bd, sd)
    for cut in (0, 1, 6):
        state = sd.clone()
        if cut:
            yc, _ = kda.kda_conv_fwd(xd[:, :cut].contiguous(), wd, bd, state, final_state=state)   # in place
            assert torch.equal(yc, y[:, :cut])
        for t in range(cut, T):
            assert (kda.kda_conv_step(xd[:, t], wd, bd, state).float() - y[:, t].float()).abs().max() <= (
                2.0 ** -6 if dtype == torch.bfloat16 else 1e-5)   # one bf16 step of values below 4
        assert torch.equal(state, sT)


def test_conv_step_against_oracle():
    for N, D, W, dtype in ((1, 8, 4, torch.bfloat16), (7, 1032, 3, torch.float32), (300, 64, 2, torch.bfloat16)):
        x, w, b, s0, _, _, cu = _inputs([1] * N, D, W, dtype, N)
        xd, wd, bd, sd = _dev(x, w, b, s0)
        y = kda.kda_conv_step(xd, wd, bd, sd, o_dtype=torch.float32, silu=D != 64)
        args = (f64(x), f64(w), f64(b), cu, f64(s0), D != 64)
        ref, ref_s = om.conv(*args)
        _close(y, ref, om.conv(*args, absolute=True)[0], 32)
        assert np.array_equal(f64(sd), ref_s)


def test_conv_column_slice():
    """x as a column slice of a wider projection, dense, packed, per token and backward."""
    B, T, D, W = 2, 33, 64, 4
    x, w, b, s0, gy, _, cu = _inputs([T] * B, D, W, torch.bfloat16, 21)
    xd, wd, bd, sd, gyd = _dev(x.view(B, T, D), w, b, s0, gy.view(B, T, D))
    wide = torch.full((B, T, 3 * D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[..., D:2 * D] = xd
    part = wide[..., D:2 * D]
    y, sT = kda.kda_conv_fwd(xd, wd, bd, sd)
    y2, sT2 = kda.kda_conv_fwd(part, wd, bd, sd)
    assert torch.equal(y, y2) and torch.equal(sT, sT2)
    cud = torch.from_numpy(cu).to(DEV)
    y3, _ = kda.kda_conv_varlen_fwd(wide.view(B * T, 3 * D)[:, D:2 * D], wd, bd, cud, sd)
    assert torch.equal(y3.view(B, T, D), y)
    for a, c in zip(kda.kda_conv_bwd(xd, wd, bd, sd, gyd), kda.kda_conv_bwd(part, wd, bd, sd, gyd)):
        assert torch.equal(a, c)
    s1, s2 = sd.clone(), sd.clone()
    assert torch.equal(kda.kda_conv_step(xd[:, 3], wd, bd, s1), kda.kda_conv_step(part[:, 3], wd, bd, s2))
    assert torch.equal(s1, s2)
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(part[:, ::2], wd, bd, sd)[0]     # the batch stride does not follow the token stride
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(wide[..., 1:D + 1], wd, bd, sd)  # not 16-byte aligned


def test_conv_rows_of_no_sequence():
    """Rows behind the last sequence stay as they were (their gradient is zero); a
    sequence that leaves the token axis is skipped and reported."""
    D, W, T = 16, 4, 50
    x, w, b, s0, gy, gsT, _ = _inputs([T, 0, 0], D, W, torch.float32, 31)
    xd, wd, bd, sd, gyd, gsd = _dev(x, w, b, s0, gy, gsT)
    for cu, good in (([0, 10, 30, 40], [0, 10, 30, 40]), ([0, 10, 30, 60], [0, 10, 30]), ([-5, 10, 30, 40], None)):
        cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
        y = torch.full((T, D), float("nan"), device=DEV)
        y, sT = kda.kda_conv_varlen_fwd(xd, wd, bd, cud, sd, y=y)
        if good is None or len(good) < 4:
            with pytest.raises(kda.KdaError):
                kda.kda_check()
        kda.kda_check()
        gx, _, _, gs0 = kda.kda_conv_varlen_bwd(xd, wd, bd, cud, sd, gyd, gsd)
        if good is None or len(good) < 4:
            with pytest.raises(kda.KdaError):
                kda.kda_check()
        kda.kda_check()
        if good is None:
            assert torch.isnan(y[:10]).all() and torch.isfinite(y[10:40]).all() and torch.isnan(y[40:]).all()
            assert torch.equal(sT[0], sd[0]) and torch.equal(gs0[0], gsd[0])
            assert (gx[:10] == 0).all() and (gx[40:] == 0).all()
            continue
        end = good[-1]
        ref, _ = om.conv(f64(x), f64(w), f64(b), good, f64(s0))
        mag, _ = om.conv(f64(x), f64(w), f64(b), good, f64(s0), absolute=True)
        _close(y[:end], ref[:end], mag[:end], 32)
        assert torch.isnan(y[end:]).all() and (gx[end:] == 0).all()
        if len(good) < 4:
            assert torch.equal(sT[2], sd[2]) and torch.equal(gs0[2], gsd[2])


def test_conv_empty_calls():
    D, W = 16, 4
    w = torch.randn(D, W, device=DEV)
    s0 = torch.randn(2, W - 1, D, device=DEV)
    y, sT = kda.kda_conv_fwd(torch.zeros(2, 0, D, device=DEV), w, None, s0)
    assert y.shape == (2, 0, D) and torch.equal(sT, s0)
    gx, gw, gb, gs0 = kda.kda_conv_bwd(torch.zeros(2, 0, D, device=DEV), w, None, s0, torch.zeros(2, 0, D, device=DEV), s0)
    assert (gw == 0).all() and torch.equal(gs0, s0)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    y, sT = kda.kda_conv_varlen_fwd(torch.zeros(0, D, device=DEV), w, None, cu)
    assert (sT == 0).all()
    assert kda.kda_conv_step(torch.zeros(0, D, device=DEV), w, None, torch.zeros(0, W - 1, D, device=DEV)).shape == (0, D)


def test_conv_non_finite_inputs_stay_in_their_reach():
    """A NaN input reaches the W outputs that read it and no other, in both directions."""
    T, D, W = 40, 8, 4
    x, w, b, _, gy, _, _ = _inputs([20, 20], D, W, torch.float32, 41)
    x[10, 3], x[18, 5], gy[12, 1] = float("nan"), float("inf"), float("nan")
    xd, wd, bd, gyd = _dev(x.view(2, 20, D), w, b, gy.view(2, 20, D))
    y, _ = kda.kda_conv_fwd(xd, wd, bd, silu=False)
    bad = ~torch.isfinite(y.view(T, D))
    assert bad[10:14, 3].all() and bad[18:20, 5].all() and bad.sum() == 6
    gx, _, _, _ = kda.kda_conv_bwd(xd, wd, bd, None, gyd)
    bad = ~torch.isfinite(gx.view(T, D))
    assert bad[7:14, 3].all() and bad[15:20, 5].all() and bad[9:13, 1].all() and not bad[:, [0, 2, 4, 6, 7]].any()
    assert not bad[20:].any() and bad.sum() == 7 + 5 + 4


def test_conv_streams_and_graphs():
    """A side stream and a captured graph give the eager result; the weight's
    gradient is the same every time."""
    B, T, D, W = 2, 70, 64, 4
    x, w, b, s0, gy, _, _ = _inputs([T] * B, D, W, torch.bfloat16, 51)
    xd, wd, bd, sd, gyd = _dev(x.view(B, T, D), w, b, s0, gy.view(B, T, D))
    y, sT = kda.kda_conv_fwd(xd, wd, bd, sd)
    grads = kda.kda_conv_bwd(xd, wd, bd, sd, gyd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, sT2 = kda.kda_conv_fwd(xd, wd, bd, sd, stream=side)
    grads2 = kda.kda_conv_bwd(xd, wd, bd, sd, gyd, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(sT, sT2) and all(torch.equal(a, c) for a, c in zip(grads, grads2))
    graph = torch.cuda.CUDAGraph()
    state = sd.clone()
    with torch.cuda.graph(graph):
        y3, _ = kda.kda_conv_fwd(xd, wd, bd, sd)
        grads3 = kda.kda_conv_bwd(xd, wd, bd, sd, gyd)
        y4 = kda.kda_conv_step(xd[:, 0], wd, bd, state)
    for _ in range(2):
        state.copy_(sd)
        y3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y) and all(torch.equal(a, c) for a, c in zip(grads, grads3))
        assert (y4.float() - y[:, 0].float()).abs().max() <= 2.0 ** -6
    del graph
