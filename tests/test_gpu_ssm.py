"""GPU: the selective scan (kda_ssm_*) against the fp64 oracle.

Tolerance.  Arithmetic is fp32 from the exact input values.  Every term of every
sum carries at most 2 T decays (forward and gradient), each off by at most 2^-21
relative (ex2.approx 2 ulp = 2^-22, and its argument, at most 2 here, rounded
twice: 2 * 2 ln 2 * 2^-24 < 2^-22), about 32 further roundings of 2^-23 (softplus,
sigmoid, products), and at most n additions of 2^-24 each, n the terms of its
longest sum (S states, D channels, T tokens).  So |error| <= (2 T + 16 + n / 8)
2^-21 times the sum of the terms' absolute values (the oracle with
absolute=True).  A bf16 output adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle.mixer as om
import gated_delta_rule_133_b200 as kda
from tests._helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "s0")
GRADS = ("gx", "gdt", "gA", "gB", "gC", "gskip", "gz", "gdt_bias", "gs0")


def _inputs(lens, D, S, G, dtype, seed, z=True, skip=True, bias=True, state=True, fast=False):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def rnd(*shape, s=1.0):
        return torch.randn(*shape, generator=g) * s
    p = {"x": rnd(T, D).to(dtype), "dt": rnd(T, D).to(dtype) - (0.0 if fast else 2.0),
         "A": -torch.rand(D, S, generator=g) * (20.0 if fast else 1.5),
         "B": rnd(T, G, S).to(dtype), "C": rnd(T, G, S).to(dtype), "skip": rnd(D) if skip else None,
         "z": rnd(T, D).to(dtype) if z else None, "dt_bias": rnd(D, s=0.3) if bias else None,
         "s0": rnd(N, D, S) if state else None}
    p["dt"] = p["dt"].to(dtype)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return p, cu, rnd(T, D), rnd(N, D, S)


def _f(p):
    return {k: f64(v) for k, v in p.items()}


def _dev(p):
    return {k: None if v is None else v.to(DEV) for k, v in p.items()}


def _lead(d, B, T):
    """Dense layout of the token-major tensors."""
    return {k: v.view(B, T, *v.shape[1:]) if v is not None and k in ("x", "dt", "B", "C", "z") else v
            for k, v in d.items()}


def _fwd(d, cu=None, **kw):
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    b = (d["skip"], d["z"], d["dt_bias"], d["s0"])
    return kda.kda_ssm_fwd(*a, *b, **kw) if cu is None else kda.kda_ssm_varlen_fwd(*a, cu, *b, **kw)


def _bwd(d, gy, gsT, cu=None, **kw):
    a = (d["x"], d["dt"], d["A"], d["B"], d["C"])
    b = (d["skip"], d["z"], d["dt_bias"], d["s0"], gy, gsT)
    return kda.kda_ssm_bwd(*a, *b, **kw) if cu is None else kda.kda_ssm_varlen_bwd(*a, cu, *b, **kw)


def _close(got, ref, mag, T, n, rounded=False, name=""):
    got = f64(got).reshape(ref.shape)
    e = (2 * T + 16 + n / 8) * 2.0 ** -21 * mag
    bound = e + (2.0 ** -8 * (np.abs(ref) + e) if rounded else 0) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (name, bad.sum(), bad.size, np.abs(got - ref).max(), np.argwhere(bad)[:3])


def _check_fwd(p, cu, got, kw, rounded=False):
    longest = int(np.diff(cu).max())
    for name, a, r, m in zip(("y", "state"), got, om.ssm(**_f(p), cu=cu, **kw), om.ssm(**_f(p), cu=cu, **kw, absolute=True)):
        _close(a, r, m, longest, p["A"].shape[1], rounded and name == "y", name)


def _check_bwd(p, cu, got, gy, gsT, kw=None):
    kw = kw or {}
    T, D = p["x"].shape
    longest = int(np.diff(cu).max())
    args = dict(_f(p), cu=cu, gy=f64(gy), gsT=f64(gsT), **kw)
    for name, a, r, m in zip(GRADS, got, om.ssm(**args), om.ssm(**args, absolute=True)):
        if a is not None:
            _close(a, r, m, longest, max(T, D), False, name)


# B, T, D, S, G
DENSE = [(2, 37, 24, 16, 1), (1, 1, 8, 16, 1), (3, 2, 64, 32, 2), (1, 130, 264, 16, 1), (2, 65, 48, 64, 2),
         (1, 33, 2064, 16, 2), (1, 96, 1600, 32, 1), (5, 31, 2048, 16, 1), (9, 7, 1040, 64, 1)]


@pytest.mark.parametrize("dtype,o_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                           (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("B,T,D,S,G", DENSE)
def test_ssm_fwd(B, T, D, S, G, dtype, o_dtype):
    p, cu, _, _ = _inputs([T] * B, D, S, G, dtype, T + D, z=T != 130, skip=T != 65, bias=T != 37, state=B < 3)
    got = _fwd(_lead(_dev(p), B, T), o_dtype=o_dtype)
    kda.kda_check()
    _check_fwd(p, cu, (got[0].view(B * T, D), got[1]), {}, o_dtype == torch.bfloat16)


LENS = [[5, 0, 1, 2, 70, 3], [1], [0, 0, 4], [64, 32, 1, 63, 33], [1] * 40, [300]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("S,G", [(16, 1), (32, 2), (64, 1)])
def test_ssm_varlen_fwd(lens, S, G, dtype):
    p, cu, _, _ = _inputs(lens, 48, S, G, dtype, len(lens) + S)
    got = _fwd(_dev(p), torch.from_numpy(cu).to(DEV), o_dtype=torch.float32)
    kda.kda_check()
    _check_fwd(p, cu, got, {})


def test_ssm_step_size_without_softplus_and_strong_decay():
    for fast, softplus in ((False, False), (True, True)):
        p, cu, gy, gsT = _inputs([50, 20], 32, 16, 1, torch.float32, 5, fast=fast)
        if not softplus:
            p["dt"], p["dt_bias"] = p["dt"].abs() * 0.1, p["dt_bias"].abs() * 0.1
        d, cud = _dev(p), torch.from_numpy(cu).to(DEV)
        got = _fwd(d, cud, softplus=softplus)
        kda.kda_check()
        # decays up to e^-60: an argument of |v| moves e^-v by |v| 2^-24 relative, |v| e^-|v| < 0.4 of the term
        _check_fwd(p, cu, got, {"use_softplus": softplus})


@pytest.mark.parametrize("N,D,S,G,dtype", [(1, 8, 16, 1, torch.bfloat16), (5, 2056, 16, 1, torch.bfloat16),
                                           (300, 64, 32, 4, torch.float32), (3, 1040, 64, 2, torch.bfloat16)])
def test_ssm_step(N, D, S, G, dtype):
    p, cu, _, _ = _inputs([1] * N, D, S, G, dtype, N + D, z=N != 5, skip=N != 3, bias=N != 300)
    d = _dev(p)
    y = kda.kda_ssm_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["s0"], d["skip"], d["z"], d["dt_bias"],
                         o_dtype=torch.float32)
    _check_fwd(p, cu, (y, d["s0"]), {})


@pytest.mark.parametrize("S", [16, 64])
def test_ssm_prompt_then_steps(S):
    """A prompt cut anywhere and continued by steps: the states' decays differ by
    roundings only (the tolerance of a run of T tokens)."""
    N, T, D = 2, 12, 64
    p, cu, _, _ = _inputs([T] * N, D, S, 1, torch.bfloat16, 8)
    d = _lead(_dev(p), N, T)
    ref, ref_s = om.ssm(**_f(p), cu=cu)
    mag, mag_s = om.ssm(**_f(p), cu=cu, absolute=True)
    for cut in (1, 5, 11):
        h = {k: v[:, :cut].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in d.items()}
        state = d["s0"].clone()
        h["s0"] = state
        y, _ = _fwd(h, final_state=state, o_dtype=torch.float32)
        ys = [y]
        for t in range(cut, T):
            ys.append(kda.kda_ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], state,
                                       d["skip"], d["z"][:, t], d["dt_bias"], o_dtype=torch.float32)[:, None])
        _close(torch.cat(ys, 1).reshape(N * T, D), ref, mag, T, S)
        _close(state, ref_s, mag_s, T, S)


def test_ssm_column_slices():
    """x, dt, z, B, C as column slices of wider projections."""
    B, T, D, S = 2, 33, 64, 16
    p, cu, gy, gsT = _inputs([T] * B, D, S, 1, torch.bfloat16, 9)
    d = _lead(_dev(p), B, T)
    proj = torch.full((B, T, 2 * D + 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    proj[..., 8:8 + D], proj[..., 16 + D:16 + 2 * D] = d["x"], d["z"]
    small = torch.full((B, T, D + 8 + 2 * S), float("nan"), dtype=torch.bfloat16, device=DEV)
    small[..., :D], small[..., D:D + S], small[..., D + S + 8:] = d["dt"], d["B"][:, :, 0], d["C"][:, :, 0]
    e = dict(d, x=proj[..., 8:8 + D], z=proj[..., 16 + D:16 + 2 * D], dt=small[..., :D],
             B=small[..., D:D + S].unsqueeze(2), C=small[..., D + S + 8:].unsqueeze(2))
    for a, c in zip(_fwd(d), _fwd(e)):
        assert torch.equal(a, c)
    g = gy.to(DEV).view(B, T, D)
    for a, c in zip(_bwd(d, g, gsT.to(DEV)), _bwd(e, g, gsT.to(DEV))):
        assert torch.equal(a, c)
    s1, s2 = d["s0"].clone(), d["s0"].clone()
    y1, y2 = (kda.kda_ssm_step(q["x"][:, 2], q["dt"][:, 2], q["A"], q["B"][:, 2], q["C"][:, 2], s, q["skip"],
                               q["z"][:, 2], q["dt_bias"]) for q, s in ((d, s1), (e, s2)))
    assert torch.equal(y1, y2) and torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D,S,G", DENSE)
def test_ssm_bwd(B, T, D, S, G, dtype):
    p, cu, gy, gsT = _inputs([T] * B, D, S, G, dtype, T + D, z=T != 130, skip=T != 65, bias=T != 37, state=B < 3)
    got = _bwd(_lead(_dev(p), B, T), gy.to(DEV).view(B, T, D), gsT.to(DEV) if T != 96 else None)
    kda.kda_check()
    _check_bwd(p, cu, got, gy, gsT if T != 96 else None)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("S,G", [(16, 1), (32, 2), (64, 1)])
def test_ssm_varlen_bwd(lens, S, G):
    p, cu, gy, gsT = _inputs(lens, 48, S, G, torch.float32, len(lens) + S)
    got = _bwd(_dev(p), gy.to(DEV), gsT.to(DEV), torch.from_numpy(cu).to(DEV))
    kda.kda_check()
    _check_bwd(p, cu, got, gy, gsT)


def test_ssm_many_sequences():
    lens = [(7 * i) % 5 for i in range(700)]
    p, cu, gy, gsT = _inputs(lens, 32, 16, 1, torch.float32, 5)
    d, cud = _dev(p), torch.from_numpy(cu).to(DEV)
    got = _fwd(d, cud)
    grads = _bwd(d, gy.to(DEV), gsT.to(DEV), cud)
    kda.kda_check()
    _check_fwd(p, cu, got, {})
    _check_bwd(p, cu, grads, gy, gsT)


@pytest.mark.parametrize("S,G,dtype", [(16, 1, torch.bfloat16), (32, 3, torch.float32), (64, 1, torch.bfloat16)])
def test_ssm_bwd_of_many_short_sequences(S, G, dtype):
    """Blocks of four warps, several sequences each: lengths of less than one turn, of
    many rounds of turns and of zero, a channel tile that is not full."""
    lens = [(13 * i) % 9 for i in range(450)]
    lens[7], lens[300] = 150, 33
    p, cu, gy, gsT = _inputs(lens, 264, S, G, dtype, 46)
    d, cud = _dev(p), torch.from_numpy(cu).to(DEV)
    grads = _bwd(d, gy.to(DEV), gsT.to(DEV), cud)
    again = _bwd(d, gy.to(DEV), gsT.to(DEV), cud)
    kda.kda_check()
    _check_bwd(p, cu, grads, gy, gsT)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_ssm_backward_without_softplus():
    p, cu, gy, gsT = _inputs([40, 7], 32, 16, 2, torch.float32, 5)
    p["dt"], p["dt_bias"] = p["dt"].abs() * 0.1, p["dt_bias"].abs() * 0.1
    got = _bwd(_dev(p), gy.to(DEV), gsT.to(DEV), torch.from_numpy(cu).to(DEV), softplus=False)
    _check_bwd(p, cu, got, gy, gsT, {"use_softplus": False})


def test_ssm_gradient_against_differences():
    """Directional derivatives of the forward agree with the gradients: fourth-order
    differences of step h = 2^-5, whose error (h^4 and outputs' rounding over h) stays
    below 2e-3 of the derivative's scale."""
    T, D, S, h = 40, 32, 16, 2.0 ** -5
    p, cu, gy, gsT = _inputs([T], D, S, 1, torch.float32, 12)
    d = _lead(_dev(p), 1, T)
    gyd, gsd = gy.to(DEV).view(1, T, D), gsT.to(DEV)
    got = dict(zip(NAMES, _bwd(d, gyd, gsd)))
    gen = torch.Generator().manual_seed(3)
    for name in NAMES:
        step = torch.randn(d[name].shape, generator=gen).to(DEV) * (0.1 if name == "A" else 1.0)
        if name == "A":
            step = -step.abs() * d["A"].abs().clamp(max=0.1)

        def loss(k):
            y, s = _fwd(dict(d, **{name: d[name] + k * h * step}))
            return ((y.double() * gyd).sum() + (s.double() * gsd).sum()).item()
        want = (got[name].double() * step).sum().item()
        scale = (got[name].double() * step).norm().item()
        fd = (8 * (loss(1) - loss(-1)) - (loss(2) - loss(-2))) / (12 * h)
        assert abs(fd - want) <= 2e-3 * scale + 1e-3, (name, fd, want, scale)


def test_ssm_rows_of_no_sequence():
    D, S, T = 16, 16, 50
    p, _, gy, gsT = _inputs([T, 0, 0], D, S, 1, torch.float32, 31)
    d, gyd, gsd = _dev(p), gy.to(DEV), gsT.to(DEV)
    for cu, end in (([0, 10, 30, 40], 40), ([0, 10, 30, 60], 30)):
        cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
        ok = [min(c, end) for c in cu]
        y = torch.full((T, D), float("nan"), device=DEV)
        _, sT = _fwd(d, cud, y=y)
        if end == 30:
            with pytest.raises(kda.KdaError):
                kda.kda_check()
            assert torch.equal(sT[2], d["s0"][2])
        grads = _bwd(d, gyd, gsd, cud)
        if end == 30:
            with pytest.raises(kda.KdaError):
                kda.kda_check()
            assert torch.equal(grads[8][2], gsd[2])
        kda.kda_check()
        assert torch.isfinite(y[:end]).all() and torch.isnan(y[end:]).all()
        f = _f(p)
        cut = {k: v[:end] if k in ("x", "dt", "B", "C", "z") else v for k, v in p.items()}
        _check_bwd(cut, np.array(ok), [g[:end] if i in (0, 1, 3, 4, 6) else g for i, g in enumerate(grads)], gy[:end], gsT)
        for i in (0, 1, 3, 4, 6):
            assert (grads[i][end:] == 0).all(), GRADS[i]


def test_ssm_empty_calls():
    D, S = 16, 16
    z = torch.zeros(2, 0, D, device=DEV)
    bc = torch.zeros(2, 0, 1, S, device=DEV)
    A, s0 = -torch.ones(D, S, device=DEV), torch.randn(2, D, S, device=DEV)
    y, sT = kda.kda_ssm_fwd(z, z, A, bc, bc, None, None, None, s0)
    assert y.shape == (2, 0, D) and torch.equal(sT, s0)
    g = kda.kda_ssm_bwd(z, z, A, bc, bc, None, None, None, s0, z, s0)
    assert (g[2] == 0).all() and torch.equal(g[8], s0)


def test_ssm_non_finite_inputs_stay_in_their_channel_and_future():
    T, D, S = 40, 16, 16
    p, cu, gy, _ = _inputs([T], D, S, 1, torch.float32, 41)
    p["x"][10, 3] = float("nan")
    p["x"][20, 5] = float("inf")
    d = _lead(_dev(p), 1, T)
    y, sT = _fwd(d)
    bad = ~torch.isfinite(y[0])
    assert bad[10:, 3].all() and bad[20:, 5].all() and bad.sum() == 30 + 20
    assert not torch.isfinite(sT[0, 3]).any() and torch.isfinite(sT[0, [0, 1, 2, 4, 6]]).all()


@pytest.mark.parametrize("mask", [float("-inf"), torch.finfo(torch.bfloat16).min, -1e4])
def test_ssm_masked_tokens_leave_the_state(mask):
    """A step size of softplus(-inf), of the type's lowest value or of a large negative
    number is zero: the state passes the token unchanged (prompt and step), the token's
    gradients of x and dt are those of the skip and zero."""
    T, D, S = 30, 16, 16
    p, cu, gy, gsT = _inputs([T], D, S, 1, torch.bfloat16, 43, bias=False)
    masked = [0, 7, 8, 21, T - 1]
    p["dt"][masked] = mask
    q = dict(p, dt=p["dt"].clone())
    q["dt"][masked] = -1e4                       # for the oracle: softplus(-1e4) = 0 in 64 bits
    d = _lead(_dev(p), 1, T)
    y, sT = _fwd(d, o_dtype=torch.float32)
    _check_fwd(q, cu, (y[0], sT), {})
    grads = _bwd(d, gy.to(DEV).view(1, T, D), gsT.to(DEV))
    _check_bwd(q, cu, grads, gy, gsT)
    assert (grads[1][0, masked] == 0).all()
    state = d["s0"].clone()
    out = kda.kda_ssm_step(d["x"][:, 7], d["dt"][:, 7], d["A"], d["B"][:, 7], d["C"][:, 7], state, d["skip"], d["z"][:, 7])
    assert torch.equal(state, d["s0"]) and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("T", [1, 7, 8, 30])
def test_ssm_infinite_decay_rate(T):
    """A state with A = -inf forgets everything at a token whose step size is above zero
    and keeps all of it at a masked one, whatever the length's remainder is."""
    D, S = 16, 16
    p, cu, gy, gsT = _inputs([T], D, S, 1, torch.bfloat16, 45, bias=False)
    p["A"][1, 3] = p["A"][5] = float("-inf")
    p["A"][7, 2] = torch.finfo(torch.float32).min
    q = dict(p, A=p["A"].clone().clamp(min=-1e8), dt=p["dt"].clone())   # exp(-1e8 Delta) = 0 in 64 bits, Delta > 1e-5
    for t in ([0] if T == 1 else [0, 3, T - 1]):
        p["dt"][t] = float("-inf")
        q["dt"][t] = -1e4
    d = _lead(_dev(p), 1, T)
    y, sT = _fwd(d, o_dtype=torch.float32)
    _check_fwd(q, cu, (y[0], sT), {})
    _check_bwd(q, cu, _bwd(d, gy.to(DEV).view(1, T, D), gsT.to(DEV)), gy, gsT)
    state = d["s0"].clone()
    kda.kda_ssm_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], state, d["skip"], d["z"][:, 0])
    assert torch.equal(state, d["s0"])


def test_ssm_nan_step_size_is_not_hidden():
    p, cu, _, _ = _inputs([12], 16, 16, 1, torch.float32, 44)
    p["dt"][5, 2] = float("nan")
    y, sT = _fwd(_lead(_dev(p), 1, 12))
    bad = ~torch.isfinite(y[0])
    assert bad[5:, 2].all() and bad.sum() == 7 and torch.isnan(sT[0, 2]).all()


def test_ssm_step_beyond_the_grid():
    """More sequences than one grid holds: every one is advanced."""
    N, D, S = 70000 * 4, 8, 16
    x = torch.ones(N, D, device=DEV)
    state = torch.arange(N, device=DEV, dtype=torch.float32).view(N, 1, 1).expand(N, D, S).contiguous()
    zero = torch.zeros(D, S, device=DEV)
    y = kda.kda_ssm_step(x, x, zero, torch.ones(N, 1, S, device=DEV), torch.ones(N, 1, S, device=DEV), state, softplus=False)
    want = torch.arange(N, device=DEV, dtype=torch.float32) + 1      # exact: decay 2^0, input 1, below 2^24
    assert torch.equal(state, want.view(N, 1, 1).expand(N, D, S))
    assert torch.equal(y, (want * S).view(N, 1).expand(N, D))


def test_ssm_streams_graphs_and_dirty_workspace():
    """A side stream, a captured graph and a workspace full of garbage give the
    eager result, bit for bit, forward and backward."""
    B, T, D, S = 2, 150, 64, 16
    p, cu, gy, gsT = _inputs([T] * B, D, S, 1, torch.bfloat16, 51)
    d = _lead(_dev(p), B, T)
    gyd, gsd = gy.to(DEV).view(B, T, D), gsT.to(DEV)
    y, sT = _fwd(d)
    grads = _bwd(d, gyd, gsd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, _ = _fwd(d, stream=side)
    grads2 = _bwd(d, gyd, gsd, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, c) for a, c in zip(grads, grads2))
    ws = torch.full((kda.ssm_bwd_workspace_size(B, T, D, S),), 0xFF, dtype=torch.uint8, device=DEV)
    assert all(torch.equal(a, c) for a, c in zip(grads, _bwd(d, gyd, gsd, workspace=ws)))
    graph = torch.cuda.CUDAGraph()
    state = d["s0"].clone()
    with torch.cuda.graph(graph):
        y3, _ = _fwd(d)
        grads3 = _bwd(d, gyd, gsd)
        y4 = kda.kda_ssm_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], state, d["skip"],
                              d["z"][:, 0], d["dt_bias"])
    for _ in range(2):
        state.copy_(d["s0"])
        y3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y) and all(torch.equal(a, c) for a, c in zip(grads, grads3))
        assert torch.isfinite(y4.float()).all()
    del graph
