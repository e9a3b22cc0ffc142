"""GPU: the launch shapes of the short convolution and the selective scan that larger
sizes reach: longer tiles, several sequences per thread or per block, offsets beyond
32 bits, calls at the same time.

Tolerances are those of the operators' own tests (test_gpu_conv.py, test_gpu_ssm.py),
with the same derivation.  A weight's gradient is a sum of at most 128 tokens in order
per tile, then of the tiles in 32 strands and of those in 5 levels: at most 128 + 1 +
tiles / 32 + 5 additions, fewer than T / 8 + 32 for every T here.

Large cases with few distinct values: channels of the convolution do not meet, so its
channels repeat 40 distinct ones (40 divides no block of channels) and the oracle
computes those.  Groups of the scan do not meet either, and the oracle computes some."""
import numpy as np
import pytest
import torch

import oracle.mixer as om
import gated_delta_rule_133_b200 as kda
from tests._helpers import f64
from tests.test_gpu_conv import _close as conv_close
from tests.test_gpu_conv import _inputs as conv_inputs
from tests.test_gpu_ssm import GRADS, _bwd, _check_fwd, _dev, _fwd, _inputs, _lead
from tests.test_gpu_ssm import _close as ssm_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
P = 40


def _spread(t, D, dim=-1):
    """Channels c of t repeated: channel i of the result is i % P of t."""
    return None if t is None else t.index_select(dim % t.dim(), torch.arange(D) % P).contiguous()


def _conv_case(lens, D, W, dtype, seed):
    x, w, b, s0, gy, gsT, cu = conv_inputs(lens, P, W, dtype, seed)
    small = (f64(x), f64(w), f64(b), cu, f64(s0))
    dev = [_spread(t, D).to(DEV) for t in (x, b, s0, gy, gsT)]
    return small, (f64(gy), f64(gsT)), (dev[0], _spread(w, D, 0).to(DEV), *dev[1:]), torch.from_numpy(cu).to(DEV)


# tokens / tile x threads per tile row against 256 threads per SM: with 2048 channels
# tiles of 16 from 1184 tokens on, of 32 from 2368, of 64 from 4736, of 128 from 9472
RAGGED = {16: [601, 0, 1, 17, 300, 2, 479], 32: [1203, 0, 1, 33, 800, 3, 560], 64: [2000, 0, 65, 1, 2, 2731, 201],
          128: [5003, 0, 129, 1, 127, 3, 4337]}


@pytest.mark.parametrize("dtype,o_dtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("tile,W", [(16, 4), (32, 4), (32, 3), (32, 2)])
def test_conv_fwd_longer_tiles(tile, W, dtype, o_dtype):
    lens, D = RAGGED[tile], 2048
    args, _, (x, w, b, s0, _, _), cu = _conv_case(lens, D, W, dtype, 60 + tile + W)
    y, sT = kda.kda_conv_varlen_fwd(x, w, b, cu, s0, o_dtype=o_dtype)
    kda.kda_check()
    ch = np.arange(D) % P
    ref, ref_s = om.conv(*args)
    mag = om.conv(*args, absolute=True)[0]
    conv_close(y, ref[:, ch], mag[:, ch], 32, o_dtype == BF16)
    assert np.array_equal(f64(sT), ref_s[..., ch])
    T = sum(lens) // 2   # the same tokens as two equal sequences
    y, sT = kda.kda_conv_fwd(x.view(2, T, D), w, b, s0[:2].contiguous(), o_dtype=o_dtype, silu=False)
    kda.kda_check()
    dense = (args[0], args[1], args[2], np.array([0, T, 2 * T]), args[4][:2], False)
    ref, ref_s = om.conv(*dense)
    conv_close(y.view(2 * T, D), ref[:, ch], om.conv(*dense, absolute=True)[0][:, ch], 32, o_dtype == BF16)
    assert np.array_equal(f64(sT), ref_s[..., ch])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tile,W,silu", [(16, 4, True), (32, 3, True), (32, 2, False), (64, 4, True), (64, 4, False),
                                         (128, 4, True)])
def test_conv_bwd_longer_tiles(tile, W, silu, dtype):
    lens, D = RAGGED[tile], 2048
    args, grads, (x, w, b, s0, gy, gsT), cu = _conv_case(lens, D, W, dtype, 160 + tile + W)
    got = kda.kda_conv_varlen_bwd(x, w, b, cu, s0, gy, gsT, silu=silu)
    again = kda.kda_conv_varlen_bwd(x, w, b, cu, s0, gy, gsT, silu=silu)
    kda.kda_check()
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    ch = np.arange(D) % P
    ref, mag = om.conv(*args, silu, *grads), om.conv(*args, silu, *grads, absolute=True)
    for i, (a, r, m) in enumerate(zip(got, ref, mag)):
        at = (ch,) if i in (1, 2) else (Ellipsis, ch)
        conv_close(a, r[at], m[at], 64 + sum(lens) / 8)
    T = sum(lens) // 2
    dense = (args[0], args[1], args[2], np.array([0, T, 2 * T]), None, silu, grads[0], None)
    got = kda.kda_conv_bwd(x.view(2, T, D), w, b, None, gy.view(2, T, D), silu=silu)
    for i, (a, r, m) in enumerate(zip(got, om.conv(*dense), om.conv(*dense, absolute=True))):
        at = (ch,) if i in (1, 2) else (Ellipsis, ch)
        conv_close(a.reshape(r[at].shape), r[at], m[at], 64 + sum(lens) / 8)


@pytest.mark.parametrize("lens", [[5, 0, 1, 2, 70, 3], [64, 64, 1, 63], [1] * 40, [300]])
def test_conv_packed_bwd_bf16(lens):
    D, W = 40, 4
    x, w, b, s0, gy, gsT, cu = conv_inputs(lens, D, W, BF16, len(lens))
    d = [t.to(DEV) for t in (x, w, b, s0, gy, gsT)]
    got = kda.kda_conv_varlen_bwd(*d[:3], torch.from_numpy(cu).to(DEV), *d[3:])
    kda.kda_check()
    args = (f64(x), f64(w), f64(b), cu, f64(s0), True, f64(gy), f64(gsT))
    for a, r, m in zip(got, om.conv(*args), om.conv(*args, absolute=True)):
        conv_close(a, r, m, 64 + sum(lens) / 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,W", [(77, 4), (130, 4), (79, 3), (80, 2)])
def test_conv_step_four_sequences_per_thread(N, W, dtype):
    """4096 channels: four sequences per thread from 76 on, with every remainder."""
    D = 4096
    args, _, (x, w, b, s0, _, _), _ = _conv_case([1] * N, D, W, dtype, N)
    wide = torch.full((N, 3 * D), float("nan"), dtype=dtype, device=DEV)
    wide[:, D:2 * D] = x
    for xs in (x, wide[:, D:2 * D]):
        state = s0.clone()
        y = kda.kda_conv_step(xs, w, b, state, o_dtype=F32)
        kda.kda_check()
        ref, ref_s = om.conv(*args)
        ch = np.arange(D) % P
        conv_close(y, ref[:, ch], om.conv(*args, absolute=True)[0][:, ch], 32)
        assert np.array_equal(f64(state), ref_s[..., ch])


@pytest.mark.parametrize("N,D,S,G,dtype", [(41, 1024, 16, 2, BF16), (38, 1032, 16, 1, F32), (39, 520, 64, 1, BF16),
                                           (21, 2080, 64, 4, F32), (23, 2056, 32, 1, BF16), (40, 1024, 32, 2, F32)])
def test_ssm_step_four_sequences_per_thread(N, D, S, G, dtype):
    """At least 148 blocks of four sequences, with every remainder; dense and as slices."""
    p, cu, _, _ = _inputs([1] * N, D, S, G, dtype, N + D, z=N != 38, skip=N != 39, bias=N != 40)
    d = _dev(p)
    wide = torch.full((N, 2 * D + 2 * G * S + 16), float("nan"), dtype=dtype, device=DEV)
    cols = {"x": (0, D), "dt": (D + 8, D), "B": (2 * D + 8, G * S), "C": (2 * D + G * S + 16, G * S)}
    e = dict(d)
    for k, (at, n) in cols.items():
        wide[:, at:at + n] = d[k].reshape(N, n)
        e[k] = wide[:, at:at + n].view(d[k].shape)
    for q in (d, e):
        state = d["s0"].clone()
        y = kda.kda_ssm_step(q["x"], q["dt"], q["A"], q["B"], q["C"], state, q["skip"], q["z"], q["dt_bias"], o_dtype=F32)
        kda.kda_check()
        _check_fwd(p, cu, (y, state), {})


@pytest.mark.parametrize("S,per,mean,dtype", [(16, 32, 200, BF16), (16, 24, 200, F32), (32, 32, 140, F32),
                                              (64, 24, 75, BF16)])
def test_ssm_bwd_wide_blocks_of_several_sequences(S, per, mean, dtype):
    """Long enough for 12 (8) warps, more sequences than blocks per channel tile (19):
    barriers and carries go on from one sequence to the next, empty and short ones
    among them."""
    G = 32
    D = per * G
    lens = [mean + 7 * i for i in range(20)] + [0, 1, 3 * mean, 9]
    p, cu, gy, gsT = _inputs(lens, D, S, G, dtype, 71 + S)
    d, cud = _dev(p), torch.from_numpy(cu).to(DEV)
    grads = _bwd(d, gy.to(DEV), gsT.to(DEV), cud)
    again = _bwd(d, gy.to(DEV), gsT.to(DEV), cud)
    y, sT = _fwd(d, cud, o_dtype=F32)
    kda.kda_check()
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    T, longest = sum(lens), max(lens)
    by_row, by_state = slice(None), slice(None)
    for g in (0, 13, G - 1):
        ch, gr = slice(g * per, (g + 1) * per), slice(g, g + 1)
        cut = {"x": (by_row, ch), "dt": (by_row, ch), "z": (by_row, ch), "A": ch, "skip": ch, "dt_bias": ch,
               "B": (by_row, gr), "C": (by_row, gr), "s0": (by_state, ch)}
        q = {k: f64(p[k])[c] for k, c in cut.items()}
        kw = dict(q, cu=cu, gy=f64(gy)[:, ch], gsT=f64(gsT)[:, ch])
        where = [cut[k] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "s0")]
        for name, a, at, r, m in zip(GRADS, grads, where, om.ssm(**kw), om.ssm(**kw, absolute=True)):
            ssm_close(a[at], r, m, longest, T, False, name)
        ref, mag = om.ssm(**q, cu=cu), om.ssm(**q, cu=cu, absolute=True)
        ssm_close(y[:, ch], ref[0], mag[0], longest, S, False, "y")
        ssm_close(sT[:, ch], ref[1], mag[1], longest, S, False, "state")


def test_captured_steps_equal_eager_ones():
    """Both steps captured together and replayed: outputs and states of the eager calls."""
    N, D, S = 41, 1024, 16
    p, _, _, _ = _inputs([1] * N, D, S, 1, BF16, 81)
    d = _dev(p)
    w, cs = torch.randn(D, 4, device=DEV), torch.randn(N, 3, D, device=DEV).to(BF16)

    def step(c, h):
        xc = kda.kda_conv_step(d["x"], w, None, c)
        return kda.kda_ssm_step(xc, d["dt"], d["A"], d["B"], d["C"], h, d["skip"], d["z"], d["dt_bias"])
    c1, h1 = cs.clone(), d["s0"].clone()
    want = [step(c1, h1), step(c1, h1)]
    c2, h2 = cs.clone(), d["s0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(c2, h2)
    c2.copy_(cs)
    h2.copy_(d["s0"])
    for w_ in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w_)
    assert torch.equal(c1, c2) and torch.equal(h1, h2)
    del graph


def test_calls_at_the_same_time():
    """Two backward passes on two streams, each with its own workspace, many times over."""
    cases = []
    for seed, T in ((91, 700), (92, 450)):
        p, cu, gy, gsT = _inputs([T] * 2, 256, 16, 1, BF16, seed)
        d = _lead(_dev(p), 2, T)
        w = torch.randn(256, 4, device=DEV)
        gyd, gsd = gy.to(DEV).view(2, T, 256), gsT.to(DEV)
        cases.append((lambda st, d=d, w=w, gyd=gyd, gsd=gsd: (
            *_bwd(d, gyd, gsd, stream=st),
            *[t for t in kda.kda_conv_bwd(d["x"], w, None, None, gyd, stream=st) if t is not None])))
    want = [c(None) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[c(st) for c, st in zip(cases, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    kda.kda_check()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_beyond_32_bits():
    """2^32 elements and more: the rows at the end are those of a call on them alone."""
    D, S, T = 4096, 16, (1 << 20) + 104
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(1, T, D, dtype=BF16, device=DEV).normal_(generator=g)
    w = torch.randn(D, 4, generator=g, device=DEV)
    cut = T - 200
    y, sT = kda.kda_conv_fwd(x, w)
    y1, s1 = kda.kda_conv_fwd(x[:, cut:], w, None, x[:, cut - 3:cut].contiguous())
    assert torch.equal(y[:, cut:], y1) and torch.equal(sT, s1)
    del y, y1
    dt = torch.empty(1, T, D, dtype=BF16, device=DEV).normal_(generator=g)
    dt -= 3
    bc = torch.empty(1, T, 1, S, dtype=BF16, device=DEV).normal_(generator=g)
    A = -torch.rand(D, S, generator=g, device=DEV)
    y, h = kda.kda_ssm_fwd(x, dt, A, bc, bc)
    ya, ha = kda.kda_ssm_fwd(x[:, :cut], dt[:, :cut], A, bc[:, :cut], bc[:, :cut])
    assert torch.equal(y[:, :cut], ya)
    yb, hb = kda.kda_ssm_fwd(x[:, cut:], dt[:, cut:], A, bc[:, cut:], bc[:, cut:], None, None, None, ha)
    assert torch.equal(y[:, cut:], yb) and torch.equal(h, hb)
    kda.kda_check()
    del x, dt, y, ya, yb
    torch.cuda.empty_cache()


def test_gradients_beyond_32_bits():
    """Saved states of more than 2^32 elements: the gradients of a sequence are those of
    its two parts, the second's state gradient handed to the first."""
    D, S, T = 4096, 16, (1 << 19) + 64
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.empty(1, T, D, dtype=BF16, device=DEV).normal_(generator=g)
    dt = torch.empty(1, T, D, dtype=BF16, device=DEV).normal_(generator=g)
    dt -= 3
    B = torch.empty(1, T, 1, S, dtype=BF16, device=DEV).normal_(generator=g)
    C = torch.empty(1, T, 1, S, dtype=BF16, device=DEV).normal_(generator=g)
    gy = torch.empty(1, T, D, device=DEV).normal_(generator=g)
    A = -torch.rand(D, S, generator=g, device=DEV)
    whole = kda.kda_ssm_bwd(x, dt, A, B, C, None, None, None, None, gy)
    kda.kda_check()
    cut = T - 512
    _, h = kda.kda_ssm_fwd(x[:, :cut], dt[:, :cut], A, B[:, :cut], C[:, :cut])
    tail = kda.kda_ssm_bwd(x[:, cut:], dt[:, cut:], A, B[:, cut:], C[:, cut:], None, None, None, h, gy[:, cut:])
    for i in (0, 1, 3, 4):
        assert torch.equal(whole[i][:, cut:], tail[i]), GRADS[i]
    near = cut - 4096
    _, h = kda.kda_ssm_fwd(x[:, :near], dt[:, :near], A, B[:, :near], C[:, :near])
    part = kda.kda_ssm_bwd(x[:, near:cut], dt[:, near:cut], A, B[:, near:cut], C[:, near:cut], None, None, None, h,
                           gy[:, near:cut], tail[8])
    for i in (0, 1, 3, 4):
        assert torch.equal(whole[i][:, near:cut], part[i]), GRADS[i]
    kda.kda_check()
    del x, dt, B, C, gy, whole, tail, part
    torch.cuda.empty_cache()


def test_most_channels():
    """2^20 channels, the limit, in one group: both operators, every direction."""
    D, S, T = 1 << 20, 16, 2
    args, grads, (x, w, b, s0, gy, gsT), cu = _conv_case([5, 2], D, 4, BF16, 31)
    ch = np.arange(D) % P
    y, sT = kda.kda_conv_varlen_fwd(x, w, b, cu, s0, o_dtype=F32)
    got = kda.kda_conv_varlen_bwd(x, w, b, cu, s0, gy, gsT)
    kda.kda_check()
    conv_close(y, om.conv(*args)[0][:, ch], om.conv(*args, absolute=True)[0][:, ch], 32)
    assert np.array_equal(f64(sT), om.conv(*args)[1][..., ch])
    ref, mag = om.conv(*args, True, *grads), om.conv(*args, True, *grads, absolute=True)
    for i, (a, r, m) in enumerate(zip(got, ref, mag)):
        at = (ch,) if i in (1, 2) else (Ellipsis, ch)
        conv_close(a, r[at], m[at], 64)
    state = s0.clone()
    y = kda.kda_conv_step(x[:2], w, b, state, o_dtype=F32)
    one = (args[0][:2], *args[1:3], np.arange(3), args[4])
    conv_close(y, om.conv(*one)[0][:, ch], om.conv(*one, absolute=True)[0][:, ch], 32)
    p, cu, gy, gsT = _inputs([T], D, S, 1, F32, 32)
    d = _lead(_dev(p), 1, T)
    _check_fwd(p, cu, _fwd(d), {})
    got = _bwd(d, gy.to(DEV).view(1, T, D), gsT.to(DEV))
    kda.kda_check()
    kw = dict({k: f64(v) for k, v in p.items()}, cu=cu, gy=f64(gy), gsT=f64(gsT))
    for name, a, r, m in zip(GRADS, got, om.ssm(**kw), om.ssm(**kw, absolute=True)):
        # sums over the channels: 32 in a tile, then the 32768 tiles in order
        ssm_close(a, r, m, T, D // 32 + 32 if name in ("gB", "gC") else S, False, name)
    state = d["s0"].clone()
    y = kda.kda_ssm_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], state, d["skip"], d["z"][:, 0],
                         d["dt_bias"])
    first = {k: v[:1] if k in ("x", "dt", "z", "B", "C") else v for k, v in p.items()}
    _check_fwd(first, np.array([0, 1]), (y, state), {})
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,T", [(65535, 2), (200000, 3)])
def test_most_sequences(N, T):
    """65535 packed sequences, the limit, are the same batch with equal lengths, bit for
    bit; a dense batch may have more, and its last sequences are those of a call on them."""
    D, S = 8, 16
    p, _, gy, gsT = _inputs([T] * N, D, S, 1, BF16, 33)
    d = _lead(_dev(p), N, T)
    w, cs = torch.randn(D, 4, device=DEV), torch.randn(N, 3, D, device=DEV).to(BF16)
    gyd, gsd, gcs = gy.to(DEV).view(N, T, D), gsT.to(DEV), torch.randn(N, 3, D, device=DEV)
    ssm = (*_fwd(d), *_bwd(d, gyd, gsd))
    conv = (*kda.kda_conv_fwd(d["x"], w, None, cs), *kda.kda_conv_bwd(d["x"], w, None, cs, gyd, gcs))
    kda.kda_check()
    if N == 65535:
        cu = torch.arange(N + 1, dtype=torch.int32, device=DEV) * T
        f = {k: v.reshape(N * T, *v.shape[2:]) if k in ("x", "dt", "z", "B", "C") else v for k, v in d.items()}
        gyf = gyd.view(N * T, D)
        ssm2 = (*_fwd(f, cu), *_bwd(f, gyf, gsd, cu))
        conv2 = (*kda.kda_conv_varlen_fwd(f["x"], w, None, cu, cs),
                 *kda.kda_conv_varlen_bwd(f["x"], w, None, cu, cs, gyf, gcs))
        kda.kda_check()
        for a, c in zip(ssm + conv, ssm2 + conv2):
            assert (a is None and c is None) or torch.equal(a.reshape(c.shape), c)
    n = 300
    t = {k: v[-n:] if k in ("x", "dt", "z", "B", "C", "s0") else v for k, v in d.items()}
    ssm3 = (*_fwd(t), *_bwd(t, gyd[-n:], gsd[-n:]))
    for i in (0, 1, 2, 3, 5, 6, 8, 10):      # y, state, gx, gdt, gB, gC, gz, gs0
        assert torch.equal(ssm[i][-n:], ssm3[i]), i
    conv3 = (*kda.kda_conv_fwd(t["x"], w, None, cs[-n:]), *kda.kda_conv_bwd(t["x"], w, None, cs[-n:], gyd[-n:], gcs[-n:]))
    for i in (0, 1, 2, 5):                   # y, state, gx, gs0
        assert torch.equal(conv[i][-n:], conv3[i]), i
