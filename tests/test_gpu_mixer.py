"""GPU: the short convolution and the selective scan as a layer uses them, in front
of each other and of the KDA layer: a prompt, then single tokens; a packed batch; a
training step's gradients through both.

Composition.  Each operator is given the previous one's GPU output, and the fp64
oracle the same tensor, so that every comparison is one operator's error: the bars
are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import oracle
import oracle.mixer as om
import gated_delta_rule_133_b200 as kda
from tests._helpers import TOL_BF16, TOL_F32, f64, norm_max_err

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Mixer:
    """in-projection -> [x | z]; conv + SiLU on x; x -> [dt | B | C]; scan; random weights."""

    def __init__(self, D, S, dtype, seed):
        g = torch.Generator().manual_seed(seed)

        def rnd(*s, f=1.0):
            return (torch.randn(*s, generator=g) * f).to(DEV)
        self.D, self.S, self.dtype = D, S, dtype
        self.win = rnd(D, 2 * D, f=D ** -0.5).to(dtype)
        self.wdt = rnd(D, D + 2 * S, f=D ** -0.5).to(dtype)
        self.weight, self.bias = rnd(D, 4, f=0.5), rnd(D, f=0.1)
        self.A, self.skip, self.dt_bias = -rnd(D, S).abs() - 0.1, rnd(D), rnd(D) - 2.0

    def project(self, u):
        return u @ self.win

    def inputs(self, xc):
        p = xc @ self.wdt
        D, S = self.D, self.S
        return p[..., :D], p[..., D:D + S].unsqueeze(-2), p[..., D + S:].unsqueeze(-2)


def _scan_bound(args, kw, T, S):
    ref, mag = om.ssm(*args, **kw), om.ssm(*args, **kw, absolute=True)
    return ref, [(2 * T + 16 + S / 8) * 2.0 ** -21 * m + 1e-37 for m in mag]


def test_prompt_then_tokens():
    """A prompt of T tokens, then steps, through column slices of the projections,
    states in place; against the oracle fed with the same intermediate tensors."""
    N, T, steps, D, S = 3, 21, 4, 64, 16
    m = Mixer(D, S, torch.bfloat16, 1)
    u = torch.randn(N, T + steps, D, generator=torch.Generator().manual_seed(2)).to(DEV).bfloat16()
    xz = m.project(u)
    x, z = xz[..., :D], xz[..., D:]
    conv_state = torch.zeros(N, 3, D, dtype=torch.bfloat16, device=DEV)
    h = torch.zeros(N, D, S, device=DEV)
    xc, _ = kda.kda_conv_fwd(x[:, :T].contiguous(), m.weight, m.bias, conv_state, final_state=conv_state)
    dt, B, C = m.inputs(xc)
    y, _ = kda.kda_ssm_fwd(xc, dt, m.A, B, C, m.skip, z[:, :T].contiguous(), m.dt_bias, h, final_state=h,
                           o_dtype=torch.float32)
    parts = [[xc], [dt], [B], [C], [y]]
    for t in range(T, T + steps):
        xt = kda.kda_conv_step(x[:, t], m.weight, m.bias, conv_state)
        dt, B, C = m.inputs(xt)
        yt = kda.kda_ssm_step(xt, dt, m.A, B, C, h, m.skip, z[:, t], m.dt_bias, o_dtype=torch.float32)
        for p, v in zip(parts, (xt, dt, B, C, yt)):
            p.append(v[:, None])
    kda.kda_check()
    L = T + steps
    cu = np.arange(N + 1) * L
    xc, dt, B, C, y = (torch.cat(p, 1) for p in parts)

    def flat(v):
        return f64(v.reshape(N * L, *v.shape[2:]))
    ref, last = om.conv(flat(x), f64(m.weight), f64(m.bias), cu)
    mag = om.conv(flat(x), f64(m.weight), f64(m.bias), cu, absolute=True)[0]
    assert (np.abs(flat(xc) - ref) <= 2.0 ** -8 * np.abs(ref) + 40 * 2.0 ** -24 * mag + 1e-37).all()
    assert np.array_equal(f64(conv_state), last)
    args = (flat(xc), flat(dt), f64(m.A), flat(B), flat(C), cu, f64(m.skip), flat(z), f64(m.dt_bias))
    (ry, rh), (by, bh) = _scan_bound(args, {}, L, S)
    assert (np.abs(flat(y) - ry) <= by).all() and (np.abs(f64(h) - rh) <= bh).all()


def test_packed_batch_equals_its_sequences():
    """A packed batch through convolution and scan gives each sequence's own result,
    bit for bit (the same work in the same order)."""
    lens, D, S = [40, 1, 0, 23, 9], 64, 32
    m = Mixer(D, S, torch.bfloat16, 3)
    u = torch.randn(sum(lens), D, generator=torch.Generator().manual_seed(4)).to(DEV).bfloat16()
    xz = m.project(u)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    xc, cs = kda.kda_conv_varlen_fwd(xz[:, :D], m.weight, m.bias, cu)
    dt, B, C = m.inputs(xc)
    y, h = kda.kda_ssm_varlen_fwd(xc, dt, m.A, B, C, cu, m.skip, xz[:, D:], m.dt_bias)
    at = 0
    for i, n in enumerate(lens):
        cut = slice(at, at + n)
        xi, ci = kda.kda_conv_fwd(xz[None, cut, :D].contiguous(), m.weight, m.bias)
        yi, hi = kda.kda_ssm_fwd(xc[None, cut], dt[None, cut].contiguous(), m.A, B[None, cut].contiguous(),
                                 C[None, cut].contiguous(), m.skip, xz[None, cut, D:].contiguous(), m.dt_bias)
        assert torch.equal(xi[0], xc[cut]) and torch.equal(ci[0], cs[i])
        assert torch.equal(yi[0], y[cut]) and torch.equal(hi[0], h[i])
        at += n


def test_training_step_through_both():
    """conv -> scan -> loss: the chained gradients against central differences of the
    fp64 oracle's composition, in a random direction of x, weight, A and dt."""
    N, T, D, S = 2, 17, 16, 16
    g = torch.Generator().manual_seed(5)

    def rnd(*s):
        return torch.randn(*s, generator=g)
    x, w, b = rnd(N, T, D), rnd(D, 4) * 0.5, rnd(D) * 0.1
    dt, A = rnd(N, T, D) - 1.0, -rnd(D, S).abs() - 0.1
    B, C, z, skip, bias, gy = rnd(N, T, 1, S), rnd(N, T, 1, S), rnd(N, T, D), rnd(D), rnd(D), rnd(N, T, D)
    d = [v.to(DEV) for v in (x, w, b, dt, A, B, C, skip, z, bias, gy)]
    xc, _ = kda.kda_conv_fwd(d[0], d[1], d[2])
    gs = kda.kda_ssm_bwd(xc, d[3], d[4], d[5], d[6], d[7], d[8], d[9], None, d[10])
    gx, gw, gb, _ = kda.kda_conv_bwd(d[0], d[1], d[2], None, gs[0])
    cu = np.arange(N + 1) * T
    v = {k: f64(t).reshape(N * T, *t.shape[2:]) if t.dim() > 2 else f64(t)
         for k, t in dict(x=x, w=w, b=b, dt=dt, A=A, B=B, C=C, z=z, skip=skip, bias=bias, gy=gy).items()}

    def loss(p):
        u, _ = om.conv(p["x"], p["w"], p["b"], cu)
        y, _ = om.ssm(u, p["dt"], p["A"], p["B"], p["C"], cu, p["skip"], p["z"], p["bias"])
        return (y * p["gy"]).sum()
    rng = np.random.default_rng(6)
    for name, grad in (("x", gx), ("w", gw), ("b", gb), ("dt", gs[1]), ("A", gs[2]), ("B", gs[3]), ("C", gs[4]),
                       ("skip", gs[5]), ("z", gs[6]), ("bias", gs[7])):
        grad = f64(grad).reshape(v[name].shape)
        step = rng.normal(size=grad.shape)
        h = 1e-5
        fd = (loss(dict(v, **{name: v[name] + h * step})) - loss(dict(v, **{name: v[name] - h * step}))) / (2 * h)
        # fp32 gradients of a chain of about 2 T decays: (2 T + 64) 2^-21 of the terms' scale
        assert abs((grad * step).sum() - fd) <= (2 * T + 64) * 2.0 ** -21 * np.abs(grad * step).sum() * 4 + 1e-6, name


@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, TOL_BF16), (torch.float32, TOL_F32)])
def test_convolution_in_front_of_the_kda_layer(dtype, tol):
    """q, k, v from one projection, each through its convolution as a column slice,
    into the chunk forward (q, k normalised there) and on with single tokens."""
    Bn, T, H, d = 1, 70, 2, 64
    D = H * d
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(Bn, T + 1, 3 * D, generator=g).to(DEV, dtype)
    w = [(torch.randn(D, 4, generator=g) * 0.5).to(DEV) for _ in range(3)]
    beta = torch.sigmoid(torch.randn(Bn, T + 1, H, generator=g)).to(DEV)
    la = -torch.nn.functional.softplus(torch.randn(Bn, T + 1, H, d, generator=g) - 3.0).to(DEV)
    heads, states = [], []
    for i in range(3):
        y, s = kda.kda_conv_fwd(qkv[:, :T, i * D:(i + 1) * D], w[i])
        heads.append(y.view(Bn, T, H, d))
        states.append(s)
    o, S = kda.kda_chunk_fwd(*heads, beta[:, :T].contiguous(), la[:, :T].contiguous(), normalize_qk=True)
    tok = [kda.kda_conv_step(qkv[:, T, i * D:(i + 1) * D], w[i], None, states[i]).view(Bn, H, d) for i in range(3)]
    S1 = S.clone()
    o1 = kda.kda_recurrent_step(*tok, beta[:, T].contiguous(), la[:, T].contiguous(), S1, normalize_qk=True)
    kda.kda_check()
    q, k, v = (np.concatenate([f64(a)[0], f64(t)]) for a, t in zip(heads, tok))
    q, k = (a / np.maximum(np.linalg.norm(a, axis=-1, keepdims=True), 1e-15) for a in (q, k))
    ro, rS = oracle.recurrence(q, k, v, f64(beta)[0], f64(la)[0], np.array([0, T + 1]), None)
    assert norm_max_err(np.concatenate([f64(o)[0], f64(o1)]), ro) <= tol
    assert norm_max_err(f64(S1), rS) <= tol
    for i in range(3):   # the convolutions themselves: the state is the last three inputs
        assert torch.equal(states[i][0], qkv[0, T - 2:T + 1, i * D:(i + 1) * D])
