"""What is measured of the short causal convolution and the selective state space scan.

Every case is one call of one of the two operators: a prompt (dense or packed), a single token per
sequence, or the backward pass of a prompt.  With ``own`` false, ``run`` computes it with elementary
torch operations; with ``own`` true it calls this repository's package.

Tensors are token-major, channels fastest.  The plain forms treat a dense batch as packed sequences
of equal length: tokens [tokens, channels] with sequence boundaries.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def _conv(name, op, seqs, tokens, channels, width, dtype, packed=False, silu=True, bias=True, states=True):
    return {"name": name, "op": "conv_" + op, "seqs": seqs, "tokens": tokens, "channels": channels, "width": width,
            "dtype": dtype, "packed": packed, "silu": silu, "bias": bias, "states": states}


def _ssm(name, op, seqs, tokens, channels, n, groups, dtype, packed=False, gated=True, states=True):
    return {"name": name, "op": "ssm_" + op, "seqs": seqs, "tokens": tokens, "channels": channels, "n": n,
            "groups": groups, "dtype": dtype, "packed": packed, "gated": gated, "states": states}


def listed():
    return [
        # the convolution before the layer in a prefill: 2 prompts of 4096 tokens, 16 heads of 128
        _conv("conv_prefill_bf16", "fwd", 2, 8192, 2048, 4, "bf16"),
        # a packed batch of 8 ragged prompts, 32 heads of 128
        _conv("conv_packed_bf16", "fwd", 8, 65536, 4096, 4, "bf16", packed=True),
        # one new token for each of 256 sequences
        _conv("conv_decode_bf16", "step", 256, 256, 4096, 4, "bf16"),
        # a training step's backward pass through the convolution
        _conv("conv_backward_bf16", "bwd", 2, 8192, 2048, 4, "bf16", states=False),
        # a short single prompt in full precision, an odd length: latency counts
        _ssm("ssm_short_fp32", "fwd", 1, 257, 768, 16, 1, "fp32"),
        # prefill of 2 prompts of 4096 tokens
        _ssm("ssm_prefill_bf16", "fwd", 2, 8192, 2048, 16, 1, "bf16"),
        # a packed batch of 8 ragged prompts
        _ssm("ssm_packed_bf16", "fwd", 8, 65536, 4096, 16, 1, "bf16", packed=True),
        # one long context
        _ssm("ssm_long_bf16", "fwd", 1, 131072, 4096, 16, 1, "bf16"),
        # one new token for each of 256 sequences
        _ssm("ssm_decode_bf16", "step", 256, 256, 4096, 16, 1, "bf16"),
        # one new token of a single sequence: the smallest call
        _ssm("ssm_decode_one_bf16", "step", 1, 1, 2048, 16, 1, "bf16"),
        # a training step's backward pass through the scan
        _ssm("ssm_backward_bf16", "bwd", 2, 8192, 2048, 16, 1, "bf16", states=False),
        # backward of a packed ragged batch in full precision, larger state, grouped B and C, odd sizes
        _ssm("ssm_backward_packed_fp32", "bwd", 5, 3001, 1040, 32, 2, "fp32", packed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the ranges of the listed ones, odd ones among them."""
    op = rng.choice(["conv_fwd", "conv_step", "conv_bwd", "ssm_fwd", "ssm_fwd", "ssm_step", "ssm_bwd", "ssm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    kind, form = op.split("_")
    if kind == "conv":
        channels = 8 * _log(rng, 32, 768)
        if form == "step":
            seqs = _log(rng, 1, 512)
            tokens, packed = seqs, False
        else:
            top = (1 << 28 if form == "fwd" else 1 << 25) // channels
            packed = rng.random() < 0.5
            seqs = _log(rng, 1, 64) if packed else rng.choice([1, 1, 2, 3, 4])
            tokens = max(seqs, _log(rng, 16, min(top, 65536)))
            tokens = tokens if packed else tokens // seqs * seqs
        return {"op": op, "seqs": seqs, "tokens": tokens, "channels": channels, "width": rng.choice([2, 3, 4, 4]),
                "dtype": dtype, "packed": packed, "silu": rng.random() < 0.8, "bias": rng.random() < 0.7,
                "states": rng.random() < 0.5}
    n = rng.choice([16, 16, 16, 32, 64])
    groups = rng.choice([1, 1, 2, 4])
    channels = 8 * groups * max(1, _log(rng, 32, 640) // groups)
    if form == "step":
        seqs = _log(rng, 1, 256)
        tokens, packed = seqs, False
    else:
        top = (1 << 32 if form == "fwd" else 1 << 28) // (channels * n)
        packed = rng.random() < 0.5
        seqs = _log(rng, 1, 64) if packed else rng.choice([1, 1, 2, 3, 4])
        tokens = max(seqs, _log(rng, 16, min(top, 65536)))
        tokens = tokens if packed else tokens // seqs * seqs
    return {"op": op, "seqs": seqs, "tokens": tokens, "channels": channels, "n": n, "groups": groups, "dtype": dtype,
            "packed": packed, "gated": rng.random() < 0.7, "states": rng.random() < 0.5}


def _lengths(case):
    """Sequence lengths: equal ones for a dense batch; for a packed one a ragged split of the tokens,
    one empty sequence and one of a single token among them where there are enough."""
    n, total = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [total // n] * n
    rng = random.Random(1000003 * n + total)
    weights = [rng.uniform(0.1, 1.0) for _ in range(n)]
    if n >= 4:
        weights[1] = 0.0
    lens = [int(total * w / sum(weights)) for w in weights]
    if n >= 4:
        lens[2] = 1
    lens[-1] += total - sum(lens)
    if lens[-1] < 0:
        lens = [0] * (n - 1) + [total]
    return lens


def _bounds(case):
    cu = [0]
    for length in _lengths(case):
        cu.append(cu[-1] + length)
    return cu


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    ty = TYPES[case["dtype"]]
    T, D, S = case["tokens"], case["channels"], case["seqs"]
    kind, form = case["op"].split("_")
    st = {"case": case, "cu": torch.tensor(_bounds(case), dtype=torch.int32, device=DEV)}
    lead = (T,) if case["packed"] or form == "step" else (S, T // S)
    if kind == "conv":
        W = case["width"]
        st["x"] = normal(*lead, D).to(ty)
        st["weight"] = normal(D, W, std=W ** -0.5)
        st["bias"] = normal(D, std=0.1) if case["bias"] else None
        has_state = case["states"] or form == "step"
        st["state"] = normal(S, W - 1, D).to(ty) if has_state else None
        if form == "bwd":
            st["grad_y"] = normal(*lead, D)
            st["grad_final"] = normal(S, W - 1, D) if has_state else None
        return st
    N, G = case["n"], case["groups"]
    st["x"] = torch.nn.functional.silu(normal(*lead, D)).to(ty)      # the scan's input leaves a SiLU
    st["dt"] = normal(*lead, D, std=0.5).to(ty)
    # step sizes spread over [1e-3, 1e-1]: the bias is their inverse softplus
    step = torch.exp(torch.rand(D, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))
    rates = torch.arange(1, N + 1, device=DEV, dtype=torch.float32).expand(D, N)
    st["A"] = -rates * torch.exp(normal(D, N, std=0.1))
    st["B"] = normal(*lead, G, N).to(ty)
    st["C"] = normal(*lead, G, N).to(ty)
    st["skip"] = 1.0 + normal(D, std=0.1)
    st["z"] = normal(*lead, D).to(ty) if case["gated"] else None
    has_state = case["states"] or form == "step"
    st["state"] = normal(S, D, N, std=0.3) if has_state else None
    if form == "bwd":
        st["grad_y"] = normal(*lead, D)
        st["grad_final"] = normal(S, D, N) if has_state else None
    return st


# ------------------------------------------------------------------------------------------- runs
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import gated_delta_rule_133_b200 as kda

    case = s["case"]
    kind, form = case["op"].split("_")
    o_dtype = TYPES[case["dtype"]]
    if kind == "conv":
        w, b, silu = s["weight"], s["bias"], case["silu"]
        if form == "step":
            return kda.kda_conv_step(s["x"], w, b, s["state"], silu=silu, o_dtype=o_dtype), s["state"]
        if form == "fwd":
            if case["packed"]:
                return kda.kda_conv_varlen_fwd(s["x"], w, b, s["cu"], s["state"], silu=silu, o_dtype=o_dtype)
            return kda.kda_conv_fwd(s["x"], w, b, s["state"], silu=silu, o_dtype=o_dtype)
        want = s["state"] is not None
        if case["packed"]:
            return kda.kda_conv_varlen_bwd(s["x"], w, b, s["cu"], s["state"], s["grad_y"], s["grad_final"], silu=silu,
                                           want_initial_state_grad=want)
        return kda.kda_conv_bwd(s["x"], w, b, s["state"], s["grad_y"], s["grad_final"], silu=silu,
                                want_initial_state_grad=want)
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    rest = (s["skip"], s["z"], s["dt_bias"])
    if form == "step":
        return kda.kda_ssm_step(*args, s["state"], *rest, o_dtype=o_dtype), s["state"]
    if form == "fwd":
        if case["packed"]:
            return kda.kda_ssm_varlen_fwd(*args, s["cu"], *rest, s["state"], o_dtype=o_dtype)
        return kda.kda_ssm_fwd(*args, *rest, s["state"], o_dtype=o_dtype)
    want = s["state"] is not None
    if case["packed"]:
        return kda.kda_ssm_varlen_bwd(*args, s["cu"], *rest, s["state"], s["grad_y"], s["grad_final"],
                                      want_initial_state_grad=want)
    return kda.kda_ssm_bwd(*args, *rest, s["state"], s["grad_y"], s["grad_final"], want_initial_state_grad=want)


def _run_plain(s):
    case = s["case"]
    kind, form = case["op"].split("_")
    return {"conv_fwd": _conv_fwd, "conv_step": _conv_step, "conv_bwd": _conv_bwd, "ssm_fwd": _ssm_fwd,
            "ssm_step": _ssm_step, "ssm_bwd": _ssm_bwd}[kind + "_" + form](s, case)


def _flat(t, lead):
    """[..., rest] -> [tokens, rest] in fp32."""
    return None if t is None else t.reshape(-1, *t.shape[lead:]).float()


def _taps(cu, T, S, W):
    """For each token and tap the row of [states ; tokens] it reads, and the rows the final states take."""
    t = torch.arange(T, device=DEV)
    start = cu.long()
    seq = torch.searchsorted(start, t, right=True) - 1
    pos = t - start[seq]
    back = torch.arange(W, device=DEV) - (W - 1)
    p = pos[:, None] + back[None, :]
    rows = torch.where(p >= 0, S * (W - 1) + t[:, None] + back[None, :], seq[:, None] * (W - 1) + p + W - 1)
    length = (start[1:] - start[:-1])[:, None]
    q = length + back[None, 1:] - 1
    i = torch.arange(S, device=DEV)[:, None]
    last = torch.where(q >= 0, S * (W - 1) + start[:-1, None] + q, i * (W - 1) + q + W - 1)
    return rows, last


def _conv_pre(s, case):
    W, S, D, T = case["width"], case["seqs"], case["channels"], case["tokens"]
    x = s["x"].reshape(T, D)
    head = s["state"].reshape(S * (W - 1), D) if s["state"] is not None else x.new_zeros(S * (W - 1), D)
    buf = torch.cat([head, x]).float()
    rows, last = _taps(s["cu"], T, S, W)
    pre = torch.zeros(T, D, device=DEV) if s["bias"] is None else s["bias"].expand(T, D)
    for j in range(W):
        pre = pre + buf[rows[:, j]] * s["weight"][:, j]
    return buf, rows, last, pre


def _conv_fwd(s, case):
    buf, _, last, pre = _conv_pre(s, case)
    y = pre / (1 + torch.exp(-pre)) if case["silu"] else pre
    return y.to(s["x"].dtype).reshape(s["x"].shape), buf[last].to(s["x"].dtype)


def _conv_step(s, case):
    full = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (full.float() * s["weight"].t()).sum(1)
    pre = pre if s["bias"] is None else pre + s["bias"]
    y = pre / (1 + torch.exp(-pre)) if case["silu"] else pre
    s["state"].copy_(full[:, 1:])
    return y.to(s["x"].dtype), s["state"]


def _conv_bwd(s, case):
    W, S, D, T = case["width"], case["seqs"], case["channels"], case["tokens"]
    buf, rows, last, pre = _conv_pre(s, case)
    dpre = s["grad_y"].reshape(T, D)
    if case["silu"]:
        sig = 1 / (1 + torch.exp(-pre))
        dpre = dpre * sig * (1 + pre * (1 - sig))
    grad = torch.zeros_like(buf)
    dw = []
    for j in range(W):
        grad.index_add_(0, rows[:, j], dpre * s["weight"][:, j])
        dw.append((dpre * buf[rows[:, j]]).sum(0, dtype=torch.float64))
    if s["grad_final"] is not None:
        grad.index_add_(0, last.reshape(-1), s["grad_final"].reshape(-1, D))
    head = S * (W - 1)
    return (grad[head:].reshape(s["x"].shape), torch.stack(dw, 1).float(),
            dpre.sum(0, dtype=torch.float64).float() if s["bias"] is not None else None,
            grad[:head].reshape(S, W - 1, D) if s["state"] is not None else None)


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 0 from h = 0, by doubling."""
    k, T = 1, a.shape[0]
    while k < T:
        b = torch.cat([b[:k], torch.addcmul(b[k:], a[k:], b[:-k])])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _ssm_parts(s, case):
    """fp32 token-major parts of a prompt, and the tokens that begin and end a sequence."""
    lead = s["x"].dim() - 1
    p = {k: _flat(s[k], lead) for k in ("x", "dt", "z", "B", "C")}
    cu = _bounds(case)
    spans = [(cu[i], cu[i + 1] - 1, i) for i in range(case["seqs"]) if cu[i + 1] > cu[i]]
    p["begin"] = [(first, i) for first, _, i in spans]
    p["end"] = [(last, i) for _, last, i in spans]
    return p


def _within(marks, lo, hi):
    return [(t - lo, i) for t, i in marks if lo <= t < hi]


def _ssm_block(s, case, p, lo, hi, carry):
    """States of tokens [lo, hi): (decay, decay cut at sequence starts, step sizes, h, h before each token)."""
    D, N, G = case["channels"], case["n"], case["groups"]
    delta = _softplus(p["dt"][lo:hi] + s["dt_bias"])
    a = torch.exp(delta[..., None] * s["A"])
    u = delta * p["x"][lo:hi]
    b = (u.reshape(-1, G, D // G, 1) * p["B"][lo:hi, :, None, :]).reshape(-1, D, N)
    begin = _within(p["begin"], lo, hi)
    cut = a.clone()
    for t, i in begin:
        cut[t] = 0
        if s["state"] is not None:
            b[t] += a[t] * s["state"][i]
    b[0] += cut[0] * carry
    h = _scan(cut, b)
    before = torch.cat([carry[None], h[:-1]])
    for t, i in begin:
        before[t] = s["state"][i] if s["state"] is not None else 0
    return a, cut, delta, u, h, before


def _block(case):
    return max(1, min(case["tokens"], (1 << 26) // (case["channels"] * case["n"])))


def _ssm_fwd(s, case):
    T, D, N, G, S = case["tokens"], case["channels"], case["n"], case["groups"], case["seqs"]
    p = _ssm_parts(s, case)
    y = torch.empty(T, D, dtype=s["x"].dtype, device=DEV)
    final = torch.zeros(S, D, N, device=DEV) if s["state"] is None else s["state"].clone()
    carry = torch.zeros(D, N, device=DEV)
    L = _block(case)
    for lo in range(0, T, L):
        hi = min(T, lo + L)
        _, _, _, _, h, _ = _ssm_block(s, case, p, lo, hi, carry)
        carry = h[-1]
        y0 = (h.reshape(-1, G, D // G, N) * p["C"][lo:hi, :, None, :]).sum(-1).reshape(-1, D) + s["skip"] * p["x"][lo:hi]
        if p["z"] is not None:
            z = p["z"][lo:hi]
            y0 = y0 * z / (1 + torch.exp(-z))
        y[lo:hi] = y0.to(y.dtype)
        for t, i in _within(p["end"], lo, hi):
            final[i] = h[t]
    return y.reshape(s["x"].shape), final


def _ssm_step(s, case):
    D, N, G, S = case["channels"], case["n"], case["groups"], case["seqs"]
    x, delta = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    b = (delta * x).reshape(S, G, D // G, 1) * s["B"].float()[:, :, None, :]
    h = torch.exp(delta[..., None] * s["A"]) * s["state"] + b.reshape(S, D, N)
    y = (h.reshape(S, G, D // G, N) * s["C"].float()[:, :, None, :]).sum(-1).reshape(S, D) + s["skip"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    s["state"].copy_(h)
    return y.to(s["x"].dtype), s["state"]


def _ssm_bwd(s, case):
    T, D, N, G, S = case["tokens"], case["channels"], case["n"], case["groups"], case["seqs"]
    p = _ssm_parts(s, case)
    L = _block(case)
    starts = list(range(0, T, L))
    carries, carry = [], torch.zeros(D, N, device=DEV)
    for lo in starts:
        carries.append(carry)
        carry = _ssm_block(s, case, p, lo, min(T, lo + L), carry)[4][-1]
    f32 = dict(device=DEV, dtype=torch.float32)
    dx, ddt = torch.empty(T, D, **f32), torch.empty(T, D, **f32)
    dz = torch.empty(T, D, **f32) if p["z"] is not None else None
    dB, dC = torch.empty(T, G, N, **f32), torch.empty(T, G, N, **f32)
    dA = torch.zeros(D, N, device=DEV, dtype=torch.float64)
    dskip, dbias = torch.zeros_like(dA[:, 0]), torch.zeros_like(dA[:, 0])
    ds0 = s["grad_final"].clone() if s["grad_final"] is not None else None
    grad_y = s["grad_y"].reshape(T, D)
    back = torch.zeros(D, N, **f32)          # what the following token hands to the last one of the block
    for lo, carry in zip(reversed(starts), reversed(carries)):
        hi = min(T, lo + L)
        a, cut, delta, u, h, before = _ssm_block(s, case, p, lo, hi, carry)
        x, C, B = p["x"][lo:hi], p["C"][lo:hi], p["B"][lo:hi]
        dy = grad_y[lo:hi]
        if dz is not None:
            z = p["z"][lo:hi]
            sig = 1 / (1 + torch.exp(-z))
            y0 = (h.reshape(-1, G, D // G, N) * C[:, :, None, :]).sum(-1).reshape(-1, D) + s["skip"] * x
            dz[lo:hi] = dy * y0 * sig * (1 + z * (1 - sig))
            dy = dy * z * sig
        src = (dy.reshape(-1, G, D // G, 1) * C[:, :, None, :]).reshape(-1, D, N)
        if s["grad_final"] is not None:
            for t, i in _within(p["end"], lo, hi):
                src[t] += s["grad_final"][i]
        src[-1] += back
        nxt = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
        g = _scan(nxt.flip(0), src.flip(0)).flip(0)
        back = cut[0] * g[0]
        ga = g * a
        if ds0 is not None:
            for t, i in _within(p["begin"], lo, hi):
                ds0[i] = ga[t]
        w = ga * before
        gd = g.reshape(-1, G, D // G, N)
        du = (gd * B[:, :, None, :]).sum(-1).reshape(-1, D)
        dB[lo:hi] = (gd * u.reshape(-1, G, D // G, 1)).sum(2)
        dC[lo:hi] = (h.reshape(-1, G, D // G, N) * dy.reshape(-1, G, D // G, 1)).sum(2)
        ddelta = (w * s["A"]).sum(-1) + du * x
        dA += (w * delta[..., None]).sum(0, dtype=torch.float64)
        dx[lo:hi] = du * delta + s["skip"] * dy
        dskip += (dy * x).sum(0, dtype=torch.float64)
        ddt[lo:hi] = ddelta / (1 + torch.exp(-(p["dt"][lo:hi] + s["dt_bias"])))
        dbias += ddt[lo:hi].sum(0, dtype=torch.float64)
    like = s["x"].shape
    return (dx.reshape(like), ddt.reshape(like), dA.float(), dB.reshape(s["B"].shape), dC.reshape(s["C"].shape),
            dskip.float(), None if dz is None else dz.reshape(like), dbias.float(),
            ds0 if s["state"] is not None else None)


# ------------------------------------------------------------------------------------------- work
def work(case):
    T, D, S = case["tokens"], case["channels"], case["seqs"]
    e = 2 if case["dtype"] == "bf16" else 4
    kind, form = case["op"].split("_")
    states = case["states"] or form == "step"
    if kind == "conv":
        W = case["width"]
        params = D * (W + (1 if case["bias"] else 0)) * 4
        rows = S * (W - 1) * D * e
        act = 4 if case["silu"] else 0
        if form == "bwd":
            extra = S * (W - 1) * D * (e + 8) if states else 0
            return {"bytes": T * D * (e + 8) + 2 * params + extra, "flops": T * D * (6 * W + 2 * act)}
        return {"bytes": T * D * 2 * e + params + rows * (2 if states else 1), "flops": T * D * (2 * W + act)}
    N, G = case["n"], case["groups"]
    params = D * (N + 2) * 4
    st = S * D * N * 4
    z = 1 if case["gated"] else 0
    if form == "bwd":
        extra = 3 * st if states else 0
        return {"bytes": T * D * ((3 if z else 2) * e + 4 + (12 if z else 8)) + T * G * N * (2 * e + 8) + 2 * params + extra,
                "flops": T * D * (24 * N + 20)}
    return {"bytes": T * D * (3 + z) * e + T * G * N * 2 * e + params + st * (2 if states else 1),
            "flops": T * D * (7 * N + 10)}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, one token after the other."""
    s = prepare(case, seed)
    kind, form = case["op"].split("_")
    d = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v) for k, v in s.items()}
    cu = _bounds(case) if form != "step" else list(range(case["seqs"] + 1))
    return _exact_conv(d, case, form, cu) if kind == "conv" else _exact_ssm(d, case, form, cu)


def _sigmoid64(v):
    return torch.special.expit(v)


def _exact_conv(d, case, form, cu):
    W, S, D, T = case["width"], case["seqs"], case["channels"], case["tokens"]
    if T * D > 1 << 29:
        return None
    x = d["x"].reshape(T, D)
    shape = d["x"].shape
    y, final, gx, gs = [], [], [], []
    gw, gb = torch.zeros(D, W, dtype=torch.float64, device=DEV), torch.zeros(D, dtype=torch.float64, device=DEV)
    for i in range(S):
        n = cu[i + 1] - cu[i]
        head = d["state"][i] if d["state"] is not None else torch.zeros(W - 1, D, dtype=torch.float64, device=DEV)
        ext = torch.cat([head, x[cu[i]:cu[i + 1]]])
        pre = sum(ext[j:j + n] * d["weight"][:, j] for j in range(W))
        if d["bias"] is not None:
            pre = pre + d["bias"]
        if form != "bwd":
            y.append(pre * _sigmoid64(pre) if case["silu"] else pre)
            final.append(ext[n:])
            continue
        gp = d["grad_y"].reshape(T, D)[cu[i]:cu[i + 1]]
        if case["silu"]:
            sg = _sigmoid64(pre)
            gp = gp * (sg + pre * sg * (1 - sg))
        ge = torch.zeros_like(ext)
        for j in range(W):
            ge[j:j + n] += gp * d["weight"][:, j]
            gw[:, j] += (gp * ext[j:j + n]).sum(0)
        gb += gp.sum(0)
        if d["grad_final"] is not None:
            ge[n:] += d["grad_final"][i]
        gs.append(ge[:W - 1])
        gx.append(ge[W - 1:])
    if form == "bwd":
        return (torch.cat(gx).reshape(shape), gw, gb if d["bias"] is not None else None,
                torch.stack(gs) if d["state"] is not None else None)
    return torch.cat(y).reshape(shape), torch.stack(final)


def _exact_ssm(d, case, form, cu):
    T, D, N, G, S = case["tokens"], case["channels"], case["n"], case["groups"], case["seqs"]
    R = D // G
    if form == "bwd" and T * D * N > 1 << 29:
        return None
    f64 = dict(dtype=torch.float64, device=DEV)
    x, dt = d["x"].reshape(T, D), d["dt"].reshape(T, D) + d["dt_bias"]
    delta = torch.logaddexp(dt, torch.zeros_like(dt))
    B, C = d["B"].reshape(T, G, N), d["C"].reshape(T, G, N)
    z = d["z"].reshape(T, D) if d["z"] is not None else None
    begin = {}
    for i in range(S):
        if cu[i + 1] > cu[i]:
            begin[cu[i]] = i
    ends = {cu[i + 1] - 1: i for i in range(S) if cu[i + 1] > cu[i]}
    zero = torch.zeros(D, N, **f64)
    init = d["state"] if d["state"] is not None else torch.zeros(S, D, N, **f64)
    final = init.clone()
    L = max(1, (1 << 24) // (D * N))
    y0 = torch.empty(T, D, **f64)
    hist = torch.empty(T, D, N, **f64) if form == "bwd" else None
    decay = torch.empty(T, D, N, **f64) if form == "bwd" else None
    h = zero
    for lo in range(0, T, L):
        hi = min(T, lo + L)
        a = torch.exp(delta[lo:hi, :, None] * d["A"])
        b = (delta[lo:hi] * x[lo:hi])[:, :, None] * B[lo:hi].repeat_interleave(R, 1)
        H = torch.empty_like(a)
        for t in range(lo, hi):
            if t in begin:
                h = init[begin[t]]
            h = torch.addcmul(b[t - lo], a[t - lo], h, out=H[t - lo])
            if t in ends:
                final[ends[t]] = h
        h = h.clone()
        y0[lo:hi] = (H * C[lo:hi].repeat_interleave(R, 1)).sum(-1)
        if hist is not None:
            hist[lo:hi], decay[lo:hi] = H, a
    y0 += d["skip"] * x
    if form != "bwd":
        y = y0 if z is None else y0 * z * _sigmoid64(z)
        return y.reshape(d["x"].shape), final
    gy = d["grad_y"].reshape(T, D)
    gz = None
    if z is not None:
        sg = _sigmoid64(z)
        gz = (gy * y0 * (sg + z * sg * (1 - sg))).reshape(d["x"].shape)
        gy = gy * z * sg
    gh0 = d["grad_final"].clone() if d["grad_final"] is not None else torch.zeros(S, D, N, **f64)
    gh = torch.empty(T, D, N, **f64)
    following = zero
    for t in range(T - 1, -1, -1):
        g = gy[t, :, None] * C[t].repeat_interleave(R, 0)
        if t in ends:
            following = gh0[ends[t]].clone()
        gh[t] = g + following
        following = decay[t] * gh[t]
        if t in begin:
            gh0[begin[t]] = following
    prev = torch.cat([zero[None], hist[:-1]])
    for t, i in begin.items():
        prev[t] = init[i]
    gC = (hist * gy[:, :, None]).reshape(T, G, R, N).sum(2)
    del hist
    prev *= decay
    del decay
    prev *= gh                                                       # d loss / d (delta A)
    gA = (prev * delta[:, :, None]).sum(0)
    gdelta = (prev * d["A"]).sum(-1)
    del prev
    gu = (gh.reshape(T, G, R, N) * B[:, :, None, :]).sum(-1).reshape(T, D)
    gB = (gh.reshape(T, G, R, N) * (delta * x).reshape(T, G, R, 1)).sum(2)
    gdelta = gdelta + gu * x
    gdt = gdelta * _sigmoid64(dt)
    return ((gu * delta + d["skip"] * gy).reshape(d["x"].shape), gdt.reshape(d["x"].shape), gA,
            gB.reshape(d["B"].shape), gC.reshape(d["C"].shape), (gy * x).sum(0), gz, gdt.sum(0),
            gh0 if d["state"] is not None else None)
