"""fp64 oracle of the short causal convolution and the selective scan, forward and
gradients, one token after the other (NumPy; shares no code with the kernels).

Packed layout: tokens [T, D] with sequence boundaries cu [N + 1]; a dense batch
is N sequences of equal length.  With ``absolute=True`` every term of every sum
enters with its absolute value (decays unchanged): that bounds the rounding
error of a computation that does the same sums in lower precision.
"""
import numpy as np


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def conv(x, w, bias, cu, s0=None, silu=True, gy=None, gsT=None, absolute=False):
    """Returns (y, final_state) or, with gy, (gx, gw, gb, gs0).  x [T, D],
    w [D, W], states [N, W - 1, D]."""
    m = np.abs if absolute else (lambda a: a)
    T, D = x.shape
    W, N = w.shape[1], len(cu) - 1
    y, sT = np.zeros((T, D)), np.zeros((N, W - 1, D))
    gx, gw, gb, gs = np.zeros((T, D)), np.zeros((D, W)), np.zeros(D), np.zeros((N, W - 1, D))
    for i in range(N):
        a, b = cu[i], cu[i + 1]
        head = np.zeros((W - 1, D)) if s0 is None else s0[i]
        ext = np.concatenate([head, x[a:b]])
        gext = np.zeros_like(ext)
        for t in range(b - a):
            window = ext[t:t + W]
            exact = (window * w.T).sum(0) + (0 if bias is None else bias)
            pre = (m(window) * m(w.T)).sum(0) + (0 if bias is None else m(bias))
            s = sigmoid(exact)
            if gy is None:
                # |silu'| <= 1.1 and |silu(v)| <= |v|: twice the sum bounds what its rounding moves
                y[a + t] = exact * s if silu and not absolute else pre * (2 if silu else 1)
                continue
            slope = s + m(exact * s * (1 - s)) if silu else 1.0
            if absolute and silu:      # the slope itself moves with pre
                slope = slope + pre
            d = m(gy[a + t]) * slope
            gext[t:t + W] += d * m(w.T)
            gw += (d * m(window)).T
            gb += d
        sT[i] = m(ext[b - a:])
        if gsT is not None:
            gext[b - a:] += m(gsT[i])
        gs[i], gx[a:b] = gext[:W - 1], gext[W - 1:]
    return (y, sT) if gy is None else (gx, gw, gb, gs)


def ssm(x, dt, A, B, C, cu, skip=None, z=None, dt_bias=None, s0=None, use_softplus=True, gy=None, gsT=None,
        absolute=False):
    """Returns (y, final_state) or, with gy, (gx, gdt, gA, gB, gC, gskip, gz, gbias,
    gs0).  x, dt, z [T, D], A [D, S], B, C [T, G, S], states [N, D, S]."""
    m = np.abs if absolute else (lambda a: a)
    T, D = x.shape
    S, G, N = A.shape[1], B.shape[1], len(cu) - 1
    R = D // G
    v = dt + (0 if dt_bias is None else dt_bias)
    delta = softplus(v) if use_softplus else v
    ddelta = sigmoid(v) if use_softplus else np.ones_like(v)
    x, B, C, u = m(x), m(B), m(C), m(delta) * m(x)
    decay = np.exp(delta[:, :, None] * A)
    delta, A = m(delta), m(A)
    Bd, Cd = np.repeat(B, R, axis=1), np.repeat(C, R, axis=1)
    sk = np.zeros(D) if skip is None else m(skip)
    gate = np.ones((T, D)) if z is None else m(z * sigmoid(z))
    y, h, before = np.zeros((T, D)), np.zeros((T, D, S)), np.zeros((T, D, S))
    sT = np.zeros((N, D, S)) if s0 is None else m(s0).copy()
    for i in range(N):
        for t in range(cu[i], cu[i + 1]):
            before[t] = sT[i]
            sT[i] = h[t] = decay[t] * sT[i] + u[t][:, None] * Bd[t]
            y[t] = (Cd[t] * h[t]).sum(-1) + sk * x[t]
    if gy is None:
        return y * gate, sT
    gy = m(gy)
    gz = None
    if z is not None:
        s = sigmoid(z)
        gz = gy * y * (s + m(z * s * (1 - s)))
    dy = gy * gate
    gh = np.zeros((T, D, S))
    gs = np.zeros((N, D, S)) if gsT is None else m(gsT).copy()
    for i in range(N):
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            gh[t] = dy[t][:, None] * Cd[t] + gs[i]
            gs[i] = decay[t] * gh[t]
    wgt = gh * decay * before
    gu = (gh * Bd).sum(-1)
    gdt = ((wgt * A).sum(-1) + gu * x) * ddelta
    gB = (gh * u[:, :, None]).reshape(T, G, R, S).sum(2)
    gC = (h * dy[:, :, None]).reshape(T, G, R, S).sum(2)
    return (gu * delta + sk * dy, gdt, (wgt * delta[:, :, None]).sum(0), gB, gC, (dy * x).sum(0), gz, gdt.sum(0), gs)
