"""Short causal convolution and selective state space scan (``kda_conv_*`` and
``kda_ssm_*`` of include/kda.h).

    y, S = kda_conv_fwd(x, weight, bias, initial_state)             # prompts [B, T, D]
    y, S = kda_conv_varlen_fwd(x, weight, bias, cu_seqlens)         # packed prompts [T, D]
    y    = kda_conv_step(x, weight, bias, state)                    # one token each, state in place
    y, h = kda_ssm_fwd(x, dt, A, B, C, skip, z, dt_bias, initial_state)
    y, h = kda_ssm_varlen_fwd(x, dt, A, B, C, cu_seqlens, skip, z, dt_bias, initial_state)
    y    = kda_ssm_step(x, dt, A, B, C, state, skip, z, dt_bias)

and their gradients (``*_bwd``).  As in the rest of the package these functions
only check arguments, allocate outputs and pass pointers; the token-major inputs
(x, dt, B, C, z) may be column slices of wider tensors (last dimension
contiguous, one stride from token to token), every other tensor is contiguous.
All tensors are on one CUDA device; the work runs on ``stream``, or on that
device's current stream, and new tensors belong to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib

__all__ = ["kda_conv_fwd", "kda_conv_varlen_fwd", "kda_conv_step", "kda_conv_bwd", "kda_conv_varlen_bwd",
           "kda_ssm_fwd", "kda_ssm_varlen_fwd", "kda_ssm_step", "kda_ssm_bwd", "kda_ssm_varlen_bwd",
           "conv_bwd_workspace_size", "ssm_fwd_workspace_size", "ssm_varlen_fwd_workspace_size",
           "ssm_bwd_workspace_size", "ssm_varlen_bwd_workspace_size"]

_DTYPES = {torch.float32: _lib.KDA_F32, torch.bfloat16: _lib.KDA_BF16}
_F32 = torch.float32


def _fail(name, what, got, want):
    raise ValueError(f"{name} {what} {got}, expected {want}")


def _dense(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor (None for None)."""
    if t is None:
        return None
    if t.shape != shape:
        _fail(name, "has shape", tuple(t.shape), tuple(shape))
    if t.dtype != dtype:
        _fail(name, "has dtype", t.dtype, dtype)
    if t.device != device:
        _fail(name, "is on", t.device, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, lead, dtype, device):
    """(pointer, row stride) of a token-major tensor whose first `lead`
    dimensions count tokens; the rest is one contiguous row."""
    if t is None:
        return None, 0
    if t.shape != shape:
        _fail(name, "has shape", tuple(t.shape), tuple(shape))
    if t.dtype != dtype:
        _fail(name, "has dtype", t.dtype, dtype)
    if t.device != device:
        _fail(name, "is on", t.device, device)
    row = 1
    for n in shape[lead:]:
        row *= n
    if t.is_contiguous():
        return t.data_ptr(), row
    stride = t.stride()
    inner = 1
    ok = True
    for i in range(len(shape) - 1, lead - 1, -1):
        ok = ok and (shape[i] == 1 or stride[i] == inner)
        inner *= shape[i]
    ld, tokens = None, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] != 1:
            if ld is None:
                ld = stride[i]
            ok = ok and stride[i] == ld * tokens
        tokens *= shape[i]
    if ld is None:
        ld = row
    if not ok or ld < row or (ld * t.element_size()) % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name} must have contiguous rows with one 16-byte aligned stride from token to token")
    return t.data_ptr(), ld


def _types(x, o_dtype, y):
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    o_dtype = y.dtype if y is not None else x.dtype if o_dtype is None else o_dtype
    if o_dtype not in _DTYPES:
        raise ValueError(f"unsupported output dtype {o_dtype}")
    return _DTYPES[x.dtype], o_dtype


def _lead(x, dims, name="x"):
    if x.dim() != dims:
        _fail(name, "has", f"{x.dim()} dimensions", dims)
    return x.shape


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield stream.cuda_stream


class _Current:
    """The device's current stream, without switching anything."""

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        return False


def _on(device, stream):
    """Context in which to allocate and launch; gives the raw stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}, expected a CUDA device")
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return _Current(device)
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    return _switched(device, stream)


def _scratch(nbytes, workspace, device):
    if nbytes == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.device != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel(), workspace


def conv_bwd_workspace_size(tokens, D, W):
    """Workspace bytes of kda_conv_bwd / kda_conv_varlen_bwd for `tokens` tokens in all."""
    return _lib.workspace_size("kda_conv_bwd_workspace_size", tokens, D, W)


def ssm_fwd_workspace_size(B, T, D, S, G=1, dtype=torch.bfloat16):
    """Workspace bytes of kda_ssm_fwd."""
    return _lib.workspace_size("kda_ssm_fwd_workspace_size", B, T, D, S, G, _DTYPES[dtype])


def ssm_varlen_fwd_workspace_size(N, T, D, S, G=1, dtype=torch.bfloat16):
    """Workspace bytes of kda_ssm_varlen_fwd for N packed sequences of T tokens in all."""
    return _lib.workspace_size("kda_ssm_varlen_fwd_workspace_size", N, T, D, S, G, _DTYPES[dtype])


def ssm_bwd_workspace_size(B, T, D, S, G=1, dtype=torch.bfloat16):
    """Workspace bytes of kda_ssm_bwd."""
    return _lib.workspace_size("kda_ssm_bwd_workspace_size", B, T, D, S, G, _DTYPES[dtype])


def ssm_varlen_bwd_workspace_size(N, T, D, S, G=1, dtype=torch.bfloat16):
    """Workspace bytes of kda_ssm_varlen_bwd for N packed sequences of T tokens in all."""
    return _lib.workspace_size("kda_ssm_varlen_bwd_workspace_size", N, T, D, S, G, _DTYPES[dtype])


# ------------------------------------------------------------------ short convolution
def kda_conv_fwd(x, weight, bias=None, initial_state=None, *, silu=True, y=None, final_state=None,
                 output_final_state=True, o_dtype=None, stream=None):
    """Causal depthwise convolution over equal-length sequences, then SiLU.

    x [B, T, D] (bf16 or fp32); weight [D, W] (W = 2..4) and bias [D] fp32;
    initial_state [B, W - 1, D] of x's dtype (the last W - 1 inputs, oldest
    first) or None.  Returns (y [B, T, D] in o_dtype, by default x's dtype;
    final_state [B, W - 1, D] or None)."""
    B, T, D = _lead(x, 3)
    return _conv_fwd(x, weight, bias, None, B, T, initial_state, silu, y, final_state, output_final_state, o_dtype,
                     stream)


def kda_conv_varlen_fwd(x, weight, bias, cu_seqlens, initial_state=None, *, silu=True, y=None, final_state=None,
                        output_final_state=True, o_dtype=None, stream=None):
    """kda_conv_fwd over N packed sequences: x [T, D], cu_seqlens [N + 1] int32
    on the device, states [N, W - 1, D]."""
    T, D = _lead(x, 2)
    return _conv_fwd(x, weight, bias, cu_seqlens, _packed(cu_seqlens, x.device), T, initial_state, silu, y,
                     final_state, output_final_state, o_dtype, stream)


def _packed(cu_seqlens, device):
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        _fail("cu_seqlens", "has shape", tuple(cu_seqlens.shape), "(N + 1,)")
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, device)
    return cu_seqlens.shape[0] - 1


def _conv_params(weight, bias, D, dev):
    if weight.dim() != 2 or weight.shape[0] != D:
        _fail("weight", "has shape", tuple(weight.shape), (D, "W"))
    return (_dense(weight, "weight", weight.shape, _F32, dev), _dense(bias, "bias", (D,), _F32, dev), weight.shape[1])


def _conv_fwd(x, weight, bias, cu, N, T, s0, silu, y, sT, want_state, o_dtype, stream):
    dev, D = x.device, x.shape[-1]
    code, o_dtype = _types(x, o_dtype, y)
    xp, ldx = _rows(x, "x", x.shape, x.dim() - 1, x.dtype, dev)
    wp, bp, W = _conv_params(weight, bias, D, dev)
    s0p = _dense(s0, "initial_state", (N, W - 1, D), x.dtype, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    sTp = _dense(sT, "final_state", (N, W - 1, D), x.dtype, dev)
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty(x.shape, dtype=o_dtype, device=dev)
            yp = y.data_ptr()
        if sT is None and want_state:
            sT = torch.empty((N, W - 1, D), dtype=x.dtype, device=dev)
            sTp = sT.data_ptr()
        tail = (s0p, yp, sTp) + ((N,) if cu is None else ()) + (T, D, W, code, _DTYPES[o_dtype],
                                                                _lib.KDA_CONV_SILU if silu else 0, st)
        if cu is None:
            _lib.call("kda_conv_fwd", xp, ldx, wp, bp, *tail)
        else:
            _lib.call("kda_conv_varlen_fwd", xp, ldx, wp, bp, cu.data_ptr(), N, *tail)
    return y, sT


def kda_conv_step(x, weight, bias, state, *, silu=True, y=None, o_dtype=None, stream=None):
    """One token per sequence: x [N, D]; state [N, W - 1, D] of x's dtype, moved on
    by one token in place.  Returns y [N, D]."""
    N, D = _lead(x, 2)
    dev = x.device
    code, o_dtype = _types(x, o_dtype, y)
    xp, ldx = _rows(x, "x", x.shape, 1, x.dtype, dev)
    wp, bp, W = _conv_params(weight, bias, D, dev)
    sp = _dense(state, "state", (N, W - 1, D), x.dtype, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty(x.shape, dtype=o_dtype, device=dev)
            yp = y.data_ptr()
        _lib.call("kda_conv_step", xp, ldx, wp, bp, sp, yp, N, D, W, code, _DTYPES[o_dtype],
                  _lib.KDA_CONV_SILU if silu else 0, st)
    return y


def kda_conv_bwd(x, weight, bias, initial_state, grad_y, grad_final_state=None, *, silu=True,
                 want_initial_state_grad=True, stream=None, workspace=None):
    """Backward of kda_conv_fwd: gradients of sum(y * grad_y) + sum(final_state * grad_final_state).

    grad_y [B, T, D] and grad_final_state [B, W - 1, D] (or None) fp32.  Returns
    fp32 (grad_x, grad_weight, grad_bias or None, grad_initial_state or None)."""
    B, T, D = _lead(x, 3)
    return _conv_bwd(x, weight, bias, None, B, T, initial_state, grad_y, grad_final_state, silu,
                     want_initial_state_grad, stream, workspace)


def kda_conv_varlen_bwd(x, weight, bias, cu_seqlens, initial_state, grad_y, grad_final_state=None, *, silu=True,
                        want_initial_state_grad=True, stream=None, workspace=None):
    """Backward of kda_conv_varlen_fwd (x, grad_y [T, D], states [N, W - 1, D])."""
    T, D = _lead(x, 2)
    return _conv_bwd(x, weight, bias, cu_seqlens, _packed(cu_seqlens, x.device), T, initial_state, grad_y,
                     grad_final_state, silu, want_initial_state_grad, stream, workspace)


def _conv_bwd(x, weight, bias, cu, N, T, s0, gy, gsT, silu, want_gs0, stream, workspace):
    dev, D = x.device, x.shape[-1]
    code, _ = _types(x, None, None)
    xp, ldx = _rows(x, "x", x.shape, x.dim() - 1, x.dtype, dev)
    wp, bp, W = _conv_params(weight, bias, D, dev)
    s0p = _dense(s0, "initial_state", (N, W - 1, D), x.dtype, dev)
    gyp = _dense(gy, "grad_y", x.shape, _F32, dev)
    gsTp = _dense(gsT, "grad_final_state", (N, W - 1, D), _F32, dev)
    nbytes = conv_bwd_workspace_size(T if cu is not None else N * T, D, W)
    with _on(dev, stream) as st:
        f32 = dict(dtype=_F32, device=dev)
        gx, gw = torch.empty(x.shape, **f32), torch.empty((D, W), **f32)
        gb = torch.empty(D, **f32) if bias is not None else None
        gs0 = torch.empty((N, W - 1, D), **f32) if want_gs0 else None
        ws, n, _keep = _scratch(nbytes, workspace, dev)
        tail = (s0p, gyp, gsTp, gx.data_ptr(), gw.data_ptr(), None if gb is None else gb.data_ptr(),
                None if gs0 is None else gs0.data_ptr()) + ((N,) if cu is None else ()) + (
                    T, D, W, code, _lib.KDA_CONV_SILU if silu else 0, ws, n, st)
        if cu is None:
            _lib.call("kda_conv_bwd", xp, ldx, wp, bp, *tail)
        else:
            _lib.call("kda_conv_varlen_bwd", xp, ldx, wp, bp, cu.data_ptr(), N, *tail)
    return gx, gw, gb, gs0


# ------------------------------------------------------------------ selective scan
def _ssm_in(x, dt, A, B, C, skip, z, dt_bias):
    """Checked (pointers and row strides in the C ABI's order, S, G)."""
    dev, D, lead = x.device, x.shape[-1], x.dim() - 1
    if A.dim() != 2 or A.shape[0] != D:
        _fail("A", "has shape", tuple(A.shape), (D, "S"))
    S = A.shape[1]
    if B.dim() != lead + 2:
        _fail("B", "has", f"{B.dim()} dimensions", lead + 2)
    G = B.shape[lead]
    bc = x.shape[:lead] + (G, S)
    ty = x.dtype
    skp, dbp = _dense(skip, "skip", (D,), _F32, dev), _dense(dt_bias, "dt_bias", (D,), _F32, dev)
    return (*_rows(x, "x", x.shape, lead, ty, dev), *_rows(dt, "dt", x.shape, lead, ty, dev),
            _dense(A, "A", A.shape, _F32, dev), *_rows(B, "B", bc, lead, ty, dev), *_rows(C, "C", bc, lead, ty, dev),
            skp, *_rows(z, "z", x.shape, lead, ty, dev), dbp), S, G


def kda_ssm_fwd(x, dt, A, B, C, skip=None, z=None, dt_bias=None, initial_state=None, *, softplus=True, y=None,
                final_state=None, output_final_state=True, o_dtype=None, stream=None, workspace=None):
    """Selective scan over equal-length sequences.

    x, dt, z [B, T, D] and B, C [B, T, G, S] (bf16 or fp32); A [D, S], skip and
    dt_bias [D], initial_state [B, D, S] fp32; skip, z, dt_bias, initial_state may
    be None.  softplus=False takes dt + dt_bias itself as the step size.  Returns
    (y [B, T, D] in o_dtype, by default x's dtype; final_state [B, D, S] or None)."""
    N, T, _ = _lead(x, 3)
    return _ssm_fwd(x, dt, A, B, C, None, N, T, skip, z, dt_bias, initial_state, softplus, y, final_state,
                    output_final_state, o_dtype, stream, workspace)


def kda_ssm_varlen_fwd(x, dt, A, B, C, cu_seqlens, skip=None, z=None, dt_bias=None, initial_state=None, *,
                       softplus=True, y=None, final_state=None, output_final_state=True, o_dtype=None, stream=None,
                       workspace=None):
    """kda_ssm_fwd over N packed sequences: x, dt, z [T, D], B, C [T, G, S],
    cu_seqlens [N + 1] int32 on the device, states [N, D, S]."""
    T, _ = _lead(x, 2)
    return _ssm_fwd(x, dt, A, B, C, cu_seqlens, _packed(cu_seqlens, x.device), T, skip, z, dt_bias, initial_state,
                    softplus, y, final_state, output_final_state, o_dtype, stream, workspace)


def _ssm_fwd(x, dt, A, B, C, cu, N, T, skip, z, dt_bias, s0, softplus, y, sT, want_state, o_dtype, stream, workspace):
    dev, D = x.device, x.shape[-1]
    code, o_dtype = _types(x, o_dtype, y)
    ins, S, G = _ssm_in(x, dt, A, B, C, skip, z, dt_bias)
    s0p = _dense(s0, "initial_state", (N, D, S), _F32, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    sTp = _dense(sT, "final_state", (N, D, S), _F32, dev)
    nbytes = _lib.workspace_size("kda_ssm_fwd_workspace_size" if cu is None else "kda_ssm_varlen_fwd_workspace_size",
                                 N, T, D, S, G, code)
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty(x.shape, dtype=o_dtype, device=dev)
            yp = y.data_ptr()
        if sT is None and want_state:
            sT = torch.empty((N, D, S), dtype=_F32, device=dev)
            sTp = sT.data_ptr()
        ws, n, _keep = _scratch(nbytes, workspace, dev)
        tail = (s0p, yp, sTp) + ((N,) if cu is None else ()) + (T, D, S, G, code, _DTYPES[o_dtype],
                                                                _lib.KDA_SSM_SOFTPLUS if softplus else 0, ws, n, st)
        if cu is None:
            _lib.call("kda_ssm_fwd", *ins, *tail)
        else:
            _lib.call("kda_ssm_varlen_fwd", *ins, cu.data_ptr(), N, *tail)
    return y, sT


def kda_ssm_step(x, dt, A, B, C, state, skip=None, z=None, dt_bias=None, *, softplus=True, y=None, o_dtype=None,
                 stream=None):
    """One token per sequence: x, dt, z [N, D], B, C [N, G, S]; state [N, D, S] fp32
    updated in place.  Returns y [N, D]."""
    N, D = _lead(x, 2)
    dev = x.device
    code, o_dtype = _types(x, o_dtype, y)
    ins, S, G = _ssm_in(x, dt, A, B, C, skip, z, dt_bias)
    sp = _dense(state, "state", (N, D, S), _F32, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty(x.shape, dtype=o_dtype, device=dev)
            yp = y.data_ptr()
        _lib.call("kda_ssm_step", *ins, sp, yp, N, D, S, G, code, _DTYPES[o_dtype],
                  _lib.KDA_SSM_SOFTPLUS if softplus else 0, st)
    return y


def kda_ssm_bwd(x, dt, A, B, C, skip, z, dt_bias, initial_state, grad_y, grad_final_state=None, *, softplus=True,
                want_initial_state_grad=True, stream=None, workspace=None):
    """Backward of kda_ssm_fwd: gradients of sum(y * grad_y) + sum(final_state * grad_final_state).

    grad_y [B, T, D] and grad_final_state [B, D, S] (or None) fp32.  Returns fp32
    (grad_x, grad_dt, grad_A, grad_B, grad_C, grad_skip, grad_z, grad_dt_bias,
    grad_initial_state), None for an input that is None and for a state gradient
    that is not wanted."""
    N, T, _ = _lead(x, 3)
    return _ssm_bwd(x, dt, A, B, C, None, N, T, skip, z, dt_bias, initial_state, grad_y, grad_final_state, softplus,
                    want_initial_state_grad, stream, workspace)


def kda_ssm_varlen_bwd(x, dt, A, B, C, cu_seqlens, skip, z, dt_bias, initial_state, grad_y, grad_final_state=None, *,
                       softplus=True, want_initial_state_grad=True, stream=None, workspace=None):
    """Backward of kda_ssm_varlen_fwd (packed layouts, states [N, D, S])."""
    T, _ = _lead(x, 2)
    return _ssm_bwd(x, dt, A, B, C, cu_seqlens, _packed(cu_seqlens, x.device), T, skip, z, dt_bias, initial_state,
                    grad_y, grad_final_state, softplus, want_initial_state_grad, stream, workspace)


def _ssm_bwd(x, dt, A, B, C, cu, N, T, skip, z, dt_bias, s0, gy, gsT, softplus, want_gs0, stream, workspace):
    dev, D = x.device, x.shape[-1]
    code, _ = _types(x, None, None)
    ins, S, G = _ssm_in(x, dt, A, B, C, skip, z, dt_bias)
    s0p = _dense(s0, "initial_state", (N, D, S), _F32, dev)
    gyp = _dense(gy, "grad_y", x.shape, _F32, dev)
    gsTp = _dense(gsT, "grad_final_state", (N, D, S), _F32, dev)
    nbytes = _lib.workspace_size("kda_ssm_bwd_workspace_size" if cu is None else "kda_ssm_varlen_bwd_workspace_size",
                                 N, T, D, S, G, code)
    with _on(dev, stream) as st:
        f32 = dict(dtype=_F32, device=dev)
        gx, gdt, gA = torch.empty(x.shape, **f32), torch.empty(x.shape, **f32), torch.empty((D, S), **f32)
        gB, gC = torch.empty(B.shape, **f32), torch.empty(C.shape, **f32)
        gskip = torch.empty(D, **f32) if skip is not None else None
        gz = torch.empty(x.shape, **f32) if z is not None else None
        gbias = torch.empty(D, **f32) if dt_bias is not None else None
        gs0 = torch.empty((N, D, S), **f32) if want_gs0 else None
        ws, n, _keep = _scratch(nbytes, workspace, dev)
        grads = (gx, gdt, gA, gB, gC, gskip, gz, gbias, gs0)
        tail = (s0p, gyp, gsTp, *(None if g is None else g.data_ptr() for g in grads)) + (
            (N,) if cu is None else ()) + (T, D, S, G, code, _lib.KDA_SSM_SOFTPLUS if softplus else 0, ws, n, st)
        if cu is None:
            _lib.call("kda_ssm_bwd", *ins, *tail)
        else:
            _lib.call("kda_ssm_varlen_bwd", *ins, cu.data_ptr(), N, *tail)
    return grads
