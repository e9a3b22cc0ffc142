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
An output (y, a state, the workspace) that shares memory with an input or another
output is refused; a final state may be the initial state itself.
All tensors are on one CUDA device; the work runs on ``stream``, or on that
device's current stream, and new tensors belong to that stream.
"""
from __future__ import annotations

import functools

import torch

from . import _lib

__all__ = ["kda_conv_fwd", "kda_conv_varlen_fwd", "kda_conv_step", "kda_conv_bwd", "kda_conv_varlen_bwd",
           "kda_ssm_fwd", "kda_ssm_varlen_fwd", "kda_ssm_step", "kda_ssm_bwd", "kda_ssm_varlen_bwd",
           "conv_bwd_workspace_size", "ssm_bwd_workspace_size", "ssm_varlen_bwd_workspace_size"]

_DTYPES = {torch.float32: _lib.KDA_F32, torch.bfloat16: _lib.KDA_BF16}
_F32 = torch.float32


# ------------------------------------------------------------------ arguments
# A decode step's kernel takes a few microseconds, so the checks of a call are
# written to pass quickly: one condition per tensor, the message only on failure.
def _explain(t, name, shape, dtype, index):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on CUDA device {index}")


def _dense(t, name, shape, dtype, index):
    """Pointer of a contiguous tensor on CUDA device `index` (None for None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
        return t.data_ptr()
    _explain(t, name, shape, dtype, index)
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, shape, lead, dtype, index):
    """(pointer, row stride) of a token-major tensor whose first `lead`
    dimensions count tokens; the rest is one contiguous row."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _explain(t, name, shape, dtype, index)
    row = shape[-1] if len(shape) == lead + 1 else shape[-1] * shape[-2]
    if t.is_contiguous():
        return t.data_ptr(), row
    stride = t.stride()
    inner, ok = 1, True
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
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    o_dtype = y.dtype if y is not None else x.dtype if o_dtype is None else o_dtype
    o_code = _DTYPES.get(o_dtype)
    if o_code is None:
        raise ValueError(f"unsupported output dtype {o_dtype}")
    return code, o_dtype, o_code


_INT_MAX = (1 << 31) - 1   # the C ABI's int: ctypes drops the bits above without a word


def _lead(x, dims):
    shape = x.shape
    if len(shape) != dims:
        raise ValueError(f"x has {len(shape)} dimensions, expected {dims}")
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:
        raise ValueError(f"x has shape {tuple(shape)}: at most {_INT_MAX} sequences and tokens each")
    return shape


def _packed(cu_seqlens, x):
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected (N + 1,)")
    if cu_seqlens.shape[0] > _INT_MAX:
        raise ValueError(f"cu_seqlens has {cu_seqlens.shape[0] - 1} sequences, at most 65535 are supported")
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, x.get_device())
    return cu_seqlens.shape[0] - 1


_current = torch.cuda.current_device


class _switched:
    """Makes `stream` (or CUDA device `index`) current for a call that names another one."""
    __slots__ = ("guards",)

    def __init__(self, index, stream):
        if index < 0:
            raise ValueError("the tensors are not on a CUDA device (there is no CPU path)")
        self.guards = (torch.cuda.device(index),)
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, the tensors on CUDA device {index}")
            self.guards += (torch.cuda.stream(stream),)

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _elsewhere(index, stream):
    """Whether a call has to switch first: to a stream of its own, or to its
    tensors' device.  (A CPU tensor's index is -1: refused by _switched.)"""
    return stream is not None or index < 0 or _current() != index


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)   # the handle without a Stream object


def _new(x, ld, dtype):
    """New tensor of x's shape on its device (ld: x's row stride)."""
    if dtype is x.dtype and ld == x.shape[-1]:   # x is contiguous: the cheapest allocation
        return torch.empty_like(x)
    return x.new_empty(x.shape, dtype=dtype)


def _scratch(nbytes, workspace, x):
    if nbytes == 0:
        return None, 0, None
    if workspace is None:
        workspace = x.new_empty(nbytes, dtype=torch.uint8)
    elif workspace.device != x.device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel(), workspace


@functools.lru_cache(maxsize=None)
def _entry(name):
    return getattr(_lib.load(), name)


def _raise(status, name):
    raise _lib.KdaError(status, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def conv_bwd_workspace_size(tokens, D, W):
    """Workspace bytes of kda_conv_bwd / kda_conv_varlen_bwd for `tokens` tokens in all."""
    return _lib.workspace_size("kda_conv_bwd_workspace_size", tokens, D, W)


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
    return _conv_fwd(x, weight, bias, cu_seqlens, _packed(cu_seqlens, x), T, initial_state, silu, y, final_state,
                     output_final_state, o_dtype, stream)


def _conv_params(weight, bias, D, dev):
    shape = weight.shape
    if len(shape) != 2 or shape[0] != D:
        raise ValueError(f"weight has shape {tuple(shape)}, expected ({D}, W)")
    return (_dense(weight, "weight", shape, _F32, dev),
            None if bias is None else _dense(bias, "bias", (D,), _F32, dev), shape[1])


def _conv_fwd(x, weight, bias, cu, N, T, s0, silu, y, sT, want_state, o_dtype, stream):
    dev, D = x.get_device(), x.shape[-1]
    code, o_dtype, o_code = _types(x, o_dtype, y)
    xp, ldx = _rows(x, "x", x.shape, x.dim() - 1, x.dtype, dev)
    wp, bp, W = _conv_params(weight, bias, D, dev)
    s0p = _dense(s0, "initial_state", (N, W - 1, D), x.dtype, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    sTp = _dense(sT, "final_state", (N, W - 1, D), x.dtype, dev)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return _conv_fwd(x, weight, bias, cu, N, T, s0, silu, y, sT, want_state, o_dtype, None)
    st = _raw_stream(dev)
    if y is None:
        y = _new(x, ldx, o_dtype)
        yp = y.data_ptr()
    if sT is None and want_state:
        sT = torch.empty_like(s0) if s0 is not None else x.new_empty((N, W - 1, D))
        sTp = sT.data_ptr()
    mode = _lib.KDA_CONV_SILU if silu else 0
    if cu is None:
        status = _entry("kda_conv_fwd")(xp, ldx, wp, bp, s0p, yp, sTp, N, T, D, W, code, o_code, mode, st)
        if status:
            _raise(status, "kda_conv_fwd")
    else:
        status = _entry("kda_conv_varlen_fwd")(
            xp, ldx, wp, bp, cu.data_ptr(), N, s0p, yp, sTp, T, D, W, code, o_code, mode, st)
        if status:
            _raise(status, "kda_conv_varlen_fwd")
    return y, sT


def kda_conv_step(x, weight, bias, state, *, silu=True, y=None, o_dtype=None, stream=None):
    """One token per sequence: x [N, D]; state [N, W - 1, D] of x's dtype, moved on
    by one token in place.  Returns y [N, D]."""
    N, D = _lead(x, 2)
    dev = x.get_device()
    code, o_dtype, o_code = _types(x, o_dtype, y)
    xp, ldx = _rows(x, "x", x.shape, 1, x.dtype, dev)
    wp, bp, W = _conv_params(weight, bias, D, dev)
    sp = _dense(state, "state", (N, W - 1, D), x.dtype, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return kda_conv_step(x, weight, bias, state, silu=silu, y=y, o_dtype=o_dtype)
    st = _raw_stream(dev)
    if y is None:
        y = _new(x, ldx, o_dtype)
        yp = y.data_ptr()
    status = _entry("kda_conv_step")(
        xp, ldx, wp, bp, sp, yp, N, D, W, code, o_code, _lib.KDA_CONV_SILU if silu else 0, st)
    if status:
        _raise(status, "kda_conv_step")
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
    return _conv_bwd(x, weight, bias, cu_seqlens, _packed(cu_seqlens, x), T, initial_state, grad_y, grad_final_state,
                     silu, want_initial_state_grad, stream, workspace)


def _conv_bwd(x, weight, bias, cu, N, T, s0, gy, gsT, silu, want_gs0, stream, workspace):
    dev, D = x.get_device(), x.shape[-1]
    code = _types(x, None, None)[0]
    xp, ldx = _rows(x, "x", x.shape, x.dim() - 1, x.dtype, dev)
    wp, bp, W = _conv_params(weight, bias, D, dev)
    s0p = _dense(s0, "initial_state", (N, W - 1, D), x.dtype, dev)
    gyp = _dense(gy, "grad_y", x.shape, _F32, dev)
    gsTp = _dense(gsT, "grad_final_state", (N, W - 1, D), _F32, dev)
    nbytes = conv_bwd_workspace_size(T if cu is not None else N * T, D, W)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return _conv_bwd(x, weight, bias, cu, N, T, s0, gy, gsT, silu, want_gs0, None, workspace)
    st = _raw_stream(dev)
    gx, gw = x.new_empty(x.shape, dtype=_F32), torch.empty_like(weight)
    gb = torch.empty_like(bias) if bias is not None else None
    gs0 = x.new_empty((N, W - 1, D), dtype=_F32) if want_gs0 else None
    ws, n, _keep = _scratch(nbytes, workspace, x)
    grads = (gx.data_ptr(), gw.data_ptr(), _ptr(gb), _ptr(gs0))
    mode = _lib.KDA_CONV_SILU if silu else 0
    if cu is None:
        status = _entry("kda_conv_bwd")(xp, ldx, wp, bp, s0p, gyp, gsTp, *grads, N, T, D, W, code, mode, ws, n, st)
        if status:
            _raise(status, "kda_conv_bwd")
    else:
        status = _entry("kda_conv_varlen_bwd")(
            xp, ldx, wp, bp, cu.data_ptr(), N, s0p, gyp, gsTp, *grads, T, D, W, code, mode, ws, n, st)
        if status:
            _raise(status, "kda_conv_varlen_bwd")
    return gx, gw, gb, gs0


# ------------------------------------------------------------------ selective scan
def _ssm_in(x, dt, A, B, C, skip, z, dt_bias):
    """Checked (pointers and row strides in the C ABI's order, S, G)."""
    dev, shape, lead, ty = x.get_device(), x.shape, x.dim() - 1, x.dtype
    D = shape[-1]
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError(f"A has shape {tuple(A.shape)}, expected ({D}, S)")
    S = A.shape[1]
    if B.dim() != lead + 2:
        raise ValueError(f"B has {B.dim()} dimensions, expected {lead + 2}")
    G = B.shape[lead]
    bc = shape[:lead] + (G, S)
    if (x.is_contiguous() and dt.dtype is ty and dt.shape == shape and dt.is_contiguous() and dt.get_device() == dev
            and A.dtype is _F32 and A.is_contiguous() and A.get_device() == dev
            and B.dtype is ty and B.shape == bc and B.is_contiguous() and B.get_device() == dev
            and C.dtype is ty and C.shape == bc and C.is_contiguous() and C.get_device() == dev
            and (z is None or (z.dtype is ty and z.shape == shape and z.is_contiguous() and z.get_device() == dev))):
        # everything dense: the common call, and the cheapest way through
        row = G * S
        return (x.data_ptr(), D, dt.data_ptr(), D, A.data_ptr(), B.data_ptr(), row, C.data_ptr(), row,
                _dense(skip, "skip", (D,), _F32, dev), None if z is None else z.data_ptr(), D,
                _dense(dt_bias, "dt_bias", (D,), _F32, dev)), S, G
    skp, dbp = _dense(skip, "skip", (D,), _F32, dev), _dense(dt_bias, "dt_bias", (D,), _F32, dev)
    return (*_rows(x, "x", shape, lead, ty, dev), *_rows(dt, "dt", shape, lead, ty, dev),
            _dense(A, "A", A.shape, _F32, dev), *_rows(B, "B", bc, lead, ty, dev), *_rows(C, "C", bc, lead, ty, dev),
            skp, *_rows(z, "z", shape, lead, ty, dev), dbp), S, G


def kda_ssm_fwd(x, dt, A, B, C, skip=None, z=None, dt_bias=None, initial_state=None, *, softplus=True, y=None,
                final_state=None, output_final_state=True, o_dtype=None, stream=None):
    """Selective scan over equal-length sequences.

    x, dt, z [B, T, D] and B, C [B, T, G, S] (bf16 or fp32); A [D, S], skip and
    dt_bias [D], initial_state [B, D, S] fp32; skip, z, dt_bias, initial_state may
    be None.  softplus=False takes dt + dt_bias itself as the step size.  Returns
    (y [B, T, D] in o_dtype, by default x's dtype; final_state [B, D, S] or None)."""
    N, T, _ = _lead(x, 3)
    return _ssm_fwd(x, dt, A, B, C, None, N, T, skip, z, dt_bias, initial_state, softplus, y, final_state,
                    output_final_state, o_dtype, stream)


def kda_ssm_varlen_fwd(x, dt, A, B, C, cu_seqlens, skip=None, z=None, dt_bias=None, initial_state=None, *,
                       softplus=True, y=None, final_state=None, output_final_state=True, o_dtype=None, stream=None):
    """kda_ssm_fwd over N packed sequences: x, dt, z [T, D], B, C [T, G, S],
    cu_seqlens [N + 1] int32 on the device, states [N, D, S]."""
    T, _ = _lead(x, 2)
    return _ssm_fwd(x, dt, A, B, C, cu_seqlens, _packed(cu_seqlens, x), T, skip, z, dt_bias, initial_state, softplus,
                    y, final_state, output_final_state, o_dtype, stream)


def _ssm_fwd(x, dt, A, B, C, cu, N, T, skip, z, dt_bias, s0, softplus, y, sT, want_state, o_dtype, stream):
    dev, D = x.get_device(), x.shape[-1]
    code, o_dtype, o_code = _types(x, o_dtype, y)
    ins, S, G = _ssm_in(x, dt, A, B, C, skip, z, dt_bias)
    s0p = _dense(s0, "initial_state", (N, D, S), _F32, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    sTp = _dense(sT, "final_state", (N, D, S), _F32, dev)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return _ssm_fwd(x, dt, A, B, C, cu, N, T, skip, z, dt_bias, s0, softplus, y, sT, want_state, o_dtype, None)
    st = _raw_stream(dev)
    if y is None:
        y = _new(x, ins[1], o_dtype)
        yp = y.data_ptr()
    if sT is None and want_state:
        sT = torch.empty_like(s0) if s0 is not None else x.new_empty((N, D, S), dtype=_F32)
        sTp = sT.data_ptr()
    mode = _lib.KDA_SSM_SOFTPLUS if softplus else 0
    if cu is None:
        status = _entry("kda_ssm_fwd")(*ins, s0p, yp, sTp, N, T, D, S, G, code, o_code, mode, st)
        if status:
            _raise(status, "kda_ssm_fwd")
    else:
        status = _entry("kda_ssm_varlen_fwd")(
            *ins, cu.data_ptr(), N, s0p, yp, sTp, T, D, S, G, code, o_code, mode, st)
        if status:
            _raise(status, "kda_ssm_varlen_fwd")
    return y, sT


def kda_ssm_step(x, dt, A, B, C, state, skip=None, z=None, dt_bias=None, *, softplus=True, y=None, o_dtype=None,
                 stream=None):
    """One token per sequence: x, dt, z [N, D], B, C [N, G, S]; state [N, D, S] fp32
    updated in place.  Returns y [N, D]."""
    N, D = _lead(x, 2)
    dev = x.get_device()
    code, o_dtype, o_code = _types(x, o_dtype, y)
    ins, S, G = _ssm_in(x, dt, A, B, C, skip, z, dt_bias)
    sp = _dense(state, "state", (N, D, S), _F32, dev)
    yp = _dense(y, "y", x.shape, o_dtype, dev)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return kda_ssm_step(x, dt, A, B, C, state, skip, z, dt_bias, softplus=softplus, y=y, o_dtype=o_dtype)
    st = _raw_stream(dev)
    if y is None:
        y = _new(x, ins[1], o_dtype)
        yp = y.data_ptr()
    status = _entry("kda_ssm_step")(
        *ins, sp, yp, N, D, S, G, code, o_code, _lib.KDA_SSM_SOFTPLUS if softplus else 0, st)
    if status:
        _raise(status, "kda_ssm_step")
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
    return _ssm_bwd(x, dt, A, B, C, cu_seqlens, _packed(cu_seqlens, x), T, skip, z, dt_bias, initial_state, grad_y,
                    grad_final_state, softplus, want_initial_state_grad, stream, workspace)


def _ssm_bwd(x, dt, A, B, C, cu, N, T, skip, z, dt_bias, s0, gy, gsT, softplus, want_gs0, stream, workspace):
    dev, D = x.get_device(), x.shape[-1]
    code = _types(x, None, None)[0]
    ins, S, G = _ssm_in(x, dt, A, B, C, skip, z, dt_bias)
    s0p = _dense(s0, "initial_state", (N, D, S), _F32, dev)
    gyp = _dense(gy, "grad_y", x.shape, _F32, dev)
    gsTp = _dense(gsT, "grad_final_state", (N, D, S), _F32, dev)
    nbytes = _lib.workspace_size("kda_ssm_bwd_workspace_size" if cu is None else "kda_ssm_varlen_bwd_workspace_size",
                                 N, T, D, S, G, code)
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return _ssm_bwd(x, dt, A, B, C, cu, N, T, skip, z, dt_bias, s0, gy, gsT, softplus, want_gs0, None,
                            workspace)
    st = _raw_stream(dev)
    f32 = dict(dtype=_F32)
    gx, gdt, gA = x.new_empty(x.shape, **f32), x.new_empty(x.shape, **f32), torch.empty_like(A)
    gB, gC = x.new_empty(B.shape, **f32), x.new_empty(C.shape, **f32)
    gskip = torch.empty_like(skip) if skip is not None else None
    gz = x.new_empty(x.shape, **f32) if z is not None else None
    gbias = torch.empty_like(dt_bias) if dt_bias is not None else None
    gs0 = x.new_empty((N, D, S), **f32) if want_gs0 else None
    ws, n, _keep = _scratch(nbytes, workspace, x)
    grads = (gx, gdt, gA, gB, gC, gskip, gz, gbias, gs0)
    mode = _lib.KDA_SSM_SOFTPLUS if softplus else 0
    if cu is None:
        status = _entry("kda_ssm_bwd")(
            *ins, s0p, gyp, gsTp, *map(_ptr, grads), N, T, D, S, G, code, mode, ws, n, st)
        if status:
            _raise(status, "kda_ssm_bwd")
    else:
        status = _entry("kda_ssm_varlen_bwd")(
            *ins, cu.data_ptr(), N, s0p, gyp, gsTp, *map(_ptr, grads), T, D, S, G, code, mode, ws, n, st)
        if status:
            _raise(status, "kda_ssm_varlen_bwd")
    return grads
