"""CPU: refusals of the short convolution's and the selective scan's entry points at
their limits (only calls that fail validation are made)."""
import ctypes

import pytest

from gated_delta_rule_133_b200 import _lib

W0 = 1 << 20   # a 256-byte aligned fake address: never dereferenced, validation fails first
BAD, UNSUP, OK = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_OK


@pytest.mark.parametrize("limit,ws,nbytes", [(0, W0, 1 << 17), (-1, W0, 1 << 17), ((1 << 32) + 1, W0, 1 << 17),
                                             (1 << 20, None, 1 << 17), (1 << 20, W0 + 16, 1 << 17), (1 << 20, W0, 4096)])
def test_scan_timeout_selftest_validation(limit, ws, nbytes):
    assert _lib.load().kda_selftest_scan_timeout(ctypes.c_longlong(limit), ws, nbytes, None) == BAD


F = 1 << 24    # fake buffers, far apart
BF16, F32 = _lib.KDA_BF16, _lib.KDA_F32


def _clashes(entry, args, out, ins, allowed=()):
    """Every output moved over every input and every other output, by their first and by
    their last bytes, is refused.  out, ins: argument index -> bytes from its address."""
    f = getattr(_lib.load(), entry)
    for i, ni in out.items():
        for j, nj in {**ins, **out}.items():
            if i == j or (i, j) in allowed:
                continue
            for at in (args[j], args[j] + (nj - 1) // 256 * 256, args[j] - (ni - 1) // 256 * 256):
                a = list(args)
                a[i] = at
                assert f(*a) == BAD, (entry, i, j, at - args[j])


def test_conv_outputs_that_share_memory():
    """kda_conv_*: 2 x 9 tokens of 64 channels, 4 taps, x bf16 in rows of 80; state rows bf16."""
    n, D = 18, 64
    x, w, b, cu, st, st32 = (n - 1) * 160 + 128, D * 16, D * 4, 12, 2 * 3 * D * 2, 2 * 3 * D * 4
    #       x  ldx w      b      s0     y      sT
    fwd = (F, 80, 2 * F, 3 * F, 4 * F, 5 * F, 6 * F, 2, 9, D, 4, BF16, F32, 1, None)
    _clashes("kda_conv_fwd", fwd, {5: n * D * 4, 6: st}, {0: x, 2: w, 3: b, 4: st}, allowed={(6, 4)})
    part = list(fwd)
    for shift in (16, st - 16, -16):          # in place as a whole, not in part
        part[6] = part[4] + shift
        assert _lib.load().kda_conv_fwd(*part) == BAD, shift
    varlen = (F, 80, 2 * F, 3 * F, 7 * F, 2, 4 * F, 5 * F, 6 * F, n, D, 4, BF16, F32, 1, None)
    _clashes("kda_conv_varlen_fwd", varlen, {7: n * D * 4, 8: st}, {0: x, 2: w, 3: b, 4: cu, 6: st}, allowed={(8, 6)})
    step = (F, 80, 2 * F, 3 * F, 4 * F, 5 * F, 2, D, 4, BF16, F32, 1, None)
    _clashes("kda_conv_step", step, {4: st, 5: 2 * D * 4}, {0: 160 + 128, 2: w, 3: b})
    size = ctypes.c_size_t(0)
    assert _lib.load().kda_conv_bwd_workspace_size(n, D, 4, ctypes.byref(size)) == OK
    #      x  ldx w      b      s0     gy     gsT    gx     gw     gb      gs0
    bwd = (F, 80, 2 * F, 3 * F, 4 * F, 5 * F, 6 * F, 7 * F, 8 * F, 9 * F, 10 * F, 2, 9, D, 4, BF16, 1, 11 * F, size.value,
           None)
    _clashes("kda_conv_bwd", bwd, {7: n * D * 4, 8: w, 9: b, 10: st32, 17: size.value},
             {0: x, 2: w, 3: b, 4: st, 5: n * D * 4, 6: st32})
    empty = list(fwd)                          # no tokens: the states are still copied
    empty[8], empty[6] = 0, empty[4] + 16
    assert _lib.load().kda_conv_fwd(*empty) == BAD


def test_ssm_outputs_that_share_memory():
    """kda_ssm_*: 2 x 9 tokens of 64 channels, 16 states, 2 groups, bf16."""
    n, D, S, G = 18, 64, 16, 2
    act, bc, A, v, cu, st = n * D * 2, n * G * S * 2, D * S * 4, D * 4, 12, 2 * D * S * 4
    ins = (F, D, 2 * F, D, 3 * F, 4 * F, G * S, 5 * F, G * S, 6 * F, 7 * F, D, 8 * F)   # x dt A B C skip z dt_bias
    sizes = {0: act, 2: act, 4: A, 5: bc, 7: bc, 9: v, 10: act, 12: v}
    fwd = ins + (9 * F, 10 * F, 11 * F, 2, 9, D, S, G, BF16, F32, 1, None)
    _clashes("kda_ssm_fwd", fwd, {14: n * D * 4, 15: st}, {**sizes, 13: st}, allowed={(15, 13)})
    part = list(fwd)
    for shift in (16, st - 16, -16):
        part[15] = part[13] + shift
        assert _lib.load().kda_ssm_fwd(*part) == BAD, shift
    varlen = ins + (12 * F, 2, 9 * F, 10 * F, 11 * F, n, D, S, G, BF16, F32, 1, None)
    _clashes("kda_ssm_varlen_fwd", varlen, {16: n * D * 4, 17: st}, {**sizes, 13: cu, 15: st}, allowed={(17, 15)})
    step = ins + (9 * F, 10 * F, 2, D, S, G, BF16, F32, 1, None)
    one = {0: 256, 2: 256, 4: A, 5: 128, 7: 128, 9: v, 10: 256, 12: v}
    _clashes("kda_ssm_step", step, {13: st, 14: 2 * D * 4}, one)
    size = ctypes.c_size_t(0)
    assert _lib.load().kda_ssm_bwd_workspace_size(2, 9, D, S, G, BF16, ctypes.byref(size)) == OK
    # s0 gy gsT | gx gdt gA gB gC gskip gz gdt_bias gs0
    bwd = ins + tuple(k * F for k in range(9, 21)) + (2, 9, D, S, G, BF16, 1, 21 * F, size.value, None)
    _clashes("kda_ssm_bwd", bwd, {16: 2 * act, 17: 2 * act, 18: A, 19: 2 * bc, 20: 2 * bc, 21: v, 22: 2 * act, 23: v,
                                  24: st, 32: size.value}, {**sizes, 13: st, 14: 2 * act, 15: st})


def test_sizes_beyond_an_int_are_refused():
    """2^32 + 5 tokens are not 5 (on the meta device: nothing is allocated)."""
    import torch
    import gated_delta_rule_133_b200 as kda

    def meta(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")
    big, w, A = (1 << 32) + 5, meta(8, 4), meta(8, 16)
    cu = meta(big + 1, dtype=torch.int32)
    for x in (meta(1, big, 8), meta(big, 1, 8)):
        bc = meta(*x.shape[:2], 1, 16)
        for call in (lambda: kda.kda_conv_fwd(x, w), lambda: kda.kda_conv_bwd(x, w, None, None, x),
                     lambda: kda.kda_ssm_fwd(x, x, A, bc, bc),
                     lambda: kda.kda_ssm_bwd(x, x, A, bc, bc, None, None, None, None, x)):
            with pytest.raises(ValueError, match="at most 2147483647"):
                call()
    x, bc = meta(big, 8), meta(big, 1, 16)
    for call in (lambda: kda.kda_conv_step(x, w, None, meta(big, 3, 8)), lambda: kda.kda_conv_varlen_fwd(x, w, None, cu),
                 lambda: kda.kda_ssm_step(x, x, A, bc, bc, meta(big, 8, 16)),
                 lambda: kda.kda_ssm_varlen_fwd(x, x, A, bc, bc, cu)):
        with pytest.raises(ValueError, match="at most 2147483647"):
            call()
    x, bc = meta(9, 8), meta(9, 1, 16)
    for call in (lambda: kda.kda_conv_varlen_fwd(x, w, None, cu), lambda: kda.kda_ssm_varlen_fwd(x, x, A, bc, bc, cu),
                 lambda: kda.kda_conv_varlen_bwd(x, w, None, cu, None, x)):
        with pytest.raises(ValueError, match="at most 65535"):
            call()
