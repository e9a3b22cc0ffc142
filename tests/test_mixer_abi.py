"""CPU: the short convolution's and the selective scan's entry points validate
their arguments on the host and refuse what they do not take, with nothing
launched (only calls that fail validation, or that have nothing to do, are made)."""
import ctypes

import pytest
import torch

import gated_delta_rule_133_b200 as kda
from gated_delta_rule_133_b200 import _lib

P = 256        # a 16-byte aligned fake address: never dereferenced, validation fails first
W0 = 1 << 20   # a 256-byte aligned one
BAD, UNSUP, OK = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_OK
BF16, F32 = _lib.KDA_BF16, _lib.KDA_F32


def _with(args, **at):
    a = list(args)
    for i, v in at.items():
        a[int(i[1:])] = v
    return a


#       x  ldx w  b  s0    y  sT    B  T  D   W  dtype o_dtype mode stream
CONV = (P, 64, P, P, None, P, None, 2, 9, 64, 4, BF16, F32, 1, None)


@pytest.mark.parametrize("at,want", [
    (dict(_0=None), BAD), (dict(_0=P + 8), BAD), (dict(_2=None), BAD), (dict(_2=P + 4), BAD), (dict(_3=P + 4), BAD),
    (dict(_4=P + 8), BAD), (dict(_5=None), BAD), (dict(_5=P + 2), BAD), (dict(_6=P + 8), BAD),
    (dict(_7=-1), BAD), (dict(_8=-1), BAD), (dict(_9=0), BAD), (dict(_10=0), BAD), (dict(_11=5), BAD),
    (dict(_12=9), BAD), (dict(_13=2), BAD), (dict(_13=-1), BAD),
    (dict(_1=63), BAD), (dict(_1=56), BAD), (dict(_1=68), BAD), (dict(_1=1 << 30), BAD),   # row strides
    (dict(_9=60, _1=64), UNSUP), (dict(_10=1), UNSUP), (dict(_10=5), UNSUP), (dict(_9=1 << 21, _1=1 << 21), UNSUP),
    (dict(_7=1 << 16, _8=1 << 16), UNSUP),                                                 # tokens beyond 31 bits
])
def test_conv_fwd_validation(at, want):
    assert _lib.load().kda_conv_fwd(*_with(CONV, **at)) == want


def test_conv_varlen_and_step_validation():
    lib = _lib.load()
    #       x  ldx w  b  cu N  s0    y  sT    T  D   W  dtype o_dtype mode stream
    varlen = (P, 64, P, P, P, 3, None, P, None, 9, 64, 4, BF16, F32, 1, None)
    for at, want in ((dict(_4=None), BAD), (dict(_4=P + 2), BAD), (dict(_5=-1), BAD), (dict(_5=65536), BAD),
                     (dict(_5=0), BAD), (dict(_9=-1), BAD), (dict(_0=None), BAD), (dict(_11=7), UNSUP)):
        assert lib.kda_conv_varlen_fwd(*_with(varlen, **at)) == want, at
    assert lib.kda_conv_varlen_fwd(*_with(varlen, _0=None, _4=None, _5=0, _7=None, _9=0)) == OK   # nothing at all
    #       x  ldx w  b  st y  N  D   W  dtype o_dtype mode stream
    step = (P, 64, P, P, P, P, 3, 64, 4, BF16, F32, 1, None)
    for at, want in ((dict(_4=None), BAD), (dict(_4=P + 8), BAD), (dict(_6=-1), BAD), (dict(_8=5), UNSUP),
                     (dict(_5=None), BAD), (dict(_10=3), BAD), (dict(_11=4), BAD)):
        assert lib.kda_conv_step(*_with(step, **at)) == want, at
    assert lib.kda_conv_step(*_with(step, _0=None, _4=None, _5=None, _6=0)) == OK


def test_conv_bwd_validation():
    lib = _lib.load()
    need = kda.conv_bwd_workspace_size(18, 64, 4)
    assert need >= 5 * 64 * 4 and kda.conv_bwd_workspace_size(0, 64, 4) == 0
    #      x  ldx w  b  s0    gy gsT   gx gw gb gs0   B  T  D   W  dtype mode ws  bytes stream
    bwd = (P, 64, P, P, None, P, None, P, P, P, None, 2, 9, 64, 4, BF16, 1, W0, need, None)
    for at, want in ((dict(_5=None), BAD), (dict(_7=None), BAD), (dict(_8=None), BAD), (dict(_9=P + 4), BAD),
                     (dict(_10=P + 4), BAD), (dict(_6=P + 4), BAD), (dict(_17=None), BAD), (dict(_17=W0 + 16), BAD),
                     (dict(_18=need - 1), BAD), (dict(_14=6), UNSUP), (dict(_16=8), BAD)):
        assert lib.kda_conv_bwd(*_with(bwd, **at)) == want, at
    out = ctypes.c_size_t(0)
    assert lib.kda_conv_bwd_workspace_size(-1, 64, 4, ctypes.byref(out)) == BAD
    assert lib.kda_conv_bwd_workspace_size(8, 64, 4, None) == BAD
    assert lib.kda_conv_bwd_workspace_size(8, 60, 4, ctypes.byref(out)) == UNSUP


# x ldx dt lddt A B ldb C ldc skip z ldz dt_bias
IN = (P, 64, P, 64, P, P, 32, P, 32, P, P, 64, P)
#            s0    y  sT    B  T  D   S   G  dtype o_dtype mode stream
SSM = IN + (None, P, None, 2, 9, 64, 16, 2, BF16, F32, 1, None)


@pytest.mark.parametrize("at,want", [
    (dict(_0=None), BAD), (dict(_0=P + 8), BAD), (dict(_2=None), BAD), (dict(_4=None), BAD), (dict(_4=P + 4), BAD),
    (dict(_5=None), BAD), (dict(_5=P + 8), BAD), (dict(_7=None), BAD), (dict(_9=P + 4), BAD), (dict(_10=P + 8), BAD),
    (dict(_12=P + 4), BAD), (dict(_13=P + 4), BAD), (dict(_14=None), BAD), (dict(_15=P + 4), BAD),
    (dict(_1=60), BAD), (dict(_3=56), BAD), (dict(_6=24), BAD), (dict(_8=36), BAD), (dict(_11=0), BAD),
    (dict(_6=1 << 30), BAD), (dict(_16=-1), BAD), (dict(_17=-1), BAD), (dict(_18=0), BAD), (dict(_19=0), BAD),
    (dict(_20=0), BAD), (dict(_21=7), BAD), (dict(_22=7), BAD), (dict(_23=2), BAD),
    (dict(_19=24, _6=64, _8=64), UNSUP), (dict(_19=128, _6=256, _8=256), UNSUP), (dict(_20=3, _6=64, _8=64), UNSUP),
    (dict(_20=16, _6=256, _8=256), UNSUP), (dict(_16=1 << 16, _17=1 << 16), UNSUP),
])
def test_ssm_fwd_validation(at, want):
    assert _lib.load().kda_ssm_fwd(*_with(SSM, **at)) == want


def test_ssm_varlen_step_and_bwd_validation():
    lib = _lib.load()
    varlen = IN + (P, 3, None, P, None, 9, 64, 16, 2, BF16, F32, 1, None)
    for at, want in ((dict(_13=None), BAD), (dict(_13=P + 1), BAD), (dict(_14=70000), BAD), (dict(_14=0), BAD),
                     (dict(_18=-1), BAD), (dict(_20=48, _6=128, _8=128), UNSUP)):
        assert lib.kda_ssm_varlen_fwd(*_with(varlen, **at)) == want, at
    step = IN + (P, P, 3, 64, 16, 2, BF16, F32, 1, None)
    for at, want in ((dict(_13=None), BAD), (dict(_13=P + 8), BAD), (dict(_14=None), BAD), (dict(_15=-1), BAD),
                     (dict(_17=20, _6=64, _8=64), UNSUP), (dict(_20=5), BAD)):
        assert lib.kda_ssm_step(*_with(step, **at)) == want, at
    assert lib.kda_ssm_step(*_with(step, _0=None, _13=None, _14=None, _15=0)) == OK
    need = kda.ssm_bwd_workspace_size(2, 9, 64, 16, 2)
    assert need >= 2 * 2 * 64 * 16 * 4   # a state per 8 tokens
    assert kda.ssm_bwd_workspace_size(2, 0, 64, 16, 2) == 0
    assert kda.ssm_varlen_bwd_workspace_size(3, 18, 64, 16, 2) > 0
    # s0 gy gsT gx gdt gA gB gC gskip gz gdt_bias gs0 B T D S G dtype mode ws bytes stream
    bwd = IN + (None, P, None, P, P, P, P, P, P, P, P, None, 2, 9, 64, 16, 2, BF16, 1, W0, need, None)
    for at, want in ((dict(_14=None), BAD), (dict(_16=None), BAD), (dict(_17=None), BAD), (dict(_18=None), BAD),
                     (dict(_19=None), BAD), (dict(_20=P + 4), BAD),
                     (dict(_21=None), BAD), (dict(_22=None), BAD), (dict(_23=None), BAD),   # wanted with their input
                     (dict(_9=None), BAD), (dict(_10=None), BAD), (dict(_12=None), BAD),    # and not without
                     (dict(_24=P + 4), BAD), (dict(_15=P + 4), BAD), (dict(_32=None), BAD), (dict(_32=W0 + 128), BAD),
                     (dict(_33=need - 1), BAD), (dict(_28=17, _6=64, _8=64), UNSUP)):
        assert lib.kda_ssm_bwd(*_with(bwd, **at)) == want, at
    out = ctypes.c_size_t(0)
    assert lib.kda_ssm_bwd_workspace_size(1, 8, 64, 16, 3, BF16, ctypes.byref(out)) == UNSUP
    assert lib.kda_ssm_varlen_bwd_workspace_size(70000, 8, 64, 16, 1, BF16, ctypes.byref(out)) == BAD


def test_outputs_that_share_memory_with_inputs():
    """y written over an input that other blocks still read: refused by its range, the
    rows' stride counted (bf16 inputs of 18 rows of 64, fp32 output: 2304 and 4608 bytes)."""
    lib = _lib.load()
    far = 1 << 24
    for at in (dict(_0=far, _5=far), dict(_0=far, _5=far + 2288), dict(_0=far, _5=far - 4592),
               dict(_0=far, _1=128, _5=far + 17 * 256 + 112)):
        assert lib.kda_conv_fwd(*_with(CONV, **at)) == BAD, at
    step = (far, 64, P, P, 8 * far, far + 256, 3, 64, 4, BF16, F32, 1, None)
    assert lib.kda_conv_step(*step) == BAD
    apart = [far * (i + 1) if v == P else v for i, v in enumerate(SSM)]
    for i, rows in ((0, 64), (2, 64), (5, 32), (7, 32), (10, 64)):     # x, dt, B, C, z
        assert lib.kda_ssm_fwd(*_with(apart, _14=apart[i] + 17 * 2 * rows)) == BAD, i
    one = apart[:13] + [20 * far, apart[0], 3, 64, 16, 2, BF16, F32, 1, None]
    assert lib.kda_ssm_step(*one) == BAD


def test_python_refuses_what_does_not_fit():
    x, w = torch.zeros(2, 8, 16), torch.zeros(16, 4)
    for call, word in (
            (lambda: kda.kda_conv_fwd(x, torch.zeros(8, 4)), "weight"),
            (lambda: kda.kda_conv_fwd(x[0], w), "dimensions"),
            (lambda: kda.kda_conv_fwd(x.double(), w), "dtype"),
            (lambda: kda.kda_conv_fwd(x, w, torch.zeros(8)), "bias"),
            (lambda: kda.kda_conv_fwd(x, w, None, torch.zeros(2, 4, 16)), "initial_state"),
            (lambda: kda.kda_conv_fwd(x, w, o_dtype=torch.float16), "output dtype"),
            (lambda: kda.kda_conv_fwd(x, w, y=torch.zeros(2, 8, 8)), "y has shape"),
            (lambda: kda.kda_conv_fwd(x, w), "CUDA"),                                   # there is no CPU path
            (lambda: kda.kda_conv_varlen_fwd(x[0], w, None, torch.zeros(3)), "cu_seqlens"),
            (lambda: kda.kda_conv_varlen_fwd(x[0], w, None, torch.zeros(2, 2, dtype=torch.int32)), "cu_seqlens"),
            (lambda: kda.kda_conv_step(x[0], w, None, torch.zeros(8, 2, 16)), "state"),
            (lambda: kda.kda_conv_bwd(x, w, None, None, torch.zeros(2, 8, 16, dtype=torch.bfloat16)), "grad_y")):
        with pytest.raises(ValueError, match=word):
            call()
    A, b = torch.zeros(16, 16), torch.zeros(2, 8, 1, 16)
    for call, word in (
            (lambda: kda.kda_ssm_fwd(x, x, torch.zeros(8, 16), b, b), "A has shape"),
            (lambda: kda.kda_ssm_fwd(x, x[:, :4], A, b, b), "dt has shape"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b[0], b), "B has"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b, b[..., :8]), "C has shape"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b, b, z=x[0]), "z has shape"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b, b, skip=torch.zeros(8)), "skip"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b, b, dt_bias=torch.zeros(16).double()), "dt_bias has dtype"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b, b, initial_state=torch.zeros(2, 16, 8)), "initial_state"),
            (lambda: kda.kda_ssm_fwd(x.transpose(0, 1), x.transpose(0, 1), A, b.transpose(0, 1), b.transpose(0, 1)),
             "stride from token to token"),
            (lambda: kda.kda_ssm_fwd(x, x, A, b, b), "CUDA"),
            (lambda: kda.kda_ssm_step(x[0], x[0], A, b[0], b[0], torch.zeros(8, 16, 4)), "state"),
            (lambda: kda.kda_ssm_bwd(x, x, A, b, b, None, None, None, None, x[0]), "grad_y")):
        with pytest.raises(ValueError, match=word):
            call()
