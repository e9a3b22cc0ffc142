"""GPU: the short convolution and the selective scan at their limits: waits that run
out, boundaries that are wrong, and the launch shapes that only larger sizes reach."""
import pytest
import torch

import gated_delta_rule_133_b200 as kda
from gated_delta_rule_133_b200 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _stream():
    return torch.cuda.current_stream().cuda_stream


def test_reverse_walk_leaves_when_its_waits_run_out():
    """Every hand-over withheld: the blocks leave, the timeout is reported once, and the
    backward pass gives what it gave before."""
    g = torch.Generator().manual_seed(1)
    T, D, S = 200, 64, 16
    x, dt, gy = (torch.randn(1, T, D, generator=g).to(DEV) for _ in range(3))
    B, C = (torch.randn(1, T, 1, S, generator=g).to(DEV) for _ in range(2))
    A = -torch.rand(D, S, generator=g).to(DEV)
    before = kda.kda_ssm_bwd(x, dt, A, B, C, None, None, None, None, gy)
    kda.kda_check()
    lib = _lib.load()
    ws = torch.empty(1 << 17, dtype=torch.uint8, device=DEV)
    assert lib.kda_selftest_scan_timeout(1 << 20, ws.data_ptr(), ws.numel(), _stream()) == _lib.KDA_OK   # ~0.5 ms each
    assert lib.kda_check(_stream()) == _lib.KDA_ERR_TIMEOUT
    assert lib.kda_check(_stream()) == _lib.KDA_OK
    after = kda.kda_ssm_bwd(x, dt, A, B, C, None, None, None, None, gy)
    kda.kda_check()
    assert all(a is b or torch.equal(a, b) for a, b in zip(before, after))


@pytest.mark.parametrize("N,T,D", [(100, 8, 64), (2000, 64, 256)])
@pytest.mark.parametrize("states", [True, False])
def test_every_bad_sequence_is_reported(N, T, D, states):
    """Mostly empty batches, far more sequences than token tiles: a sequence that leaves
    the token axis is reported wherever it stands, with and without final states."""
    x, w = torch.randn(T, D, device=DEV), torch.randn(D, 4, device=DEV)
    bc, A = torch.randn(T, 1, 16, device=DEV), -torch.rand(D, 16, device=DEV)
    for k in (0, 1, 31, 32, N // 2, N - 1):
        cu = torch.tensor([0] + [T if k else T + 4] + [T if i < k else T + 4 for i in range(1, N)],
                          dtype=torch.int32, device=DEV)
        for call in (lambda: kda.kda_conv_varlen_fwd(x, w, None, cu, output_final_state=states),
                     lambda: kda.kda_conv_varlen_bwd(x, w, None, cu, None, x, want_initial_state_grad=states),
                     lambda: kda.kda_ssm_varlen_fwd(x, x, A, bc, bc, cu, output_final_state=states),
                     lambda: kda.kda_ssm_varlen_bwd(x, x, A, bc, bc, cu, None, None, None, None, x,
                                                    want_initial_state_grad=states)):
            call()
            with pytest.raises(kda.KdaError) as e:
                kda.kda_check()
            assert e.value.status == _lib.KDA_ERR_INVALID_ARG
            kda.kda_check()


def test_neighbours_in_one_buffer():
    """Tensors that touch without sharing memory are taken, and give what tensors of
    their own do; so does a state updated in place."""
    g = torch.Generator().manual_seed(2)
    N, T, D, S = 2, 16, 64, 16

    def arena(*shapes):
        sizes = [torch.Size(s).numel() for s in shapes]
        return [p.view(s) for p, s in zip(torch.empty(sum(sizes), device=DEV).split(sizes), shapes)]
    w, A = torch.randn(D, 4, generator=g).to(DEV), -torch.rand(D, S, generator=g).to(DEV)
    x, y, s0, sT = arena((N, T, D), (N, T, D), (N, 3, D), (N, 3, D))
    x.copy_(torch.randn(N, T, D, generator=g))
    s0.copy_(torch.randn(N, 3, D, generator=g))
    want = kda.kda_conv_fwd(x.clone(), w, None, s0.clone())
    kda.kda_conv_fwd(x, w, None, s0, y=y, final_state=sT)
    assert torch.equal(y, want[0]) and torch.equal(sT, want[1])
    kda.kda_conv_fwd(x, w, None, s0, y=y, final_state=s0)
    assert torch.equal(y, want[0]) and torch.equal(s0, want[1])
    x2, y, B, h, hT = arena((N, T, D), (N, T, D), (N, T, 1, S), (N, D, S), (N, D, S))
    for t in (x2, B, h):
        t.copy_(torch.randn(t.shape, generator=g))
    want = kda.kda_ssm_fwd(x2.clone(), x, A, B, B, None, None, None, h.clone())
    kda.kda_ssm_fwd(x2, x, A, B, B, None, None, None, h, y=y, final_state=hT)
    assert torch.equal(y, want[0]) and torch.equal(hT, want[1])
    kda.kda_ssm_fwd(x2, x, A, B, B, None, None, None, h, y=y, final_state=h)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    pool = torch.randn(N + 1, D, S, device=DEV)
    with pytest.raises(kda.KdaError):
        kda.kda_ssm_fwd(x2, x, A, B, B, None, None, None, pool[:N], final_state=pool[1:])
    kda.kda_check()


@pytest.mark.parametrize("cu", [[50, 100, 0, 50], [10, 0, 100], [0, 30, 20, 100], [0, 100, 99], [0] * 40 + [60, 40] + [100] * 40])
def test_decreasing_boundaries_are_reported(cu):
    """A token's sequence is searched for in order, so boundaries that decrease may leave
    rows out (the first list: rows 0 to 50 of a convolution): never without a report."""
    T, D = 100, 64
    x, w = torch.randn(T, D, device=DEV), torch.randn(D, 4, device=DEV)
    bc, A = torch.randn(T, 1, 16, device=DEV), -torch.rand(D, 16, device=DEV)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    for call in (lambda: kda.kda_conv_varlen_fwd(x, w, None, cu),
                 lambda: kda.kda_conv_varlen_bwd(x, w, None, cu, None, x),
                 lambda: kda.kda_ssm_varlen_fwd(x, x, A, bc, bc, cu),
                 lambda: kda.kda_ssm_varlen_bwd(x, x, A, bc, bc, cu, None, None, None, None, x)):
        call()
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check()
        assert e.value.status == _lib.KDA_ERR_INVALID_ARG
        kda.kda_check()
