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
