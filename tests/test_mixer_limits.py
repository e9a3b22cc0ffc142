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
