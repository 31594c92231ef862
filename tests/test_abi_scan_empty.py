"""gla_scan_bwd_saved without states to read: saved buffers of 0 bytes (host-only: nothing is launched)."""
import ctypes

import pytest

from linear_rnn_b200 import _lib
from linear_rnn_b200._lib import GlaProblem


@pytest.mark.parametrize("B,H,L", [(0, 3, 4), (2, 0, 4), (0, 0, 0), (0, 3, 0)])
def test_an_empty_problem_needs_neither_saved_states_nor_workspace(B, H, L):
    p = GlaProblem(B, H, L, 8, 8, 64, 1.0, _lib.GLA_BF16, _lib.GLA_GATE_PER_KEY, 0)
    assert _lib.lib.gla_scan_saved_bytes(ctypes.byref(p)) == 0
    null = [None] * 10
    assert _lib.lib.gla_scan_bwd_saved(ctypes.byref(p), 0, *null, 0, None) == _lib.GLA_OK
    assert _lib.lib.gla_scan_bwd(ctypes.byref(p), 0, *null[:9], 0, None) == _lib.GLA_OK
    assert _lib.lib.gla_scan_bwd_saved(ctypes.byref(p), 9, *null, 0, None) == _lib.GLA_ERR_INVALID_ARG


def test_with_tokens_the_states_or_a_workspace_are_needed():
    p = GlaProblem(1, 1, 1, 8, 8, 64, 1.0, _lib.GLA_BF16, _lib.GLA_GATE_PER_KEY, 0)
    args = lambda saved, ws: [ctypes.c_void_p(16)] * 2 + [None, ctypes.c_void_p(16), None, saved] \
        + [ctypes.c_void_p(16)] * 2 + [None, ws]
    fn = _lib.lib.gla_scan_bwd_saved
    assert fn(ctypes.byref(p), 0, *args(None, None), 0, None) == _lib.GLA_ERR_INVALID_ARG
    assert fn(ctypes.byref(p), 0, *args(None, ctypes.c_void_p(16)), 16, None) == _lib.GLA_ERR_WORKSPACE


def test_the_wait_diagnostic_validates_before_launch():
    for polls in (0, (1 << 20) + 1):
        assert _lib.lib.gla_debug_scan_wait_timeout(polls, None) == _lib.GLA_ERR_INVALID_ARG
