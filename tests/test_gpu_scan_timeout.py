"""A bounded wait of gla_scan_* that gives up is reported: without a fault, by waits that nothing completes."""
import pytest
import torch

from linear_rnn_b200 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def scan():
    from linear_rnn_b200 import ops
    x, g = torch.randn(1, 2, 5000, 64, device="cuda"), -torch.rand(1, 2, 5000, 64, device="cuda")
    o, _ = ops.gla_scan_fwd(x, g)
    grads = ops.gla_scan_bwd(x, g, None, torch.ones_like(x))
    return o, grads["dx"], grads["dg"]


def test_a_wait_that_gives_up_is_reported_once():
    from linear_rnn_b200 import ops
    outs = scan()
    assert ops.gla_scan_check_device_status() == _lib.GLA_OK
    assert all(torch.isfinite(t).all() for t in outs)
    side = torch.cuda.Stream()
    assert _lib.lib.gla_debug_scan_wait_timeout(2000, side.cuda_stream) == _lib.GLA_OK
    side.synchronize()
    assert ops.gla_scan_check_device_status() == _lib.GLA_ERR_TIMEOUT      # from any stream of the device
    assert ops.gla_scan_check_device_status(torch.cuda.current_device()) == _lib.GLA_OK
    outs = scan()
    assert ops.gla_scan_check_device_status() == _lib.GLA_OK
    assert all(torch.isfinite(t).all() for t in outs)
