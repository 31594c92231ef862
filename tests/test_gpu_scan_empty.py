"""The training pair of gla_scan_* on empty problems, with a saved-states buffer of the size asked for (none)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("size", [(2, 3, 0, 8), (0, 3, 4, 8), (2, 0, 4, 8), (0, 0, 0, 1)], ids=str)
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16], ids=str)
def test_training_pair_of_nothing(size, io):
    from linear_rnn_b200 import ops
    B, H, L, D = size
    x, dO, g = (torch.empty(*size, dtype=t, device="cuda") for t in (io, io, torch.float32))
    h0, dhT = torch.randn(B, H, D, device="cuda"), torch.randn(B, H, D, device="cuda")
    saved = torch.empty(ops.gla_scan_saved_bytes(ops.make_scan_problem(x)), dtype=torch.uint8, device="cuda")
    assert saved.numel() == 0
    o, hT = ops.gla_scan_fwd(x, g, h0, saved_states=saved)
    grads = ops.gla_scan_bwd(x, g, h0, dO, dhT, saved_states=saved)
    assert torch.equal(hT, h0) and torch.equal(grads["dh0"], dhT)
    assert o.shape == grads["dx"].shape == grads["dg"].shape == x.shape
    assert (ops.gla_scan_bwd(x, g, None, dO, None, saved_states=saved)["dh0"] == 0).all()
