"""gla_scan_decode on a token in host memory: the caller may write the token's buffers again once the call
returned, as a loop that fills one pinned buffer per step does."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("pinned", [False, True])
def test_host_token_may_be_overwritten_after_the_call(pinned):
    from linear_rnn_b200 import ops
    gen = torch.Generator().manual_seed(1)
    B, H, D = 64, 16, 256
    x, g = torch.randn(B, H, 1, D, generator=gen), -torch.rand(B, H, 1, D, generator=gen)
    state = torch.randn(B, H, D, generator=gen)
    want_state = state.cuda()
    want = ops.gla_scan_decode(x.cuda(), g.cuda(), want_state)
    xs, gs = (x.pin_memory(), g.pin_memory()) if pinned else (x.clone(), g.clone())
    got_state = state.cuda()
    work = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    for _ in range(8):          # the stream is busy for some milliseconds
        work = work @ work * 1e-3
    got = ops.gla_scan_decode(xs, gs, got_state)
    xs.fill_(float("nan"))
    gs.fill_(float("nan"))
    assert torch.equal(got, want) and torch.equal(got_state, want_state)
