"""The sigmoid gate of gla_headnorm_* far from 0, where its slope p (1 - p) is small against 1.

u = 2^-24. The exponential e = e^-z is within 4 u (the hardware's 2^x) and 2 u of products, with bf16 data |z| u more
from the rounded product; p = 1 / (1 + e) within that and 3 u, q = 1 - p = e p within both and u. So the slope p q is
within 3 (6 u + |z| u) + 8 u = (26 + 3 |z|) u of itself, n within 54 u N (N = max |r| rstd, as in test_gpu_norms), and
three products add 4 u. A stored value adds half a step of its type."""
import numpy as np
import pytest
import torch

from oracle import norms
from test_gpu_norms import EPS, HALF, IO, U, f64, row_bound, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 99, 130, 1000])
def test_the_slope_of_a_wide_open_or_shut_sigmoid(D, io):
    from linear_rnn_b200 import ops
    gen = torch.Generator().manual_seed(81)
    o, dy = torch.randn(2, 3, 7, D, generator=gen).to(IO[io]), torch.randn(2, 7, 3, D, generator=gen).to(IO[io])
    z = (80 * torch.rand(2, 7, 3, D, generator=gen) - 40).to(IO[io])
    g = ops.gla_headnorm_bwd(o.cuda(), z.cuda(), None, dy.cuda(), act="sigmoid", eps=EPS)
    n = norms.norm(f64(o), "rms", EPS).transpose(0, 2, 1, 3)
    N, _ = row_bound(f64(o), "rms")
    e = np.exp(-np.abs(f64(z)))
    slope = e / (1 + e) ** 2
    ref = f64(dy) * n * slope
    tol = np.abs(f64(dy)) * slope * U * (54 * N.transpose(0, 2, 1, 3) + (30 + 3 * np.abs(f64(z))) * np.abs(n))
    within(g["dz"], ref, HALF[IO[io]] * (np.abs(ref) + tol) + tol, "dz")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gates_at_the_ends_of_their_type(io):
    """Gates of plus and minus infinity and of the type's largest numbers: the sigmoid is exactly 0 or 1, its slope 0."""
    from linear_rnn_b200 import ops
    big = torch.finfo(IO[io]).max
    z = torch.tensor([-float("inf"), -big, big, float("inf")] * 4).to(IO[io]).view(1, 1, 1, 16).cuda()
    o, dy = torch.randn(1, 1, 1, 16, device="cuda").to(IO[io]), torch.randn(1, 1, 1, 16, device="cuda").to(IO[io])
    y = ops.gla_headnorm_fwd(o, z, None, act="sigmoid", eps=EPS)
    g = ops.gla_headnorm_bwd(o, z, None, dy, act="sigmoid", eps=EPS)
    plain = ops.gla_headnorm_fwd(o, None, None, eps=EPS)
    assert torch.equal(y, torch.where(z > 0, plain, torch.zeros_like(plain)))
    assert (g["dz"] == 0).all() and torch.isfinite(g["do"]).all()
    nan = torch.full_like(z, float("nan"))
    assert torch.isnan(ops.gla_headnorm_fwd(o, nan, None, act="sigmoid", eps=EPS)).all()
    assert torch.isnan(ops.gla_headnorm_bwd(o, nan, None, dy, act="sigmoid", eps=EPS)["dz"]).all()
