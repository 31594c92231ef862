"""gla_scan_* where products of decays leave fp32's range although every state stays inside it: the
results are those of the token-by-token recurrence, whatever runs and tiles are composed.

Bounds are test_gpu_scan's: they count one rounding of every decay, product and sum, which also holds for
decays above 1. Where a state is infinite, the kind of number is compared: infinities stay infinite (no
decay is 0 unless its gate is -inf), NaN stays NaN."""
import numpy as np
import pytest
import torch

from oracle import scan
from test_gpu_scan import IO, bounds, cuda, f64, within

pytestmark = pytest.mark.gpu

# (L, D): one tile, a few tiles of a cluster, rows of tiles; by TMA, by copies of 4, 2 and 1 channel(s)
SIZES = [(100, 32), (128, 36), (256, 32), (200, 64), (700, 33), (700, 34), (2300, 64), (9000, 36)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def run(x, g, h0, dO, dhT, kind="plain"):
    from linear_rnn_b200 import ops
    xd, gd, sd, dOd, dhd = cuda(x, g, h0, dO, dhT)
    saved = torch.empty(ops.gla_scan_saved_bytes(ops.make_scan_problem(xd)), dtype=torch.uint8, device="cuda")
    o, hT = ops.gla_scan_fwd(xd, gd, sd, input=kind, saved_states=saved)
    got = {"o": o, "hT": hT, **ops.gla_scan_bwd(xd, gd, sd, dOd, dhd, input=kind, saved_states=saved)}
    ro, rT = scan.scan_fwd(f64(x), f64(g), f64(h0), kind)
    return got, {"o": ro, "hT": rT, **scan.scan_bwd(f64(x), f64(g), f64(h0), f64(dO), f64(dhT), kind)}


def check(x, g, h0, dO, dhT, io, kind="plain"):
    got, ref = run(x, g, h0, dO, dhT, kind)
    tol = bounds(f64(x), f64(g), f64(h0), f64(dO), f64(dhT), kind, io)
    for name in got:
        # subnormal numbers round by half of 2^-149 (2^-133 in bf16); a few of them make a sum
        within(got[name], ref[name], tol[name] + 2.0 ** -128, name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [0.7, 1.0, 25.0])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_growing_gates_over_zero_states(size, gate, io):
    """Every state and every gradient is 0, while a tile's decays (g = 1: e^128) or a run's (25: e^100) are not fp32
    numbers. The last 20 tokens forget and start anew with data."""
    L, D = size
    gen = torch.Generator().manual_seed(1)
    x, dO = torch.zeros(2, 1, L, D), torch.zeros(2, 1, L, D)
    g = torch.full((2, 1, L, D), gate)
    x[:, :, -20:] = torch.randn(2, 1, 20, D, generator=gen)
    dO[:, :, -20:] = torch.randn(2, 1, 20, D, generator=gen)
    g[:, :, -20:] = -0.1
    g[:, :, -20] = float("-inf")
    x, dO = x.to(IO[io]), dO.to(IO[io])
    check(x, g, None, dO, None, IO[io])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_growing_gates_under_zero_gradients(size, io):
    """The other way round: data and gradients at the first 20 tokens only, a start behind them, then growth."""
    L, D = size
    gen = torch.Generator().manual_seed(2)
    x, dO = torch.zeros(1, 2, L, D), torch.zeros(1, 2, L, D)
    g = torch.full((1, 2, L, D), 1.0)
    x[:, :, :20] = torch.randn(1, 2, 20, D, generator=gen)
    dO[:, :, :20] = torch.randn(1, 2, 20, D, generator=gen)
    g[:, :, :20] = -0.1
    g[:, :, 20] = float("-inf")
    h0 = torch.randn(1, 2, D, generator=gen)
    x, dO = x.to(IO[io]), dO.to(IO[io])
    check(x, g, h0, dO, None, IO[io])


@pytest.mark.parametrize("size", [(170, 32), (200, 33), (200, 64), (240, 34)], ids=str)
def test_small_states_grow_past_the_range_of_one_tile(size):
    """States from 1e-33: a tile's decays (g = 0.7: e^89.6) pass fp32's range, the states do not."""
    L, D = size
    gen = torch.Generator().manual_seed(3)
    x = 1e-33 * torch.randn(2, 2, L, D, generator=gen)
    h0 = 1e-33 * torch.randn(2, 2, D, generator=gen)
    dO = 1e-33 * torch.randn(2, 2, L, D, generator=gen)
    g = torch.full((2, 2, L, D), 0.7)
    g[:, :, 190:] = -0.5
    check(x, g, h0, dO, 1e-33 * torch.randn(2, 2, D, generator=gen), torch.float32)


def test_growth_then_a_start_within_a_tile():
    """A tile's decays pass fp32's range before a start makes their product 0; the states before are small."""
    gen = torch.Generator().manual_seed(4)
    for L, D in ((384, 32), (500, 33)):
        x, dO = 1e-30 * torch.randn(1, 2, L, D, generator=gen), torch.randn(1, 2, L, D, generator=gen)
        g = torch.full((1, 2, L, D), -0.2)
        g[:, :, 130:245] = 0.9         # e^103
        dO[:, :, 100:246] = 0
        g[:, :, 246] = float("-inf")
        x[:, :, 246:] *= 1e30
        check(x, g, None, dO, None, torch.float32)


@pytest.mark.parametrize("gate", [-1.0, -30.0])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_an_infinite_state_stays_infinite(size, gate):
    """Products of e^-1 over a tile, or of e^-30 over four tokens, are 0 in fp32; the state is not multiplied by
    0 at any token, except at a start, where 0 times infinity is NaN."""
    L, D = size
    gen = torch.Generator().manual_seed(5)
    x, dO = torch.randn(1, 2, L, D, generator=gen), torch.randn(1, 2, L, D, generator=gen)
    g = torch.full((1, 2, L, D), gate)
    x[0, 0, 5, 3], x[0, 1, 7, 4], x[0, 0, L // 2, 9] = float("inf"), float("-inf"), float("inf")
    dO[0, 0, L - 3, 10], dO[0, 1, L // 3, 11] = float("-inf"), float("inf")
    g[0, 0, L - 30, 9] = float("-inf")
    with np.errstate(invalid="ignore", over="ignore"):
        got, ref = run(x, g, None, dO, None)
    for name in ("o", "hT", "dx", "dh0"):
        r, v = ref[name], f64(got[name])
        assert np.array_equal(np.isnan(v), np.isnan(r)), name
        assert np.array_equal(v[np.isinf(r)], r[np.isinf(r)]) and np.isfinite(v[np.isfinite(r)]).all(), name
