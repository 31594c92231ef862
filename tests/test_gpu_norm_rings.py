"""gla_addnorm_* on both sides of every rule for the stages of its ring (rows enough for several turns of it), against the
oracle with test_gpu_norms' bounds."""
import pytest
import torch

from test_gpu_norms import check_addnorm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# blocks of 64, 96, 128, 160, 192 and 224 threads; pieces of 8, 4 and 2 elements and odd rows
@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("D", [514, 1021, 1028, 1535, 2046, 2048, 2305, 2576, 2602, 2901, 3004, 3500])
def test_rows_around_the_rules_of_the_ring(D, kind, io, res):
    check_addnorm(4000 if D < 1100 else 1300, D, io, res, kind, rscale=D % 3 == 0, w=True, resid=True, dr=True, seed=D)
