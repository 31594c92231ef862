"""Sizes beyond the descriptors' 32 bits are refused instead of wrapped to small ones (host-only: meta tensors)."""
import pytest
import torch

from linear_rnn_b200 import _lib, ops

BIG = (1 << 32) + 5


@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_sizes_past_32_bits_are_refused(at):
    shape = [1, 1, 1, 1]
    shape[at] = BIG
    x = torch.empty(*shape, dtype=torch.bfloat16, device="meta")
    for make in (lambda: ops.make_scan_problem(x), lambda: ops._headnorm_problem(x, None, "silu", "rms", 1e-6)):
        with pytest.raises(ops.GlaError) as e:
            make()
        assert e.value.status == _lib.GLA_ERR_UNSUPPORTED


def test_columns_past_32_bits_are_refused():
    x = torch.empty(1, BIG, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ops.GlaError) as e:
        ops._addnorm_problem(x, torch.bfloat16, "rms", 1e-6, 1.0)
    assert e.value.status == _lib.GLA_ERR_UNSUPPORTED


def test_the_largest_sizes_arrive_whole():
    x = torch.empty(1, 1, (1 << 31) - 1, 1, dtype=torch.bfloat16, device="meta")
    assert ops.make_scan_problem(x).L == (1 << 31) - 1
    assert ops._headnorm_problem(x, None, "silu", "rms", 1e-6).L == (1 << 31) - 1
