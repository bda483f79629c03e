"""The bound that test_gpu_heads_weights.py puts on outputs holds for weights of two bf16 and not for one (no GPU)."""
import pytest
import torch

from weights_bound import bound, outputs


@pytest.mark.parametrize("positions", [8, 60, 700, 5000])
def test_one_bf16_breaks_it(positions):
    g = torch.Generator().manual_seed(positions)
    x, v = torch.randn((16, positions), generator=g, dtype=torch.float64), torch.randn((positions, 128), generator=g, dtype=torch.float64)
    w = torch.softmax(x, 1)
    tol = bound(w @ v, w @ v.abs(), 0.0, 2.0 ** -8)
    off = lambda parts: ((outputs(x, v, parts) - w @ v).abs() / tol).max().item()
    assert off(2) <= 1 and off(1) > 2
