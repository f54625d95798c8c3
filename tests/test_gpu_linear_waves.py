"""moe_linear with more tiles than the grid has CTAs or pairs: several tiles per
worker, whole waves followed by K shares, in both output types -- single CTAs
(up to 64 tokens) and pairs (fp32 results sum their segments anew per tile)."""
import pytest
import torch

from test_gpu_linear import check

pytestmark = pytest.mark.gpu

# 148 SMs: tiles of 128 channels over 148 CTAs up to 64 tokens, of 256 channels over 74 pairs above
SINGLE = [(7, 19200, 1040), (1, 38016, 72), (16, 40001, 520), (64, 38000, 200), (9, 19072, 8200), (33, 57000, 1032), (60, 20000, 8200)]
PAIRS = [(300, 9480, 2048), (70, 20008, 1544), (200, 19001, 520), (400, 9480, 136), (1000, 5128, 1032),
         (193, 38000, 72), (577, 6400, 4104), (300, 10000, 8200)]


@pytest.mark.parametrize("T,N,K", SINGLE + PAIRS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("silu", True, True)], ids=["plain", "all"])
def test_waves(T, N, K, dtype, act, bias, residual):
    out = check(T, N, K, act, bias, residual, dtype, seed=41).clone()
    assert torch.equal(check(T, N, K, act, bias, residual, dtype, seed=41), out)
