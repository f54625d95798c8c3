"""Workspace sizes at the ends of their ranges, on a host without a GPU."""
import ctypes

import pytest

import routed_expert_ffn_renorm_b200 as moe

from test_abi import _cfg


@pytest.mark.parametrize("kw", [dict(), dict(hidden=5120, n_routed_experts=512, num_experts_per_tok=10),
                                dict(shared_intermediate_size=128, n_routed_experts=1, num_experts_per_tok=1)])
def test_empty_batch_has_a_workspace(kw):
    """T = 0 is a valid batch: its workspace holds the head and no more than one token's."""
    lib = moe.load_library()
    c = _cfg(**kw)
    empty, one = (lib.moe_workspace_bytes(ctypes.byref(c), T) for T in (0, 1))
    assert 8192 <= empty <= one


@pytest.mark.parametrize("N,K", [(1, 8), (4096, 4096), (131072, 5120), (300, 65536)])
def test_a_linear_workspace_serves_fewer_tokens(N, K):
    lib = moe.load_library()
    sizes = [lib.moe_linear_workspace_bytes(T, N, K) for T in range(0, 2100)]
    assert sizes == sorted(sizes) and sizes[0] == 8192
    assert sizes[-1] <= lib.moe_linear_workspace_bytes(100000, N, K) < 43 << 20
