"""A misaligned pointer to a single value is refused like any other, before any launch (host without a GPU)."""
import ctypes

import pytest

import routed_expert_ffn_renorm_b200 as moe

from test_abi import FAKE, _cfg

ODD = ctypes.c_void_p((1 << 20) + 2)  # never dereferenced


def test_budget_count():
    lib = moe.load_library()
    c = _cfg(budget=2)
    n = lib.moe_workspace_bytes(ctypes.byref(c), 4)
    assert lib.moe_budget(ctypes.byref(c), 4, FAKE, FAKE, FAKE, FAKE, ODD, FAKE, n, None) == -1


@pytest.mark.parametrize("fn,kind", [("moe_forward", moe._Weights), ("moe_forward_nvfp4", moe._WeightsNVFP4),
                                     ("moe_forward_few", moe._Weights),
                                     ("moe_forward_few_mxfp8", moe._WeightsMXFP8)])
def test_layer_outputs(fn, kind):
    lib = moe.load_library()
    c = _cfg(budget=2, shared_intermediate_size=128)
    n = lib.moe_workspace_bytes(ctypes.byref(c), 4)
    w, aux = kind(*([FAKE.value] * len(kind._fields_))), moe._Aux()
    aux.n_dropped = ODD
    assert getattr(lib, fn)(ctypes.byref(c), 4, FAKE, FAKE, ctypes.byref(w), FAKE, ctypes.byref(aux), FAKE, n,
                            None) == -1
