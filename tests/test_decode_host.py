"""The decode operators' argument checks (few-token layer, linear map,
verification), on a host without a GPU: bad calls are refused before any CUDA
work."""
import ctypes

import pytest

import routed_expert_ffn_renorm_b200 as moe

from test_abi import FAKE, MISALIGNED, _cfg

KINDS = {"moe_forward_few": moe._Weights, "moe_forward_few_mxfp8": moe._WeightsMXFP8,
         "moe_forward_few_nvfp4": moe._WeightsNVFP4}


def _full(kind):
    return kind(*([FAKE.value] * len(kind._fields_)))


@pytest.mark.parametrize("fn", KINDS)
def test_few_refusals(fn):
    lib = moe.load_library()
    call, kind = getattr(lib, fn), KINDS[fn]
    c = _cfg(shared_intermediate_size=128)
    w = _full(kind)
    need = lib.moe_workspace_bytes(ctypes.byref(c), 16)

    def go(cfg=c, T=16, x=FAKE, logits=FAKE, weights=w, out=FAKE, aux=None, ws=FAKE, n=need):
        return call(ctypes.byref(cfg), T, x, logits, None if weights is None else ctypes.byref(weights), out,
                    None if aux is None else ctypes.byref(aux), ws, n, None)

    assert go(T=0, x=None, logits=None, weights=None, out=None, ws=None, n=0) == 0
    assert go(T=-1) == -1
    assert go(T=17) == -2
    assert go(T=1 << 20) == -2
    assert go(cfg=_cfg(hidden=200)) == -2
    for bad in (dict(x=None), dict(x=MISALIGNED), dict(logits=MISALIGNED), dict(out=None), dict(ws=MISALIGNED),
                dict(weights=None)):
        assert go(**bad) == -1, bad
    assert go(n=need - 1) == -3
    for name in ("counts", "offsets", "perm", "slot_pos"):  # nothing is dispatched
        a = moe._Aux()
        setattr(a, name, FAKE)
        assert go(aux=a) == -1, name
    a = moe._Aux()
    a.topk_w = MISALIGNED
    assert go(aux=a) == -1
    for name, _ in kind._fields_:
        bad = _full(kind)
        setattr(bad, name, None)
        # the router projection is only read without logits
        assert go(weights=bad, logits=None if name == "w_router" else FAKE) == -1, name
    if fn != "moe_forward_few":  # block-scaled weights come in 128-wide steps
        assert go(cfg=_cfg(moe_intermediate_size=192), n=1 << 40) == -2


def test_a_workspace_serves_fewer_tokens():
    lib = moe.load_library()
    for kw in (dict(), dict(shared_intermediate_size=2048, hidden=5120, n_routed_experts=256)):
        c = _cfg(**kw)
        need = [lib.moe_workspace_bytes(ctypes.byref(c), T) for T in (1, 2, 8, 9, 15, 16, 17, 31, 64, 100, 1000)]
        assert need == sorted(need)


def test_linear_sizes_at_the_limits():
    lib = moe.load_library()
    most = 2 ** 31 - 512
    assert lib.moe_linear_workspace_bytes(most, 1, 8) > 0 and lib.moe_linear_workspace_bytes(1, most, 8) > 0
    for sizes in ((most + 1, 1, 8), (1, most + 1, 8), (1, 1, most + 8), (most, 1024, 8), (1, most, 1024)):
        assert lib.moe_linear_workspace_bytes(*sizes) == 0


def test_linear_refusals():
    lib = moe.load_library()
    need = lib.moe_linear_workspace_bytes(5, 7, 16)
    assert need >= 8192
    assert lib.moe_linear_workspace_bytes(5, 7, 12) == 0
    assert lib.moe_linear_workspace_bytes(-1, 7, 16) == 0
    assert lib.moe_linear_workspace_bytes(5, 0, 16) == 0

    def go(T=5, N=7, K=16, x=FAKE, w=FAKE, bias=None, act=0, residual=None, out=FAKE, f32=0, ws=FAKE, n=need):
        return lib.moe_linear(T, N, K, x, w, bias, act, residual, out, f32, ws, n, None)

    assert go(T=0, x=None, w=None, out=None, ws=None, n=0) == 0
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(x=None), dict(w=MISALIGNED), dict(bias=MISALIGNED),
                dict(residual=MISALIGNED), dict(out=None), dict(ws=None), dict(act=4), dict(act=-1), dict(f32=2),
                dict(residual=FAKE, f32=1)):  # in place only where the types agree
        assert go(**bad) == -1, bad
    assert go(K=12) == -2
    assert go(T=1 << 30, N=1 << 20, n=1 << 60) == -2
    assert go(n=need - 1) == -3


def test_verify_refusals():
    lib = moe.load_library()

    def go(B=2, L=3, V=10, p=FAKE, q=None, draft=FAKE, length=None, u=FAKE, us=FAKE, tokens=FAKE, n=FAKE):
        return lib.moe_verify(B, L, V, p, q, draft, length, u, us, tokens, n, None)

    assert go(B=0, p=None, draft=None, u=None, us=None, tokens=None, n=None) == 0
    for bad in (dict(B=-1), dict(L=-1), dict(V=0), dict(p=None), dict(p=MISALIGNED), dict(q=MISALIGNED),
                dict(draft=None), dict(length=MISALIGNED), dict(u=None), dict(us=MISALIGNED), dict(tokens=None),
                dict(n=None)):
        assert go(**bad) == -1, bad
    assert go(B=1 << 27) == -2


def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        moe.moe_linear(x, w, torch.zeros(2, 4), torch.zeros(8192, dtype=torch.uint8))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        moe.moe_verify(torch.zeros(1, 2, 4), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1), torch.zeros(1),
                       torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
