"""The few-token calls refuse weights, outputs and workspaces that the kernel
would read or write out of range: other types, sizes or devices.  The checks are
run on host tensors (device index -1), the calls themselves on a GPU."""
import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe

E, I, H, Is = 4, 128, 256, 128
CFG = moe.MoEConfig(H, E, I, 2, Is)
CALLS = ("moe_forward_few", "moe_forward_few_mxfp8", "moe_forward_few_nvfp4")


def weights(fn, device="cpu"):
    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)

    def bf(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=device)

    def f32(*shape):
        return torch.zeros(shape, device=device)
    shapes = dict(w_gate=(E, I, H), w_up=(E, I, H), w_down=(E, H, I), ws_gate=(Is, H), ws_up=(Is, H), ws_down=(H, Is))
    common = dict(ws_gate_vec=bf(H), w_router=bf(E, H))
    if fn == "moe_forward_few":
        return moe.MoEWeights(**{n: bf(*s) for n, s in shapes.items()}, **common)
    per, step = (1, 32) if fn.endswith("mxfp8") else (2, 16)
    f = {n: u8(*s[:-1], s[-1] // per) for n, s in shapes.items()}
    f.update({n + "_scale": u8(*s[:-1], s[-1] // step) for n, s in shapes.items()})
    if per == 1:
        return moe.MoEWeightsMXFP8(**f, **common)
    return moe.MoEWeightsNVFP4(**f, **common, w_gate_tscale=f32(E), w_up_tscale=f32(E), w_down_tscale=f32(E),
                               ws_tscale=f32(3))


def check(fn, w, cfg=CFG, device=-1, router=True):
    moe._check_few_weights(fn, cfg, w, device, router)


@pytest.mark.parametrize("fn", CALLS)
def test_every_field_is_checked(fn):
    check(fn, weights(fn))
    for name, t in vars(weights(fn)).items():
        other = torch.float32 if t.dtype != torch.float32 else torch.bfloat16
        for bad in (None, t.to(other), t[:-1]):
            w = weights(fn)
            setattr(w, name, bad)
            with pytest.raises(ValueError, match=name):
                check(fn, w)
    with pytest.raises(ValueError, match="w_gate"):
        check(fn, weights(fn), device=0)
    check(fn, weights(fn), cfg=moe.MoEConfig(H, E, I, 2))  # without a shared expert its weights are not looked at
    w = weights(fn)
    w.w_router = None
    check(fn, w, router=False)


def test_the_formats_are_not_taken_for_one_another():
    for fn in CALLS:
        for other in CALLS:
            if fn != other:
                with pytest.raises(ValueError):
                    check(fn, weights(other))


def test_packed_scales_of_the_quantisers_shape_or_flat():
    for fn in CALLS[1:]:
        w = weights(fn)
        w.w_gate_scale, w.ws_down_scale = w.w_gate_scale.flatten(), w.ws_down_scale.flatten()
        check(fn, w)


def test_outputs():
    T, k = 5, 2
    for name, t in (("topk_idx", torch.zeros(T, k)), ("topk_idx", torch.zeros(T * k - 1, dtype=torch.int32)),
                    ("topk_w", torch.zeros(T, k, dtype=torch.bfloat16)), ("sgate", torch.zeros(T - 1)),
                    ("keff", torch.zeros(T, dtype=torch.int64)), ("expert_kept", torch.zeros(E - 1, dtype=torch.uint8)),
                    ("n_dropped", torch.zeros(0, dtype=torch.int32)), ("logits", torch.zeros(T, E - 1))):
        with pytest.raises(ValueError, match=f"aux {name}"):
            moe._few_aux(CFG, T, {name: t}, -1)
    with pytest.raises(ValueError, match="no output"):
        moe._few_aux(CFG, T, {"topk_ids": torch.zeros(T, k, dtype=torch.int32)}, -1)


def test_host_tensors_are_a_value_error():
    """Also where there is no GPU to name as the current device."""
    x, ws = torch.zeros(2, H, dtype=torch.bfloat16), torch.zeros(8192, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x is on cpu"):
        moe.moe_forward_few(CFG, x, None, weights("moe_forward_few"), x.clone(), ws)
    with pytest.raises(ValueError, match="x is on cpu"):
        moe.moe_linear(x, x.clone(), torch.zeros(2, 2), ws)
    i = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="target_probs is on cpu"):
        moe.moe_verify(torch.zeros(1, 2, 4), i[:, :1], torch.zeros(1, 1), torch.zeros(1), i, i[0, :1])


@pytest.mark.gpu
@pytest.mark.parametrize("fn", CALLS)
def test_calls(fn):
    T = 3
    w = weights(fn, "cuda")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 5.0)
    ws = torch.zeros(moe.workspace_bytes(CFG, T), dtype=torch.uint8, device="cuda")
    call = getattr(moe, fn)
    for other in CALLS:
        if other != fn:
            with pytest.raises(ValueError):
                call(CFG, x, None, weights(other, "cuda"), out, ws)
    with pytest.raises(ValueError):
        call(CFG, x, None, w, out, ws.cpu())
    with pytest.raises(ValueError):
        call(CFG, x, None, w, out, ws, aux={"keff": torch.zeros(T - 1, dtype=torch.int32, device="cuda")})
    assert (out == 5.0).all()
    keff = torch.full((T + 1,), 9, dtype=torch.int32, device="cuda")  # a larger buffer is taken
    call(CFG, x, None, w, out, ws, aux={"keff": keff})
    assert moe.status_read(ws) == 0
    assert (out == 0).all() and keff.tolist() == [2] * T + [9]


@pytest.mark.gpu
def test_linear_workspace_on_its_device():
    x, w = torch.zeros(2, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 16, dtype=torch.bfloat16,
                                                                                device="cuda")
    with pytest.raises(ValueError, match="ws"):
        moe.moe_linear(x, w, torch.zeros(2, 4, device="cuda"), torch.zeros(moe.linear_workspace_bytes(2, 4, 16),
                                                                           dtype=torch.uint8))
