"""The few-token layer (moe_forward_few and its MXFP8 / NVFP4 forms) against
the 64-bit reference, within the elementwise bound of its roundings."""
import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe
from routed_expert_ffn_renorm_b200 import workloads as W

import decode_ref as ref
from parity_util import lib_config, weights_of

pytestmark = pytest.mark.gpu

FORMS = {"bf16": (None, moe.moe_forward_few), "mxfp8": (moe.pack_mxfp8, moe.moe_forward_few_mxfp8),
         "nvfp4": (moe.pack_nvfp4, moe.moe_forward_few_nvfp4)}


def workspace(c, T):
    ws = torch.full((moe.workspace_bytes(c, T),), 0xAB, dtype=torch.uint8, device="cuda")  # scratch holds anything
    moe.status_clear(ws)
    return ws


def run(cfg, inp, fmt="bf16", logits="given", ws=None, aux=None):
    pack, call = FORMS[fmt]
    w = weights_of(inp)
    w = pack(w) if pack else w
    c = lib_config(cfg)
    ws = workspace(c, cfg.T) if ws is None else ws
    out = torch.full((cfg.T + 1, cfg.H), 7.0, dtype=torch.bfloat16, device="cuda")  # one row behind the last
    call(c, inp.x, None if logits is None else inp.logits, w, out[:cfg.T], ws, aux=aux)
    assert moe.status_read(ws) == 0
    assert (out[cfg.T] == 7.0).all()
    return out[:cfg.T], w


def check(cfg, inp, fmt="bf16", logits="given", ws=None):
    T, k, E = cfg.T, cfg.k, cfg.E
    dev = "cuda"
    aux = {"topk_idx": torch.empty(T, k, dtype=torch.int32, device=dev),
           "topk_w": torch.empty(T, k, dtype=torch.float32, device=dev),
           "keff": torch.empty(T, dtype=torch.int32, device=dev),
           "logits": torch.empty(T, E, dtype=torch.float32, device=dev),
           "expert_kept": torch.zeros(E, dtype=torch.uint8, device=dev),
           "n_dropped": torch.zeros(1, dtype=torch.int32, device=dev)}
    if cfg.Is:
        aux["sgate"] = torch.empty(T, dtype=torch.float32, device=dev)
    if logits is None:
        out, w = run(cfg, inp, fmt, None, ws, aux)
        lg = aux["logits"]
        want = inp.x.double() @ inp.w_router.double().T
        bound = cfg.H * ref.F32 * (inp.x.double().abs() @ inp.w_router.double().abs().T) + 1e-30
        assert ((lg.double() - want).abs() <= bound).all()
    else:
        del aux["logits"]
        out, w = run(cfg, inp, fmt, logits, ws, aux)
        lg = inp.logits
    chosen, drop = ref.route(lg, k, cfg.norm_topk, cfg.topp, cfg.budget)
    idx, tw, keff = aux["topk_idx"].cpu(), aux["topk_w"].cpu(), aux["keff"].cpu()
    for t, kept in enumerate(chosen):
        n = len(kept)
        assert int(keff[t]) == n
        assert idx[t].tolist() == [e for e, _ in kept] + [-1] * (k - n)
        torch.testing.assert_close(tw[t, :n].double(), torch.tensor([v for _, v in kept], dtype=torch.float64),
                                   rtol=4e-6, atol=0)
    if cfg.budget:
        assert int(aux["n_dropped"]) == drop
        used = {e for kept in chosen for e, _ in kept}
        if drop:
            assert {e for e in range(E) if aux["expert_kept"][e]} >= used
            assert int(aux["expert_kept"].sum()) == cfg.budget
    gv = inp.ws_gvec if cfg.Is else None
    want, bound = ref.layer(inp.x, ref.weights64(w), chosen, gv)
    diff = (out.double() - want).abs()
    assert (diff <= bound).all(), float((diff / bound).max())
    return out


def cfg_(**kw):
    base = dict(name="few", T=7, H=256, E=8, I=128, k=2)
    base.update(kw)
    return W.MoEConfig(**base)


SHAPES = [
    dict(T=1), dict(T=2, E=1, k=1), dict(T=7, I=64, H=128), dict(T=8, Is=64), dict(T=9, Is=192, I=192, H=384),
    dict(T=16, E=40, k=6, Is=128), dict(T=16, E=130, k=5, I=64), dict(T=3, E=257, k=8, I=64, norm_topk=False),
    dict(T=16, E=1024, k=32, I=64, H=128), dict(T=5, H=1152, I=320, E=16, k=4, Is=448),
    dict(T=13, E=512, k=10, I=64, Is=128, zipf_alpha=1.0), dict(T=1, H=5120, E=4, I=1024, k=2, Is=2048),
    dict(T=16, E=64, k=64 // 2, I=64, topp=0.5), dict(T=11, E=33, k=4, topp=0.9, norm_topk=False),
    dict(T=16, E=128, k=8, I=64, budget=4, zipf_alpha=1.2), dict(T=16, E=300, k=8, I=64, budget=1),
    dict(T=9, E=24, k=6, budget=5, topp=0.6, Is=64), dict(T=6, E=24, k=3, budget=7, norm_topk=False),
]


@pytest.mark.parametrize("kw", SHAPES, ids=lambda kw: "_".join(f"{a}{b}" for a, b in kw.items()))
@pytest.mark.parametrize("logits", ["given", None], ids=["given", "projected"])
def test_layer(kw, logits):
    cfg = cfg_(**kw)
    inp = W.make_inputs(cfg, device="cuda", seed=3, router=True, gate_std=0.5)
    check(cfg, inp, "bf16", logits)


@pytest.mark.parametrize("kw", [
    dict(T=1), dict(T=16, E=5, k=5, Is=128), dict(T=7, H=384, I=256, E=40, k=3, Is=384),
    dict(T=9, H=1152, I=128, E=130, k=8, budget=6), dict(T=2, H=5120, I=512, E=6, k=2, Is=1024),
], ids=lambda kw: "_".join(f"{a}{b}" for a, b in kw.items()))
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_block_scaled(kw, fmt):
    cfg = cfg_(**kw)
    inp = W.make_inputs(cfg, device="cuda", seed=4, router=True, gate_std=0.5)
    check(cfg, inp, fmt, None)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_block_scaled_odd_blocks(fmt):
    """Blocks of zeros, of one value and of tiny and large values, negative zeros."""
    cfg = cfg_(T=5, H=256, I=128, E=3, k=2, Is=128)
    inp = W.make_inputs(cfg, device="cuda", seed=5, gate_std=0.5)
    for w in (inp.w_gate, inp.w_up, inp.w_down, inp.ws_gate, inp.ws_up, inp.ws_down):
        w = w.view(-1, w.shape[-1])
        w[0] = 0.0
        w[1, :32] = -0.0
        w[2] *= 2.0 ** -40
        w[3, 5] = 1.5
        w[4, ::3] = 0.0
        w[5, 32:64] *= 2.0 ** 18
    check(cfg, inp, fmt)


@pytest.mark.parametrize("kw", [dict(T=16, E=520, k=12, H=2048, I=64), dict(T=1, E=9, k=2, H=5120, I=64, Is=64),
                                dict(T=16, E=600, k=8, H=3584, I=64, Is=128), dict(T=5, E=1024, k=32, H=1024, I=64, Is=64),
                                dict(T=16, E=256, k=8, H=1152, I=64, Is=1024, budget=9, topp=0.8)],
                         ids=lambda kw: "_".join(f"{a}{b}" for a, b in kw.items()))
def test_projection_split_along_k(kw):
    """The router's product cut along H over the CTAs, its routing with and without a shared expert."""
    cfg = cfg_(**kw)
    check(cfg, W.make_inputs(cfg, device="cuda", seed=15, router=True, gate_std=0.5), "bf16", None)


def test_logits_of_all_ones_bits():
    """Every logit the NaN of all ones: the experts are distinct and in range, other tokens unharmed."""
    for Is in (0, 64):
        cfg = cfg_(T=3, E=40, k=5, I=64, Is=Is)
        inp = W.make_inputs(cfg, device="cuda", seed=16, gate_std=0.5)
        good = run(cfg, inp)[0].clone()
        inp.logits[1].view(torch.int32).fill_(-1)
        idx = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device="cuda")
        out, _ = run(cfg, inp, aux={"topk_idx": idx})
        assert torch.equal(out[[0, 2]], good[[0, 2]])
        assert idx[1].tolist() == list(range(cfg.k))


def test_equal_logits_keep_the_lower_expert():
    cfg = cfg_(T=4, E=70, k=5, I=64)
    inp = W.make_inputs(cfg, device="cuda", seed=6)
    inp.logits[0] = 0.0
    inp.logits[1, 10:40] = 9.0
    inp.logits[2, ::2] = -0.0
    inp.logits[2, 1::2] = 0.0
    inp.logits[3] = -3.0e38
    check(cfg, inp)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_nonfinite_token_stays_its_own(value):
    """A token with an infinity or NaN spoils no other token, routed with it or not."""
    cfg = cfg_(T=12, E=6, k=2, Is=64)
    inp = W.make_inputs(cfg, device="cuda", seed=7, gate_std=0.5)
    good = check(cfg, inp)
    good = good.clone()
    inp.x[5, 17] = value
    out, _ = run(cfg, inp)
    rows = [t for t in range(cfg.T) if t != 5]
    assert torch.equal(out[rows], good[rows])
    assert not torch.isfinite(out[5]).all()


def test_dropped_everywhere_gives_the_shared_expert_alone():
    """A token that loses all its experts to the budget keeps the shared expert, or zero."""
    for Is in (0, 64):
        cfg = cfg_(T=3, E=6, k=1, Is=Is, budget=1)
        inp = W.make_inputs(cfg, device="cuda", seed=8, gate_std=0.5)
        inp.logits[:] = 0.0
        inp.logits[0, 2] = inp.logits[1, 2] = 5.0
        inp.logits[2, 4] = 1.0
        out = check(cfg, inp)
        if not Is:
            assert (out[2] == 0).all()


def test_same_bits_every_run_and_after_moe_forward():
    """One workspace serves both forms of the layer in turn; results do not depend on what ran before."""
    cfg = cfg_(T=16, E=32, k=4, Is=192, I=192)
    inp = W.make_inputs(cfg, device="cuda", seed=9, router=True, gate_std=0.5)
    c = lib_config(cfg)
    ws = workspace(c, cfg.T)
    first = check(cfg, inp, ws=ws).clone()
    big = torch.empty_like(first)
    moe.moe_forward(c, inp.x, inp.logits, weights_of(inp), big, ws)
    for logits in ("given", None, "given"):
        out, _ = run(cfg, inp, "bf16", logits, ws)
    assert torch.equal(out, first)
    again = torch.empty_like(first)
    moe.moe_forward(c, inp.x, inp.logits, weights_of(inp), again, ws)
    assert torch.equal(again, big)
    assert float((big.float() - first.float()).norm() / big.float().norm()) < 5e-3
    small = W.MoEConfig(**{**cfg.__dict__, "T": 3})  # fewer tokens in the larger workspace
    sub = W.MoEInputs(inp.x[:3], inp.logits[:3], *[getattr(inp, n) for n in (
        "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down", "ws_gvec", "w_router")])
    out3, _ = run(small, sub, ws=ws)
    check(small, sub, ws=ws)
    out, _ = run(cfg, inp, ws=ws)
    assert torch.equal(out, first)


def test_two_streams_at_once():
    cfg = cfg_(T=16, H=1024, E=16, I=256, k=4, Is=256)
    inp = [W.make_inputs(cfg, device="cuda", seed=s, router=True, gate_std=0.5) for s in (10, 11)]
    c = lib_config(cfg)
    want = [run(cfg, i, "bf16", None)[0].clone() for i in inp]
    ws = [workspace(c, cfg.T) for _ in inp]
    out = [torch.empty_like(o) for o in want]
    streams = [torch.cuda.Stream() for _ in inp]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            moe.moe_forward_few(c, inp[i].x, None, weights_of(inp[i]), out[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert moe.status_read(ws[i]) == 0
        assert torch.equal(out[i], want[i])


def test_captured_and_replayed_on_new_inputs():
    cfg = cfg_(T=7, H=512, E=16, I=192, k=3, Is=64)
    a, b = (W.make_inputs(cfg, device="cuda", seed=s, router=True, gate_std=0.5) for s in (12, 13))
    b = W.MoEInputs(b.x, b.logits, *[getattr(a, n) for n in (
        "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down", "ws_gvec", "w_router")])
    c = lib_config(cfg)
    want = [run(cfg, i, "bf16", None)[0].clone() for i in (a, b)]
    ws, x = workspace(c, cfg.T), a.x.clone()
    out = torch.empty_like(want[0])
    w = weights_of(a)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        moe.moe_forward_few(c, x, None, w, out, ws)
    for i, inp in ((1, b), (0, a), (1, b)):
        x.copy_(inp.x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    assert moe.status_read(ws) == 0


def test_binding_refusals():
    cfg = cfg_(T=4, Is=64)
    inp = W.make_inputs(cfg, device="cuda", seed=14)
    c, w = lib_config(cfg), weights_of(inp)
    ws = workspace(c, 16)
    out = torch.empty_like(inp.x)
    with pytest.raises(ValueError):
        moe.moe_forward_few(c, inp.x, inp.logits[:3], w, out, ws)
    with pytest.raises(ValueError):
        moe.moe_forward_few(c, inp.x, inp.logits, w, out.float(), ws)
    with pytest.raises(ValueError):
        moe.moe_forward_few(c, inp.x, None, w, out, ws)  # no router projection either
    with pytest.raises(ValueError):
        moe.moe_forward_few(c, inp.x[:, ::2], inp.logits, w, out, ws)
    for name in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down", "ws_gate_vec"):
        bad = weights_of(inp)
        setattr(bad, name, getattr(bad, name)[:-1])
        with pytest.raises(ValueError):
            moe.moe_forward_few(c, inp.x, inp.logits, bad, out, ws)
    with pytest.raises(moe.MoEError) as e:
        big = torch.zeros(17, cfg.H, dtype=torch.bfloat16, device="cuda")
        moe.moe_forward_few(c, big, torch.zeros(17, cfg.E, device="cuda"), w, big.clone(),
                            torch.zeros(moe.workspace_bytes(c, 17), dtype=torch.uint8, device="cuda"))
    assert e.value.code == -2
    with pytest.raises(moe.MoEError) as e:
        moe.moe_forward_few(c, inp.x, inp.logits, w, out, ws[:1024])
    assert e.value.code == -3
    empty = inp.x[:0]
    moe.moe_forward_few(c, empty, inp.logits[:0], w, out[:0], ws)  # a no-op
