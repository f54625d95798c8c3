"""One speculative decoding step through the operators together, as a server
runs them: the few-token layer over a drafted block with its residual, the
head's logits, the softmax, the verification -- eager and as one CUDA graph."""
import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe
from routed_expert_ffn_renorm_b200 import workloads as W

import decode_ref as ref
from parity_util import lib_config, weights_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [1, 7])
def test_step(L):
    T, H, V = L + 1, 512, 3000  # the block and the token before it
    cfg = W.MoEConfig("step", T=T, H=H, E=16, I=192, k=2, Is=128)
    inp = W.make_inputs(cfg, device="cuda", seed=21, router=True, gate_std=0.5)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    wo = (torch.randn(H, H, generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
    head = (torch.randn(V, H, generator=g, device="cuda") * 8).to(torch.bfloat16)
    c, w = lib_config(cfg), weights_of(inp)
    ws = torch.zeros(moe.workspace_bytes(c, T), dtype=torch.uint8, device="cuda")
    ws_l = torch.zeros(max(moe.linear_workspace_bytes(T, H, H), moe.linear_workspace_bytes(T, V, H)),
                       dtype=torch.uint8, device="cuda")
    y, z = torch.empty_like(inp.x), torch.empty_like(inp.x)
    logits, probs = torch.empty(T, V, device="cuda"), torch.empty(1, T, V, device="cuda")
    draft = torch.randint(0, V, (1, L), generator=g, device="cuda").int()
    u, us = torch.rand(1, L, generator=g, device="cuda"), torch.rand(1, generator=g, device="cuda")
    tokens, n = torch.empty(1, T, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")

    def step():
        moe.moe_forward_few(c, inp.x, None, w, y, ws)
        moe.moe_linear(y, wo, z, ws_l, residual=inp.x)
        moe.moe_linear(z, head, logits, ws_l)
        torch.softmax(logits, -1, out=probs[0])
        moe.moe_verify(probs, draft, u, us, tokens, n)

    step()
    lg = inp.x.double() @ inp.w_router.double().T
    chosen, _ = ref.route(lg, 2, True, 0.0, 0)
    want, bound = ref.layer(inp.x, ref.weights64(w), chosen, inp.ws_gvec)
    assert ((y.double() - want).abs() <= bound).all()
    want, bound = ref.linear(y, wo, None, "none", inp.x, False)
    assert ((z.double() - want).abs() <= bound).all()
    want, bound = ref.linear(z, head, None, "none", None, True)
    assert ((logits.double() - want).abs() <= bound).all()
    draft[0, 0] = int(probs[0, 0].argmax())  # the first drafted token mostly stays
    step()
    want = ref.verify(probs.cpu(), None, draft.cpu(), None, u.cpu(), us.cpu())
    assert torch.equal(tokens.cpu(), want[0]) and torch.equal(n.cpu(), want[1])
    first = tokens.clone(), logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        tokens.zero_()
        logits.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, first[0]) and torch.equal(logits, first[1])
    assert moe.status_read(ws) == 0 and moe.status_read(ws_l) == 0


def test_operators_side_by_side_on_three_streams():
    """The cooperative layer, shared linear tiles and verifications at the same
    time, each stream with its own workspace: the same bits as alone."""
    cfg = W.MoEConfig("side", T=9, H=1024, E=24, I=192, k=3, Is=256)
    inp = W.make_inputs(cfg, device="cuda", seed=22, router=True, gate_std=0.5)
    c, w = lib_config(cfg), weights_of(inp)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)

    def n(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    sizes = [(7, 3000, 2048), (200, 640, 4096), (300, 5000, 256)]
    maps = [(n(T, K), n(N, K), n(T, N)) for T, N, K in sizes]
    probs = torch.softmax(2 * torch.randn(6, 5, 3001, generator=g, device="cuda"), -1)
    draft = torch.randint(0, 3001, (6, 4), generator=g, device="cuda").int()
    u, us = torch.rand(6, 4, generator=g, device="cuda"), torch.rand(6, generator=g, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = torch.zeros(moe.workspace_bytes(c, cfg.T), dtype=torch.uint8, device="cuda")
    ws_l = torch.zeros(max(moe.linear_workspace_bytes(*s) for s in sizes), dtype=torch.uint8, device="cuda")
    y, outs = torch.empty_like(inp.x), [torch.empty_like(r) for _, _, r in maps]
    tokens, count = torch.empty(6, 5, dtype=torch.int32, device="cuda"), torch.empty(6, dtype=torch.int32, device="cuda")

    def layer(stream):
        moe.moe_forward_few(c, inp.x, None, w, y, ws, stream=stream)

    def linear(stream):
        for (x, m, r), out in zip(maps, outs):
            moe.moe_linear(x, m, out, ws_l, activation="silu", residual=r, stream=stream)

    def verify(stream):
        moe.moe_verify(probs, draft, u, us, tokens, count, stream=stream)

    calls = (layer, linear, verify)
    torch.cuda.synchronize()
    for call in calls:
        call(streams[0])
    torch.cuda.synchronize()
    alone = [t.clone() for t in (y, *outs, tokens, count)]
    for t in (y, *outs, tokens, count):
        t.zero_()
    torch.cuda.synchronize()
    for i in range(40):
        for call, stream in zip(calls, streams):
            call(stream)
    torch.cuda.synchronize()
    assert moe.status_read(ws) == 0 and moe.status_read(ws_l) == 0
    for got, want in zip((y, *outs, tokens, count), alone):
        assert torch.equal(got, want)
