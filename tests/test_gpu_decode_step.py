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
