"""moe_verify against the definition in Python floats: equal tokens and counts."""
import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe

import decode_ref as ref

pytestmark = pytest.mark.gpu


def make(B, L, V, seed, onehot=False, ragged=False, spread=2.0):
    g = torch.Generator()
    g.manual_seed(seed)
    z = torch.randn(B, L + 1, V, generator=g) * spread
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :L] + 0.5 * torch.randn(B, L, V, generator=g), -1)
    draft = torch.multinomial(q.reshape(-1, V), 1, generator=g).reshape(B, L).int() if L else torch.zeros(
        B, 0, dtype=torch.int32)
    length = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32) if ragged else None
    return p, None if onehot else q, draft, length, torch.rand(B, L, generator=g), torch.rand(B, generator=g)


def run(p, q, draft, length, u, us):
    def c(t):
        return None if t is None else t.cuda()
    B, L1, _ = p.shape
    tokens = torch.full((B + 1, L1), 77, dtype=torch.int32, device="cuda")
    n = torch.full((B + 1,), 77, dtype=torch.int32, device="cuda")
    moe.moe_verify(c(p), c(draft), c(u), c(us), tokens[:B], n[:B], draft_probs=c(q), draft_len=c(length))
    torch.cuda.synchronize()
    assert (tokens[B] == 77).all() and int(n[B]) == 77
    return tokens[:B].cpu(), n[:B].cpu()


def check(*args):
    got, want = run(*args), ref.verify(*args)
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0], want[0])
    return got


@pytest.mark.parametrize("B,L,V", [(1, 0, 1), (1, 1, 1), (3, 0, 50), (1, 7, 5), (4, 7, 127), (5, 3, 128), (2, 33, 129),
                                   (8, 7, 1000), (3, 70, 1023), (64, 4, 4096), (2, 7, 16385), (3, 7, 32768),
                                   (2, 2, 131072), (1, 1, 200003)])
@pytest.mark.parametrize("onehot", [False, True], ids=["probs", "onehot"])
@pytest.mark.parametrize("ragged", [False, True], ids=["full", "ragged"])
def test_verify(B, L, V, onehot, ragged):
    check(*make(B, L, V, B * 1000 + L + V, onehot, ragged))


def test_flat_and_peaked_rows():
    for spread in (0.0, 0.01, 12.0, 40.0):
        check(*make(16, 5, 5000, 5, spread=spread))


def test_every_acceptance_length():
    p, q, draft, _, u, us = make(9, 8, 300, 6)
    u[:] = 0.0  # p > 0 at every drafted token: all stay
    for b in range(9):
        if b < 8:
            p[b, b, draft[b, b]] = 0.0  # u q = 0 is not below 0
    _, n = check(p, q, draft, None, u, us)
    assert n.tolist() == list(range(9))


def test_tokens_outside_the_vocabulary_end_the_block():
    p, q, draft, _, u, us = make(4, 5, 64, 7)
    u[:] = 0.0
    draft[0, 0], draft[1, 2], draft[2, 4] = -1, 64, 2 ** 31 - 1
    _, n = check(p, q, draft, None, u, us)
    assert n.tolist() == [0, 2, 4, 5]


def test_what_lies_behind_a_block_is_not_looked_at():
    p, q, draft, _, u, us = make(6, 6, 200, 8)
    length = torch.tensor([0, 1, 2, 3, 6, 4], dtype=torch.int32)
    want = check(p, q, draft, length, u, us)
    for b in range(6):
        n = int(length[b])
        draft[b, n:] = -7
        u[b, n:] = float("nan")
        q[b, n:] = float("nan")
        p[b, n + 1:] = float("nan")
    got = run(p, q, draft, length, u, us)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    length[4], length[0] = 99, -5  # clamped to the block
    got = run(p, q, draft, length, u, us)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_without_residual_mass():
    """p <= q everywhere draws from p; a row without mass gives -1."""
    p, q, draft, _, u, us = make(3, 2, 500, 9)
    q[:, 0] = p[:, 0]
    u[:, 0] = 1.0  # u q < p fails at equality
    p[1] = 0.0
    q[1] = 0.0
    tokens, n = check(p, q, draft, None, u, us)
    assert n.tolist() == [0, 0, 0] and int(tokens[1, 0]) == -1


def test_draws_at_the_ends():
    p, q, draft, _, u, us = make(6, 1, 1000, 10)
    u[:] = 0.0
    p[:, 1, :100] = 0.0
    p[:, 1, 900:] = 0.0
    us[:] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, -1.0, float("nan")])
    tokens, _ = check(p, q, draft, None, u, us)
    assert tokens[:, 1].tolist() == [100, 899, 899, 899, 100, 100]


def test_nonfinite_and_negative_entries_carry_no_mass():
    p, q, draft, _, u, us = make(8, 3, 700, 11)
    p[:, :, 5], p[:, :, 6], p[:, :, 7], p[:, :, 699] = float("nan"), float("inf"), -1.0, float("nan")
    q[:, :, 9] = float("nan")
    draft[0, 0], draft[1, 1], draft[2, 0] = 5, 9, 7  # compared with a NaN or below 0: refused
    tokens, n = check(p, q, draft, None, u, us)
    assert int(n[0]) == 0 and int(n[1]) <= 1 and int(n[2]) == 0
    assert not torch.isin(tokens, torch.tensor([6])).any()


def test_rows_of_any_alignment():
    for V in (4097, 4098, 4099, 4100):
        check(*make(3, 4, V, V))


def test_two_streams_and_graph():
    data = [make(20, 6, 3001, s) for s in (12, 13)]
    want = [run(*d) for d in data]
    dev = [[None if t is None else t.cuda() for t in d] for d in data]
    toks = [torch.empty(20, 7, dtype=torch.int32, device="cuda") for _ in data]
    ns = [torch.empty(20, dtype=torch.int32, device="cuda") for _ in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (p, q, d, _, u, us) in enumerate(dev):
            moe.moe_verify(p, d, u, us, toks[i], ns[i], draft_probs=q, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(toks[i].cpu(), want[i][0]) and torch.equal(ns[i].cpu(), want[i][1])
    p, q, d, _, u, us = [None if t is None else t.clone() for t in dev[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_verify(p, d, u, us, toks[0], ns[0], draft_probs=q)
    for i in (1, 0):
        for dst, src in zip((p, q, d, u, us), [t for t in dev[i] if t is not None]):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(toks[0].cpu(), want[i][0]) and torch.equal(ns[0].cpu(), want[i][1])


def test_binding_refusals():
    p, q, d, _, u, us = [None if t is None else t.cuda() for t in make(2, 3, 40, 14)]
    toks, n = torch.empty(2, 4, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_verify(p.bfloat16(), d, u, us, toks, n, draft_probs=q)
    with pytest.raises(ValueError):
        moe.moe_verify(p, d.long(), u, us, toks, n, draft_probs=q)
    with pytest.raises(ValueError):
        moe.moe_verify(p, d, u, us, toks[:, :3], n, draft_probs=q)
    with pytest.raises(ValueError):
        moe.moe_verify(p, d, u, us, toks, n, draft_probs=q[:, :2])
    with pytest.raises(ValueError):
        moe.moe_verify(p.transpose(0, 1).contiguous().transpose(0, 1), d, u, us, toks, n, draft_probs=q)
    moe.moe_verify(p[:0], d[:0], u[:0], us[:0], toks[:0], n[:0])  # a no-op
