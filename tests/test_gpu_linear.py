"""moe_linear against the 64-bit product, within the bound of its sums and roundings."""
import pytest
import torch

import routed_expert_ffn_renorm_b200 as moe

import decode_ref as ref

pytestmark = pytest.mark.gpu


def workspace(T, N, K):
    ws = torch.full((moe.linear_workspace_bytes(T, N, K),), 0xAB, dtype=torch.uint8, device="cuda")
    moe.status_clear(ws)
    return ws


def make(T, N, K, bias, residual, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    return (n(T, K), (n(N, K).float() / K ** 0.5).to(torch.bfloat16), n(N) if bias else None,
            n(T, N) if residual else None)


def check(T, N, K, act="none", bias=False, residual=False, dtype=torch.bfloat16, seed=0, ws=None):
    x, w, b, r = make(T, N, K, bias, residual, seed)
    ws = workspace(T, N, K) if ws is None else ws
    buf = torch.full((T * N + 64,), 7.0, dtype=dtype, device="cuda")  # 64 values behind the last
    out = buf[:T * N].view(T, N)
    moe.moe_linear(x, w, out, ws, bias=b, activation=act, residual=r)
    assert moe.status_read(ws) == 0
    assert (buf[T * N:] == 7.0).all()
    want, bound = ref.linear(x, w, b, act, r, dtype == torch.float32)
    diff = (out.double() - want).abs()
    assert (diff <= bound).all(), float((diff / bound).max())
    return out


SIZES = [(1, 1, 8), (1, 7, 8), (1, 128, 64), (2, 129, 72), (7, 1000, 520), (8, 64, 5120), (9, 257, 136),
         (16, 4096, 1024), (16, 130, 8200), (17, 128, 64), (17, 333, 200), (31, 1, 64), (33, 640, 2048), (64, 127, 72),
         (100, 1001, 1032), (128, 256, 64), (129, 511, 4096), (224, 5120, 640), (255, 384, 1160), (256, 256, 256),
         (257, 2049, 64), (1000, 777, 328), (1023, 1280, 512), (2500, 130, 72), (4097, 513, 136)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("act,bias,residual,dtype", [
    ("none", False, False, torch.float32), ("none", True, True, torch.bfloat16),
    ("silu", True, False, torch.float32), ("gelu", False, True, torch.bfloat16),
    ("relu", True, True, torch.float32)], ids=["plain", "bias_res", "silu", "gelu_res", "relu_all"])
def test_linear(T, N, K, act, bias, residual, dtype):
    check(T, N, K, act, bias, residual, dtype)


@pytest.mark.parametrize("T,N,K", [(1, 300, 8192), (16, 256, 4096), (70, 384, 5128), (200, 128, 8192)])
def test_fp32_out_keeps_the_sums(T, N, K):
    """fp32 results leave the tensor cores every 512 columns: 32 additions to an
    accumulator, each losing less than 2^-23 of the magnitudes added so far for
    the sum and as much for aligning its products, then the segments' fp32 sum."""
    x, w, _, _ = make(T, N, K, False, False, 8)
    out = torch.empty(T, N, device="cuda")
    moe.moe_linear(x, w, out, workspace(T, N, K))
    want, mag = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    assert ((out.double() - want).abs() <= (2 * 32 + (K + 511) // 512 + 16) * ref.F32 * mag).all()
    # half an ulp lost on average in each addition
    assert float((out.double() - want).norm() / want.norm()) < 32 * 2.0 ** -24


@pytest.mark.parametrize("T,N,K", [(280, 9608, 72), (300, 9480, 2048), (5000, 1032, 72), (70, 20008, 40),
                                   (2049, 4104, 264), (4100, 1288, 2056)])
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("silu", True, True), ("none", False, True)],
                         ids=["plain", "all", "res"])
def test_many_tiles(T, N, K, act, bias, residual):
    """Whole waves of tiles: ragged last tokens and channels, K at the border of the staged epilogue."""
    out = check(T, N, K, act, bias, residual, seed=9)
    if residual:  # in place
        x, w, b, r = make(T, N, K, bias, residual, 9)
        moe.moe_linear(x, w, r, workspace(T, N, K), bias=b, activation=act, residual=r)
        assert torch.equal(r, out)


def test_large_values_and_activation_tails():
    for act in ("gelu", "silu", "relu"):
        x, w, b, _ = make(20, 96, 64, True, False, 3)
        x, b = x * 30, b * 20
        for T in (4, 20):
            out = torch.empty(T, 96, device="cuda")
            moe.moe_linear(x[:T].contiguous(), w, out, workspace(T, 96, 64), bias=b, activation=act)
            want, bound = ref.linear(x[:T], w, b, act, None, True)
            assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("T", [5, 40, 300])
def test_residual_in_place(T):
    x, w, b, r = make(T, 200, 136, True, True, 4)
    ws = workspace(T, 200, 136)
    out = torch.empty_like(r)
    moe.moe_linear(x, w, out, ws, bias=b, activation="silu", residual=r)
    moe.moe_linear(x, w, r, ws, bias=b, activation="silu", residual=r)
    assert torch.equal(r, out)


@pytest.mark.parametrize("T", [6, 60])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_nonfinite_row_stays_its_own(T, value):
    x, w, _, _ = make(T, 300, 200, False, False, 5)
    ws = workspace(T, 300, 200)
    good, out = torch.empty(T, 300, device="cuda"), torch.empty(T, 300, device="cuda")
    moe.moe_linear(x, w, good, ws)
    x[3, 100] = value
    moe.moe_linear(x, w, out, ws)
    rows = [t for t in range(T) if t != 3]
    assert torch.equal(out[rows], good[rows])
    assert not torch.isfinite(out[3]).any()


def test_one_workspace_many_sizes_and_same_bits():
    ws = torch.full((max(moe.linear_workspace_bytes(*s) for s in SIZES),), 0xCD, dtype=torch.uint8, device="cuda")
    moe.status_clear(ws)
    first = [check(*s, seed=i, ws=ws).clone() for i, s in enumerate(SIZES)]
    for i, s in reversed(list(enumerate(SIZES))):
        assert torch.equal(check(*s, seed=i, ws=ws), first[i])


@pytest.mark.parametrize("T,N,K", [(7, 4096, 1024), (200, 640, 2048)])
def test_two_streams_and_graph(T, N, K):
    data = [make(T, N, K, True, True, s) for s in (6, 7)]
    want = []
    for x, w, b, r in data:
        o = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_linear(x, w, o, workspace(T, N, K), bias=b, activation="gelu", residual=r)
        want.append(o)
    ws = [workspace(T, N, K) for _ in data]
    out = [torch.empty_like(o) for o in want]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (x, w, b, r) in enumerate(data):
            moe.moe_linear(x, w, out[i], ws[i], bias=b, activation="gelu", residual=r, stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    x, w, b, r = [t.clone() for t in data[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear(x, w, out[0], ws[0], bias=b, activation="gelu", residual=r)
    for i in (1, 0, 1):
        for dst, src in zip((x, w, b, r), data[i]):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i])
    assert moe.status_read(ws[0]) == 0


def test_binding_refusals():
    x, w, b, r = make(4, 32, 64, True, True)
    ws = workspace(4, 32, 64)
    out = torch.empty(4, 32, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(activation="tanh"), dict(bias=b[:31]), dict(bias=b.float()), dict(residual=r.T),
               dict(residual=r.float())):
        with pytest.raises(ValueError):
            moe.moe_linear(x, w, out, ws, **kw)
    for args in ((x.float(), w, out), (x, w[:, :32], out), (x, w, out[:3]), (x, w, out.half())):
        with pytest.raises(ValueError):
            moe.moe_linear(*args, ws)
    with pytest.raises(moe.MoEError):
        moe.moe_linear(x, w, out, ws[:4096])
    with pytest.raises(moe.MoEError):
        moe.linear_workspace_bytes(4, 32, 60)
    moe.moe_linear(x[:0], w, out[:0], ws)  # a no-op
