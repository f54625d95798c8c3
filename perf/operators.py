"""Measured cases of the operators of one speculative decoding step.

layer   the whole routed MoE layer for a few tokens (moe_forward_few and its
        MXFP8 / NVFP4 forms): routing, expert FFN, shared expert, combine
linear  out = residual + act(x W^T + bias) (moe_linear), one row to many
verify  drafted tokens against the target's probabilities with given random
        numbers (moe_verify)

With ``own`` false, run() computes the operators from elementary torch
operations in 32 bits (64 where a border decides); with ``own`` true it makes
the calls a user of the library makes.
"""
import math

import torch

own = False

FEW_MAX = 16  # tokens of the few-token layer


# ------------------------------------------------------------------- cases --
def _layer(name, T, H, E, I, k, Is=0, router=False, budget=0, topp=0.0, alpha=0.0, fmt="bf16"):
    return {"name": name, "op": "layer", "T": T, "H": H, "E": E, "I": I, "k": k, "Is": Is, "router": router,
            "budget": budget, "topp": topp, "alpha": alpha, "fmt": fmt}


def _linear(name, T, N, K, act="none", bias=False, residual=False, out="bf16"):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "act": act, "bias": bias, "residual": residual,
            "out": out}


def _verify(name, B, L, V, ragged=False, onehot=False):
    return {"name": name, "op": "verify", "B": B, "L": L, "V": V, "ragged": ragged, "onehot": onehot}


def listed():
    return [
        # one token through the tiny layer: pure latency
        _layer("layer_tiny_1", 1, 256, 8, 128, 2),
        # the drafter layer (16 x 1024 experts, shared 2048) extending one sequence by one token
        _layer("layer_drafter_1", 1, 5120, 16, 1024, 2, Is=2048, router=True),
        # ... and drafting one request's 7-token block
        _layer("layer_drafter_7", 7, 5120, 16, 1024, 2, Is=2048, router=True),
        # a batch of positions under an expert budget
        _layer("layer_budget_16", 16, 4096, 128, 1536, 8, budget=12, alpha=1.2),
        # the large 256-expert layer decoding eight sequences
        _layer("layer_large_8", 8, 7168, 256, 2048, 8, router=True, alpha=1.0),
        # the many-narrow-experts drafter layer, MXFP8 weights, one 7-token block
        _layer("layer_narrow_mxfp8_7", 7, 5120, 512, 512, 10, Is=2048, router=True, alpha=1.0, fmt="mxfp8"),
        # the drafter layer with NVFP4 weights, two 7-token blocks
        _layer("layer_drafter_nvfp4_14", 14, 5120, 16, 1024, 2, Is=2048, router=True, fmt="nvfp4"),
        # the output head on a drafted block: fp32 logits over a vocabulary
        _linear("linear_head_7", 7, 131072, 5120, out="f32"),
        # the dense FFN's down projection on 32 blocks, bias and residual added
        _linear("linear_dense_224", 224, 5120, 17408, bias=True, residual=True),
        # a long prompt through a square projection with every epilogue part, an odd number of rows
        _linear("linear_long_8191", 8191, 7168, 7168, act="silu", bias=True, residual=True),
        # one request's block verified
        _verify("verify_1", 1, 7, 32768),
        # 32 requests over a large vocabulary, blocks of different lengths
        _verify("verify_32", 32, 7, 131072, ragged=True),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["layer", "layer", "linear", "verify"])
    if op == "layer":
        fmt = rng.choice(["bf16", "bf16", "mxfp8", "nvfp4"])
        step = 64 if fmt == "bf16" else 128
        T = _spread(rng, 1, FEW_MAX)
        H = _spread(rng, 256, 6144, 128)
        I = _spread(rng, 128, 2048, step)
        E = _spread(rng, 8, 192)
        k = min(E, _spread(rng, 1, 8))
        Is = rng.choice([0, _spread(rng, 128, 2048, step)])
        return _layer("", T, H, E, I, k, Is=Is, router=rng.random() < 0.5,
                      budget=rng.choice([0, 0, _spread(rng, 1, 24)]), topp=rng.choice([0.0, 0.0, 0.7]),
                      alpha=rng.choice([0.0, 1.0, 1.5]), fmt=fmt)
    if op == "linear":
        T, N, K = _spread(rng, 1, 8192), _spread(rng, 64, 16384), _spread(rng, 64, 8192, 8)
        while T * N * K > 2 ** 38:
            T = T // 2 + 1
        return _linear("", T, N, K, act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                       residual=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    return _verify("", _spread(rng, 1, 32), _spread(rng, 1, 16), _spread(rng, 1000, 131072),
                   ragged=rng.random() < 0.5, onehot=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs --
def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _mxfp8_pack(w):
    """bf16 [.., R, K] -> E4M3 codes (uint8) and UE8M0 scales in the FFN's layout [rows/64][K/128][64][4]."""
    b = w.float().unflatten(-1, (-1, 32))
    e = torch.floor(torch.log2(b.abs().amax(-1).clamp_min(2.0 ** -126))) - 8.0
    codes = (b * torch.exp2(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s = (e + 127.0).to(torch.uint8).reshape(-1, 64, w.shape[-1] // 128, 4)
    return codes.reshape(w.shape), s.permute(0, 2, 1, 3).contiguous()


def _nvfp4_pack(w):
    """bf16 [n, R, K] -> E2M1 codes (two per byte), E4M3 block scales [rows/64][K/128][64][8], fp32 matrix scales."""
    b = w.float().unflatten(-1, (-1, 16))
    ts = (b.abs().amax((1, 2, 3)) / (6.0 * 448.0)).clamp_min(1e-30)
    t = ts.view(-1, 1, 1)
    sb = (b.abs().amax(-1) / (6.0 * t)).to(torch.float8_e4m3fn)
    v = b / (sb.float() * t).clamp_min(1e-30).unsqueeze(-1)
    mag = torch.bucketize(v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device))
    code = (mag + 8 * (v < 0)).to(torch.uint8).reshape(w.shape)
    s = sb.view(torch.uint8).reshape(-1, 64, w.shape[-1] // 128, 8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.permute(0, 2, 1, 3).contiguous(), ts


def _weights(gen, E, R, K, fmt):
    """E matrices [R, K] ~ N(0, 0.02) in the format: a dict of w, s (packed block scales), t (matrix scales)."""
    if fmt == "bf16":
        return {"w": _normal(gen, (E, R, K), 0.02)}
    parts = []
    for e0 in range(0, E, 32):  # bounded fp32 temporaries
        w = _normal(gen, (min(32, E - e0), R, K), 0.02)
        parts.append(_mxfp8_pack(w) if fmt == "mxfp8" else _nvfp4_pack(w))
    return dict(zip("wst", [torch.cat(p) for p in zip(*parts)]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "layer":
        T, H, E, I, Is = (case[n] for n in ("T", "H", "E", "I", "Is"))
        s["x"] = _normal(gen, (T, H), 0.02)
        bias = -case["alpha"] * torch.log1p(torch.arange(E, device="cuda", dtype=torch.float32))
        if case["router"]:  # x W_r^T is about N(0, 1)
            s["w_router"] = _normal(gen, (E, H), 1.0 / (0.02 * math.sqrt(H)))
            s["logits"] = None
        else:
            s["logits"] = _normal(gen, (T, E), 1.0, torch.float32) + bias
        for n, e, r, c in (("gate", E, I, H), ("up", E, I, H), ("down", E, H, I)):
            s[n] = _weights(gen, e, r, c, case["fmt"])
        if Is:
            for n, r, c in (("s_gate", Is, H), ("s_up", Is, H), ("s_down", H, Is)):
                s[n] = _weights(gen, 1, r, c, case["fmt"])
            s["gvec"] = _normal(gen, (H,), 0.5)
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        odt = torch.float32 if case["out"] == "f32" else torch.bfloat16
        s["x"] = _normal(gen, (T, K), 1.0)
        s["w"] = _normal(gen, (N, K), 1.0 / math.sqrt(K))
        s["bias"] = _normal(gen, (N,), 0.5) if case["bias"] else None
        s["residual"] = _normal(gen, (T, N), 1.0) if case["residual"] else None
        s["out"] = torch.empty(T, N, dtype=odt, device="cuda")
    else:
        B, L, V = case["B"], case["L"], case["V"]
        # a drafter near its target: logits of spread 2, the draft's perturbed
        z = _normal(gen, (B, L + 1, V), 2.0, torch.float32)
        s["p"] = torch.softmax(z, -1)
        s["q"] = None if case["onehot"] else torch.softmax(z[:, :L] + _normal(gen, (B, L, V), 0.3, torch.float32), -1)
        cdf = (s["p"][:, :L] if case["onehot"] else s["q"]).double().cumsum(-1)
        at = torch.rand(B, L, 1, generator=gen, device="cuda", dtype=torch.float64) * cdf[..., -1:]
        s["draft"] = torch.searchsorted(cdf, at, right=True).squeeze(-1).clamp_max(V - 1).to(torch.int32)
        if case["onehot"]:  # a greedy drafter mostly proposes the target's favourite
            s["draft"] = torch.where(at.squeeze(-1) / cdf[..., -1] < 0.8, s["p"][:, :L].argmax(-1), s["draft"]).int()
        s["len"] = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32) if case["ragged"] else None
        s["u"] = torch.rand(B, L, generator=gen, device="cuda")
        s["u_sample"] = torch.rand(B, generator=gen, device="cuda")
        s["tokens"] = torch.empty(B, L + 1, dtype=torch.int32, device="cuda")
        s["n"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


# -------------------------------------------------------------- plain form --
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _unpack_scales(s, R, per):
    """[.. * R / 64][K / 128][64][per] -> [.., R, K / 128 * per]"""
    return s.permute(0, 2, 1, 3).reshape(-1, R, s.shape[1] * per)


def _dense(m, pick, fmt):
    """The picked matrices in fp32: [len(pick), R, K]."""
    w = m["w"][pick]
    if fmt == "bf16":
        return w.float()
    n, R = w.shape[:2]
    per = 4 if fmt == "mxfp8" else 8
    sc = m["s"].reshape(m["w"].shape[0], R // 64, -1, 64, per)[pick].flatten(0, 1)
    sc = _unpack_scales(sc, R, per)
    if fmt == "mxfp8":
        v = w.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
        return (v * torch.exp2(sc.float() - 127.0).unsqueeze(-1)).flatten(2)
    lut = torch.tensor(_E2M1, device=w.device)
    v = lut[torch.stack((w & 15, w >> 4), -1).flatten(2).int()].unflatten(-1, (-1, 16))
    v = v * sc.view(torch.float8_e4m3fn).float().unsqueeze(-1) * m["t"][pick].view(n, 1, 1, 1)
    return v.flatten(2)


def _routing(c, logits):
    """Top-k experts and their weights [T, k]; dropped slots have weight 0."""
    k = c["k"]
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    idx = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    w = w / w.sum(-1, keepdim=True)
    live = torch.ones_like(w, dtype=torch.bool)
    if 0.0 < c["topp"] < 1.0:
        live = w.cumsum(-1) - w < c["topp"]
        live[:, 0] = True
        w = w * live
        w = w / w.sum(-1, keepdim=True)
    if c["budget"]:
        agg = torch.zeros(c["E"], device=w.device, dtype=torch.float64)
        agg = agg.index_add(0, idx.flatten(), w.double().flatten()).float()
        used = torch.zeros(c["E"], device=w.device, dtype=torch.bool).index_fill(0, idx[live], True)
        order = torch.sort(torch.where(used, agg, torch.full_like(agg, -1.0)), descending=True, stable=True).indices
        keep = torch.zeros_like(used).index_fill(0, order[:c["budget"]], True) & used
        live = live & keep[idx]
        w = w * live
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, w)
    return idx, w, live


def _layer_plain(s):
    c, fmt = s["case"], s["case"]["fmt"]
    x = s["x"].float()
    logits = s["logits"] if s["logits"] is not None else x @ s["w_router"].float().T
    idx, w, live = _routing(c, logits)
    pick, place = torch.unique(idx[live], return_inverse=True)
    dense = torch.zeros(c["T"], pick.numel(), device=x.device)
    dense[live.nonzero()[:, 0], place] = w[live]
    g, u = x @ _dense(s["gate"], pick, fmt).transpose(1, 2), x @ _dense(s["up"], pick, fmt).transpose(1, 2)
    h = g / (1.0 + torch.exp(-g)) * u * dense.T.unsqueeze(-1)
    out = (h @ _dense(s["down"], pick, fmt).transpose(1, 2)).sum(0)
    if c["Is"]:
        one = torch.zeros(1, dtype=torch.int64, device=x.device)
        g, u = x @ _dense(s["s_gate"], one, fmt)[0].T, x @ _dense(s["s_up"], one, fmt)[0].T
        z = x @ s["gvec"].float()
        y = (g / (1.0 + torch.exp(-g)) * u) @ _dense(s["s_down"], one, fmt)[0].T
        out = out + y / (1.0 + torch.exp(-z)).unsqueeze(-1)
    return out.to(torch.bfloat16)


def _act(v, act):
    if act == "relu":
        return v.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v / (1.0 + torch.exp(-v)) if act == "silu" else v


def _linear_plain(s):
    v = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _act(v, s["case"]["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["out"].dtype)


def _verify_plain(s):
    B, L, V = s["case"]["B"], s["case"]["L"], s["case"]["V"]
    at = torch.arange(B, device="cuda")
    slot = torch.arange(L, device="cuda")
    px = s["p"][:, :L].gather(2, s["draft"].long().unsqueeze(-1)).squeeze(-1).double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(2, s["draft"].long().unsqueeze(-1)).squeeze(-1).double()
    n_in = torch.full((B,), L, device="cuda") if s["len"] is None else s["len"].long()
    ok = (s["u"].double() * qx < px) & (slot < n_in.unsqueeze(1))
    n = ok.long().cumprod(1).sum(1)
    p = s["p"][at, n].double()
    refused = n < n_in
    j = n.clamp_max(L - 1)
    if s["q"] is None:
        q = torch.zeros_like(p).scatter(1, s["draft"].long().gather(1, j.unsqueeze(1)), 1.0)
    else:
        q = s["q"][at, j].double()
    r = (p - q * refused.unsqueeze(1)).clamp_min(0.0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    cdf = r.cumsum(1)
    t = torch.searchsorted(cdf, s["u_sample"].double().unsqueeze(1) * cdf[:, -1:], right=True).clamp_max(V - 1)
    col = torch.arange(L + 1, device="cuda")
    drafted = torch.cat((s["draft"], s["draft"][:, :1]), 1)
    tokens = torch.where(col < n.unsqueeze(1), drafted, torch.where(col == n.unsqueeze(1), t.int(), -1))
    return {"tokens": tokens.int(), "n_accepted": n.int()}


# --------------------------------------------------------------- own calls --
def _layer_handle(s, moe):
    """What a program keeps of a layer: its configuration, weights and workspace."""
    c, fmt = s["case"], s["case"]["fmt"]
    cfg = moe.MoEConfig(hidden=c["H"], n_routed_experts=c["E"], moe_intermediate_size=c["I"],
                        num_experts_per_tok=c["k"], shared_intermediate_size=c["Is"], budget=c["budget"],
                        topp=c["topp"])
    names = {"w_gate": "gate", "w_up": "up", "w_down": "down"}
    if c["Is"]:
        names.update(ws_gate="s_gate", ws_up="s_up", ws_down="s_down")
    kw = {n: s[m]["w"][0] if n.startswith("ws_") else s[m]["w"] for n, m in names.items()}
    if fmt != "bf16":
        kw.update({n + "_scale": s[m]["s"] for n, m in names.items()})
    if fmt == "nvfp4":
        kw.update(w_gate_tscale=s["gate"]["t"], w_up_tscale=s["up"]["t"], w_down_tscale=s["down"]["t"])
        if c["Is"]:
            kw["ws_tscale"] = torch.cat([s[m]["t"] for m in ("s_gate", "s_up", "s_down")])
    kind = {"bf16": moe.MoEWeights, "mxfp8": moe.MoEWeightsMXFP8, "nvfp4": moe.MoEWeightsNVFP4}[fmt]
    call = {"bf16": moe.moe_forward_few, "mxfp8": moe.moe_forward_few_mxfp8, "nvfp4": moe.moe_forward_few_nvfp4}[fmt]
    weights = kind(**kw, ws_gate_vec=s.get("gvec"), w_router=s.get("w_router"))
    ws = torch.empty(moe.workspace_bytes(cfg, c["T"]), dtype=torch.uint8, device="cuda")
    moe.status_clear(ws)
    return call, cfg, weights, ws


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import routed_expert_ffn_renorm_b200 as moe
        if op == "layer":
            if "handle" not in s:
                s["handle"] = _layer_handle(s, moe)
            call, cfg, weights, ws = s["handle"]
            call(cfg, s["x"], s["logits"], weights, s["out"], ws)
            return s["out"]
        if op == "linear":
            if "handle" not in s:
                c = s["case"]
                s["handle"] = torch.empty(moe.linear_workspace_bytes(c["T"], c["N"], c["K"]), dtype=torch.uint8,
                                          device="cuda")
                moe.status_clear(s["handle"])
            moe.moe_linear(s["x"], s["w"], s["out"], s["handle"], bias=s["bias"], activation=s["case"]["act"],
                           residual=s["residual"])
            return s["out"]
        moe.moe_verify(s["p"], s["draft"], s["u"], s["u_sample"], s["tokens"], s["n"], draft_probs=s["q"],
                       draft_len=s["len"])
        return {"tokens": s["tokens"], "n_accepted": s["n"]}
    return {"layer": _layer_plain, "linear": _linear_plain, "verify": _verify_plain}[op](s)


# ------------------------------------------------------------ least work ----
def work(case):
    c = case
    if c["op"] == "layer":
        per = {"bf16": 2.0, "mxfp8": 1.0 + 1 / 32, "nvfp4": 0.5 + 1 / 16}[c["fmt"]]
        # experts the batch reaches: the expected union under the case's popularity (independent draws)
        pop = [(e + 1.0) ** -(c["alpha"] if not c["router"] else 0.0) for e in range(c["E"])]
        tot = sum(pop)
        union = sum(1.0 - (1.0 - min(1.0, c["k"] * v / tot)) ** c["T"] for v in pop)
        union = max(float(c["k"]), min(union, float(c["E"]), float(c["T"] * c["k"])))
        if c["budget"]:
            union = min(union, float(c["budget"]))
        weights = 3.0 * c["H"] * (union * c["I"] + c["Is"])
        router = c["E"] * c["H"] * 2.0 if c["router"] else c["T"] * c["E"] * 4.0
        flops = 6.0 * c["T"] * c["H"] * (c["k"] * c["I"] + c["Is"]) + (2.0 * c["T"] * c["E"] * c["H"] if c["router"] else 0.0)
        return {"bytes": weights * per + router + 4.0 * c["T"] * c["H"], "flops": flops}
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        o = 4 if c["out"] == "f32" else 2
        return {"bytes": 2.0 * (T * K + N * K) + o * T * N + 2.0 * N * c["bias"] + 2.0 * T * N * c["residual"],
                "flops": 2.0 * T * N * K}
    rows = 1 if c["onehot"] else 2
    return {"bytes": 4.0 * c["B"] * (rows * c["V"] + 4 * c["L"] + 3), "flops": 3.0 * c["B"] * c["V"]}


# ----------------------------------------------------- 64-bit definition ----
def _decode64(m, e, fmt):
    """Matrix e in 64 bits, element by element from the format's definition."""
    w = m["w"][e]
    if fmt == "bf16":
        return w.double()
    R = w.shape[0]
    if fmt == "mxfp8":
        code = w.long()
        ex, man = (code >> 3) & 15, code & 7
        v = torch.where(ex > 0, (8 + man).double() * 2.0 ** (ex - 10).double(), man.double() * 2.0 ** -9)
        v = torch.where(code > 127, -v, v)
        per, step = 4, 32
    else:
        code = torch.empty(R, 2 * w.shape[1], dtype=torch.int64, device=w.device)
        code[:, 0::2], code[:, 1::2] = w.long() & 15, w.long() >> 4
        ex, man = (code >> 1) & 3, code & 1
        v = torch.where(ex > 0, (2 + man).double() * 2.0 ** (ex - 2).double(), man.double() * 0.5)
        v = torch.where(code > 7, -v, v)
        per, step = 8, 16
    K = v.shape[1]
    r = torch.arange(R, device=w.device).unsqueeze(1)
    b = torch.arange(K // step, device=w.device).unsqueeze(0)
    flat = m["s"].flatten()
    at = (((e * R + r) // 64 * (K // 128) + b // per) * 64 + r % 64) * per + b % per
    sc = flat[at].long()
    if fmt == "mxfp8":
        sc = 2.0 ** (sc - 127).double()
    else:
        sx, sm = (sc >> 3) & 15, sc & 7
        sc = torch.where(sx > 0, (8 + sm).double() * 2.0 ** (sx - 10).double(), sm.double() * 2.0 ** -9)
        sc = sc * m["t"][e].double()
    return v * sc.repeat_interleave(step, 1)


def _ffn64(x, s, names, e, fmt):
    g, u = x @ _decode64(s[names[0]], e, fmt).T, x @ _decode64(s[names[1]], e, fmt).T
    return (g * torch.sigmoid(g) * u) @ _decode64(s[names[2]], e, fmt).T


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        k, fmt = case["k"], case["fmt"]
        x = s["x"].double()
        logits = s["logits"].double() if s["logits"] is not None else x @ s["w_router"].double().T
        prob = torch.softmax(logits, -1).tolist()
        chosen = []
        for row, l in zip(prob, logits.tolist()):
            best = sorted(range(len(l)), key=lambda e: (-l[e], e))[:k]
            kept = [(e, row[e]) for e in best]
            total = sum(v for _, v in kept)
            kept = [(e, v / total) for e, v in kept]
            if 0.0 < case["topp"] < 1.0:
                n, mass = 0, 0.0
                while n < k and (n == 0 or mass < case["topp"]):
                    mass += kept[n][1]
                    n += 1
                kept = [(e, v / mass) for e, v in kept[:n]]
            chosen.append(kept)
        if case["budget"]:
            agg = {}
            for kept in chosen:
                for e, v in kept:
                    agg[e] = agg.get(e, 0.0) + v
            alive = set(sorted(agg, key=lambda e: (-agg[e], e))[:case["budget"]])
            for t, kept in enumerate(chosen):
                left = [(e, v) for e, v in kept if e in alive]
                total = sum(v for _, v in left)
                chosen[t] = [(e, v / total) for e, v in left]
        out = torch.zeros_like(x)
        for e in sorted({e for kept in chosen for e, _ in kept}):
            rows = [t for t, kept in enumerate(chosen) if any(f == e for f, _ in kept)]
            w = torch.tensor([dict(chosen[t])[e] for t in rows], dtype=torch.float64, device=x.device)
            out[rows] += w.unsqueeze(1) * _ffn64(x[rows], s, ("gate", "up", "down"), e, fmt)
        if case["Is"]:
            out += torch.sigmoid(x @ s["gvec"].double()).unsqueeze(1) * _ffn64(x, s, ("s_gate", "s_up", "s_down"), 0, fmt)
        return out
    if case["op"] == "linear":
        x, w = s["x"], s["w"]
        v = torch.empty(case["T"], case["N"], dtype=torch.float64, device=x.device)
        for n0 in range(0, case["N"], 8192):
            v[:, n0:n0 + 8192] = x.double() @ w[n0:n0 + 8192].double().T
        if s["bias"] is not None:
            v += s["bias"].double()
        f = {"none": lambda a: a, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
             "silu": torch.nn.functional.silu}[case["act"]]
        v = f(v)
        return v if s["residual"] is None else v + s["residual"].double()
    B, L, V = case["B"], case["L"], case["V"]
    tokens = torch.full((B, L + 1), -1, dtype=torch.int32)
    counts = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n_in = L if s["len"] is None else int(s["len"][b])
        n = 0
        while n < n_in:
            d = int(s["draft"][b, n])
            q = 1.0 if s["q"] is None else float(s["q"][b, n, d])
            if not float(s["u"][b, n]) * q < float(s["p"][b, n, d]):
                break
            tokens[b, n] = d
            n += 1
        r = s["p"][b, n].double().clone()
        if n < n_in:
            if s["q"] is None:
                r[int(s["draft"][b, n])] -= 1.0
            else:
                r -= s["q"][b, n].double()
        r = torch.relu(r)
        if float(r.sum()) <= 0.0:
            r = s["p"][b, n].double()
        c = r.cumsum(0)
        tokens[b, n] = min(V - 1, int((c <= float(s["u_sample"][b]) * c[-1]).sum()))
        counts[b] = n
    return {"tokens": tokens, "n_accepted": counts}
