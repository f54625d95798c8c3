"""64-bit references of the decode operators, and the elementwise error each
may have, from the sizes alone.

Rounding to bf16 moves a value by at most 2^-8 of itself, an fp32 sum of n
products by at most n 2^-23 of the sum of their magnitudes (every partial sum
rounded or truncated once), whatever the order.
"""
import math

import torch

BF16 = 2.0 ** -8
F32 = 2.0 ** -23


def dense(m, scale=None, tscale=None, per=0):
    """Matrices [n, R, K] in fp64 from bf16 values or codes with packed scales."""
    if scale is None:
        return m.double()
    w = m if m.dim() == 3 else m.unsqueeze(0)
    n, R = w.shape[:2]
    if per == 4:  # E4M3 codes, a power of two per 32
        v = w.view(torch.float8_e4m3fn).double()
        step = 32
    else:  # E2M1 codes, low nibble first, an E4M3 scale per 16
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                           device=w.device)
        v = torch.stack((lut[(w & 15).long()], lut[(w >> 4).long()]), -1).flatten(2)
        step = 16
    K = v.shape[2]
    s = scale.reshape(n, R // 64, K // 128, 64, per).permute(0, 1, 3, 2, 4).reshape(n, R, K // step)
    s = torch.exp2(s.double() - 127) if per == 4 else s.view(torch.float8_e4m3fn).double()
    v = v * s.repeat_interleave(step, 2)
    if tscale is not None:
        v = v * tscale.double().reshape(n, 1, 1)
    return v if m.dim() == 3 else v[0]


def weights64(w):
    """gate, up, down, shared gate, up, down of any of the weight classes, in fp64."""
    names = ["w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down"]
    out = []
    for i, n in enumerate(names):
        m = getattr(w, n)
        if m is None:
            out.append(None)
            continue
        sc = getattr(w, n + "_scale", None)
        ts = getattr(w, n + "_tscale", None)
        if sc is not None and hasattr(w, "ws_tscale"):
            ts = ts if i < 3 else w.ws_tscale[i - 3]
            out.append(dense(m, sc, ts, 8))
        else:
            out.append(dense(m, sc, None, 4))
    return out


def route(logits, k, norm, topp, budget):
    """[(expert, weight), ...] of each token, and the number of experts the budget dropped."""
    chosen = []
    for row in logits.double().cpu().tolist():
        m = max(row)
        z = sum(math.exp(v - m) for v in row)
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        kept = [(e, math.exp(row[e] - m) / z) for e in best]
        if norm:
            s = sum(w for _, w in kept)
            kept = [(e, w / s) for e, w in kept]
        if 0 < topp < 1:
            n, mass = 1, kept[0][1]
            while n < k and mass < topp:
                mass += kept[n][1]
                n += 1
            if norm and n < k:
                s = sum(w for _, w in kept[:n])
                kept = [(e, w / s) for e, w in kept]
            kept = kept[:n]
        chosen.append(kept)
    agg = {}
    for kept in chosen:
        for e, w in kept:
            agg[e] = agg.get(e, 0.0) + w
    drop = max(0, len(agg) - budget) if budget else 0
    if drop:
        alive = set(sorted(agg, key=lambda e: (-agg[e], e))[:budget])
        for t, kept in enumerate(chosen):
            left = [(e, w) for e, w in kept if e in alive]
            if norm and 0 < len(left) < len(kept):
                s = sum(w for _, w in left)
                left = [(e, w / s) for e, w in left]
            chosen[t] = left
    return chosen, drop


def layer(x, w, chosen, gvec=None):
    """The layer's output [T, H] in fp64 and its elementwise error bound for a
    bf16 result.  Gate and up are fp32 sums of H products; h keeps 2^-16 of
    itself (a bf16 and its remainder), and a few fp32 roundings of the SwiGLU
    and the gate weight (within 4e-6); out is an fp32 sum over all channels."""
    wg, wu, wd, sg, su, sd = w
    x = x.double()
    T, H = x.shape
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    chans = len({e for c in chosen for e, _ in c}) * wg.shape[1] + (0 if sg is None else sg.shape[0])

    def add(t, g_w, u_w, d_w, weight):
        g, u = g_w @ x[t], u_w @ x[t]
        dg, du = H * F32 * (g_w.abs() @ x[t].abs()), H * F32 * (u_w.abs() @ x[t].abs())
        s = g * torch.sigmoid(g)
        h = s * u * weight
        dh = weight * (1.1 * dg * (u.abs() + du) + s.abs() * du) + h.abs() * (2.0 ** -16 + 6e-6)
        out[t] += d_w @ h
        err[t] += d_w.abs() @ (dh + (chans + 64) * F32 * h.abs())

    for t, kept in enumerate(chosen):
        for e, weight in kept:
            add(t, wg[e], wu[e], wd[e], weight)
        if sg is not None:
            add(t, sg, su, sd, float(torch.sigmoid(gvec.double() @ x[t])))
    return out, err + BF16 * out.abs() + 1e-37


def linear(x, w, bias, act, residual, f32):
    """out in fp64 and its bound: the fp32 sum, the activation (slope at most
    1.13, a few ulps of itself) and, for bf16, the rounding."""
    x, w = x.double(), w.double()
    v = x @ w.T
    err = (x.shape[1] + 2) * F32 * (x.abs() @ w.abs().T)
    if bias is not None:
        v = v + bias.double()
        err = err + F32 * v.abs()
    f = {"none": lambda a: a, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu}[act]
    y = f(v)
    err = 1.13 * err + (0 if act in ("none", "relu") else 8 * F32 * (y.abs() + v.abs().clamp_max(16) * y.abs()))
    if residual is not None:
        y = y + residual.double()
    return y, err + (F32 if f32 else BF16) * y.abs() + 1e-37


def verify(p, q, draft, length, u, us):
    """Tokens and accepted counts by the definition, in Python floats (fp64)."""
    B, L1, V = p.shape
    L = L1 - 1
    tokens, counts = [], []
    for b in range(B):
        n_in = L if length is None else min(max(int(length[b]), 0), L)
        row, n, refused = [], 0, False
        while n < n_in:
            d = int(draft[b, n])
            if not 0 <= d < V:
                break
            qx = 1.0 if q is None else float(q[b, n, d])
            if not float(u[b, n]) * qx < float(p[b, n, d]):
                refused = True
                break
            row.append(d)
            n += 1

        def masses(sub):
            r = p[b, n].double()
            if sub and q is None:
                r = r.clone()
                r[int(draft[b, n])] -= 1.0
            elif sub:
                r = r - q[b, n].double()
            return torch.where((r > 0) & torch.isfinite(r), r, torch.zeros_like(r))

        r = masses(refused)
        if refused and float(r.sum()) == 0.0:
            r = masses(False)
        c = r.cumsum(0)
        t = float(us[b])
        t = (t if t > 0 else 0.0) * float(c[-1])
        hit = torch.nonzero((c > t) & (r > 0))
        live = torch.nonzero(r > 0)
        row.append(int(hit[0]) if len(hit) else int(live[-1]) if len(live) else -1)
        tokens.append(row + [-1] * (L - n))
        counts.append(n)
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32)
