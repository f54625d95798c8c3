// The whole routed layer for a few tokens (at most 16) in one kernel.
//
//   logits_t = W_r x_t (or given);  softmax, top-k, top-p trim, budget as the
//   stage kernels do them;
//   h[t, e] = w[t, e] silu(W_gate[e] x_t) * (W_up[e] x_t)   for the kept (t, e),
//   out_t   = sum_e W_down[e] h[t, e] + sigmoid(g . x_t) FFN_shared(x_t),
//
// the gate weight folded into h, so that the down projection is one product
// over the concatenated intermediate channels of the experts in use.
//
// One cooperative grid, one CTA per SM.  Every CTA routes all tokens itself
// (the routing is a few microseconds of work and saves a launch and a round
// trip); the grid meets twice: after the projection's logits, and after h.
#include <atomic>

#include "few.cuh"
#include "front.cuh"
#include "quant_codec.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {
using namespace tc;

constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewMaxSlots = kFewMaxTokens * kMaxTopK;

struct FewRouting {
    int32_t idx[kFewMaxSlots];
    float w[kFewMaxSlots];
    int32_t keff[kFewMaxTokens];
    uint32_t mask[kMaxExperts];  // tokens of each expert
    float agg[kMaxExperts];
    uint16_t list[kFewMaxSlots];  // experts in use, ascending
    int nu, ndrop, stop;
};

// Every CTA of the grid has arrived on *ctr (from zero) and its writes are visible.
__device__ bool grid_meet(int32_t *ctr, int32_t *status, int *stop) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(ctr, 1);
        const unsigned long long t0 = globaltimer();
        *stop = 0;
        while (ld_acquire(ctr) < (int)gridDim.x)
            if (globaltimer() - t0 > kWaitLimitNs) {
                atomicOr(status, MOE_STATUS_TIMEOUT);
                *stop = 1;
                break;
            }
    }
    __syncthreads();
    return *stop == 0;
}

template <int V>
__device__ __noinline__ int few_route_token(int t, const FewArgs &a, FewRouting &r, int lane) {
    return route_token<V, false>(t, a.E, a.k, a.norm_topk, a.topp, a.logits, r.idx, r.w, nullptr, lane);
}

// Route all tokens, apply the budget, list the experts in use (whole block).
__device__ void few_route(const FewArgs &a, FewRouting &r) {
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, Tk = a.T * a.k;
    for (int t = tid >> 5; t < a.T; t += nthr >> 5) {
        int c;
        if (a.E <= 128)
            c = few_route_token<4>(t, a, r, lane);
        else if (a.E <= 256)
            c = few_route_token<8>(t, a, r, lane);
        else if (a.E <= 512)
            c = few_route_token<16>(t, a, r, lane);
        else
            c = few_route_token<32>(t, a, r, lane);
        if (lane == 0) r.keff[t] = c;
    }
    for (int e = tid; e < kMaxExperts; e += nthr) r.mask[e] = 0;
    __syncthreads();
    for (int s = tid; s < Tk; s += nthr)
        if (r.idx[s] >= 0 && r.idx[s] < a.E) atomicOr(&r.mask[r.idx[s]], 1u << (s / a.k));
    __syncthreads();
    int mine = 0;
    for (int e = tid; e < a.E; e += nthr) mine += r.mask[e] != 0;
    if (tid == 0) r.nu = 0;
    __syncthreads();
    if (mine) atomicAdd(&r.nu, mine);
    __syncthreads();
    const int nu = r.nu;
    const bool cut = a.budget > 0 && nu > a.budget;
    if (cut) {
        // the sum of the weights routed to each expert, tokens then slots ascending
        for (int e = tid; e < a.E; e += nthr) {
            float s = 0.f;
            if (r.mask[e])
                for (int i = 0; i < Tk; ++i)
                    if (r.idx[i] == e) s += r.w[i];
            r.agg[e] = s;
        }
        __syncthreads();
        // rank in (sum descending, id ascending); the others leave
        bool drop[(kMaxExperts + 255) / 256];
        int n = 0;
        for (int e = tid; e < a.E; e += nthr, ++n) {
            int rank = 0;
            for (int o = 0; o < a.E; ++o)
                rank += r.mask[o] != 0 && (r.agg[o] > r.agg[e] || (r.agg[o] == r.agg[e] && o < e));
            drop[n] = r.mask[e] == 0 || rank >= a.budget;
        }
        __syncthreads();
        n = 0;
        for (int e = tid; e < a.E; e += nthr, ++n)
            if (drop[n]) r.mask[e] = 0;
        __syncthreads();
        for (int t = tid; t < a.T; t += nthr) {
            int32_t *ti = r.idx + t * a.k;
            float *tw = r.w + t * a.k;
            const int valid = r.keff[t];
            int c = 0;
            for (int j = 0; j < valid; ++j)
                if (r.mask[ti[j]]) {
                    const int e = ti[j];
                    const float w = tw[j];
                    ti[c] = e;
                    tw[c] = w;
                    ++c;
                }
            for (int j = c; j < a.k; ++j) {
                ti[j] = -1;
                tw[j] = 0.f;
            }
            if (a.norm_topk && c > 0 && c < valid) {
                float s = 0.f;
                for (int j = 0; j < c; ++j) s += tw[j];
                for (int j = 0; j < c; ++j) tw[j] = tw[j] / s;
            }
            r.keff[t] = c;
        }
    }
    __syncthreads();
    if (tid < 32) {
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const bool in = e0 + lane < a.E && r.mask[e0 + lane] != 0;
            const unsigned b = __ballot_sync(0xffffffffu, in);
            if (in) r.list[n + __popc(b & ((1u << lane) - 1u))] = (uint16_t)(e0 + lane);
            n += __popc(b);
        }
        if (lane == 0) {
            r.nu = n;
            r.ndrop = nu - n;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {  // the routing's optional outputs
        for (int s = tid; s < Tk; s += nthr) {
            if (a.idx) a.idx[s] = r.idx[s];
            if (a.w) a.w[s] = r.w[s];
        }
        for (int t = tid; t < a.T; t += nthr)
            if (a.keff) a.keff[t] = r.keff[t];
        if (a.budget > 0 && a.kept)
            for (int e = tid; e < a.E; e += nthr) a.kept[e] = r.mask[e] != 0;
        if (a.budget > 0 && a.n_dropped && tid == 0) *a.n_dropped = r.ndrop;
    }
}

__device__ __forceinline__ float few_weight(const FewArgs &a, const FewRouting &r, int t, int e) {
    for (int j = 0; j < r.keff[t]; ++j)
        if (r.idx[t * a.k + j] == e) return r.w[t * a.k + j];
    return 0.f;
}

// Eight consecutive weights of row r from column k (a multiple of 8) of a [rows, K] matrix.
template <int FMT>
__device__ __forceinline__ void load8(const FewMatrix &m, size_t r, int K, int k, float (&v)[8]) {
    if constexpr (FMT == 0) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(m.w) + r * K + k));
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else if constexpr (FMT == 1) {
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(m.w) + r * K + k));
        const int se = (int)m.sf[((r / 64 * (K / 128) + k / 128) * 64 + r % 64) * 4 + k % 128 / 32] - 127;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = bf16_bits_to_f32(quant::e4m3_scaled_bf16((uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3))), se));
    } else {
        const uint32_t q =
            __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(m.w) + (r * K + k) / 2));
        const uint8_t sc = m.sf[((r / 64 * (K / 128) + k / 128) * 64 + r % 64) * 8 + k % 128 / 16];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = bf16_bits_to_f32(quant::nvfp4_scaled_bf16((uint8_t)((q >> (4 * i)) & 15u), sc));
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// acc[t] += row r of m . x_t over K columns (x bf16 or fp32 [T, ldx]), this lane's share.
template <int FMT, class X>
__device__ __forceinline__ void row_dots(const FewMatrix &m, size_t r, int K, const X *x, size_t ldx, uint32_t tokens,
                                         int lane, float (&acc)[kFewMaxTokens]) {
    for (int k = lane * 8; k < K; k += 256) {
        float w[8];
        load8<FMT>(m, r, K, k, w);
#pragma unroll
        for (int t = 0; t < kFewMaxTokens; ++t)
            if ((tokens >> t) & 1u)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float xv;
                    if constexpr (sizeof(X) == 2)
                        xv = bf16_bits_to_f32(x[t * ldx + k + i]);
                    else
                        xv = __ldcg(x + t * ldx + k + i);
                    acc[t] = fmaf(w[i], xv, acc[t]);
                }
    }
}

template <int FMT>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const FewArgs a) {
    __shared__ FewRouting r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gw = blockIdx.x * kFewWarps + warp, nw = gridDim.x * kFewWarps;
    const uint32_t all = (1u << a.T) - 1u;
    float *h = static_cast<float *>(a.h);
    if (a.project) {
        const FewMatrix m{a.w_router, nullptr, nullptr};
        for (int e = gw; e < a.E; e += nw) {
            float acc[kFewMaxTokens] = {};
            row_dots<0>(m, e, a.H, a.x, a.H, all, lane, acc);
#pragma unroll
            for (int t = 0; t < kFewMaxTokens; ++t)
                if (t < a.T) {
                    const float s = warp_sum(acc[t]);
                    if (lane == 0) a.logits[(size_t)t * a.E + e] = s;
                }
        }
        if (!grid_meet(a.sync, a.status, &r.stop)) return;
    }
    few_route(a, r);
    if (a.Is > 0)
        for (int t = gw; t < a.T; t += nw) {
            float z = 0.f;
            for (int i = lane; i < a.H; i += 32)
                z = fmaf(bf16_bits_to_f32(a.x[(size_t)t * a.H + i]), bf16_bits_to_f32(a.gvec[i]), z);
            z = warp_sum(z);
            if (lane == 0) a.sgate[t] = 1.f / (1.f + expf(-z));
        }
    const int nu = r.nu, Kt = a.Is + nu * a.I;  // columns of h: shared first, then the experts in list order
    for (int c = gw; c < Kt; c += nw) {
        const bool sh = c < a.Is;
        const int u = sh ? 0 : (c - a.Is) / a.I, i = sh ? c : (c - a.Is) % a.I;
        const int e = sh ? 0 : r.list[u];
        const uint32_t tokens = sh ? all : r.mask[e];
        const FewMatrix &mg = sh ? a.s_gate : a.gate, &mu = sh ? a.s_up : a.up;
        const size_t row = sh ? (size_t)i : (size_t)e * a.I + i;
        float g[kFewMaxTokens] = {}, up[kFewMaxTokens] = {};
        row_dots<FMT>(mg, row, a.H, a.x, a.H, tokens, lane, g);
        row_dots<FMT>(mu, row, a.H, a.x, a.H, tokens, lane, up);
        const float tg = FMT == 2 ? mg.ts[e] : 1.f, tu = FMT == 2 ? mu.ts[e] : 1.f;
        const float td = FMT == 2 ? (sh ? a.s_down.ts[0] : a.down.ts[e]) : 1.f;
#pragma unroll
        for (int t = 0; t < kFewMaxTokens; ++t)
            if (t < a.T) {
                const float gs = warp_sum(g[t]) * tg, us = warp_sum(up[t]) * tu;
                float v = 0.f;
                if ((tokens >> t) & 1u) {
                    v = gs / (1.f + expf(-gs)) * us * td;
                    if (!sh) v *= few_weight(a, r, t, e);
                }
                if (lane == 0) h[(size_t)t * Kt + c] = v;
            }
    }
    if (!grid_meet(a.sync + 1, a.status, &r.stop)) return;
    for (int o = gw; o < a.H; o += nw) {
        float acc[kFewMaxTokens] = {};
        if (a.Is > 0) {
            row_dots<FMT>(a.s_down, o, a.Is, h, Kt, all, lane, acc);
#pragma unroll
            for (int t = 0; t < kFewMaxTokens; ++t)
                if (t < a.T) acc[t] *= __ldcg(a.sgate + t);
        }
        for (int u = 0; u < nu; ++u) {
            const int e = r.list[u];
            row_dots<FMT>(a.down, (size_t)e * a.H + o, a.I, h + a.Is + (size_t)u * a.I, Kt, r.mask[e], lane, acc);
        }
#pragma unroll
        for (int t = 0; t < kFewMaxTokens; ++t)
            if (t < a.T) {
                const float s = warp_sum(acc[t]);
                if (lane == 0) a.out[(size_t)t * a.H + o] = f32_to_bf16_bits(s);
            }
    }
    // the last CTA out leaves the counters at zero
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(a.sync + 2, 1) == (int)gridDim.x - 1) {
        a.sync[0] = 0;
        a.sync[1] = 0;
        a.sync[2] = 0;
    }
}

template <int FMT>
cudaError_t launch_fmt(const FewArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sm_count());
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few_kernel<FMT>, a);
}

}  // namespace

size_t few_h_bytes(int T, int E, int I, int k, int Is) {
    const size_t used = (size_t)std::min(E, T * k);
    return (size_t)kFewMaxTokens * (used * I + Is) * 4;
}

cudaError_t launch_few(const FewArgs &a, int fmt, cudaStream_t st) {
    return fmt == 0 ? launch_fmt<0>(a, st) : fmt == 1 ? launch_fmt<1>(a, st) : launch_fmt<2>(a, st);
}

}  // namespace moe
