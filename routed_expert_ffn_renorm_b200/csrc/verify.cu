// Verification of drafted tokens against the target's probabilities
// (speculative sampling; the drafter layers of SpecForge PR #943 draft the
// 7-token blocks this checks).
//
//   token x_i of a request stays while  u_i q_i(x_i) < p_i(x_i);
//   at the first refused one, j, the next token is drawn from
//   max(p_j - q_j, 0) normalised, after a block that stayed whole from p_L:
//   the first v whose running sum passes u total.
//
// A cluster of 8 CTAs per request, no workspace: every CTA decides the
// block's length itself (2 L gathered probabilities), sums its eighth of the
// vocabulary row, and the eight totals meet through distributed shared
// memory; the CTA whose range holds u total scans its warps' sums, the warp that
// holds it the sums it kept of its segment's eighths, and only that eighth is
// read again (from L2).  The row is read from HBM once: 8 V bytes
// per request, the bound for large batches; a small one is bound by the chain
// token -> p(x) -> row -> exchange -> segment: one request over 32768 tokens takes
// 5.7 us, 32 over 131072 10.7 us (3.1 TB/s; 15.5 us when the whole segment was
// read again).
//
// The sums are fp64: a token changes when a running sum crosses u total, and
// over V sums an fp32 error of 1e-7 would move one draw in a hundred at
// V = 131072.  The products u q and the differences p - q of fp32 values are
// exact or rounded once in fp64.
#include "front.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {
using namespace tc;

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerCluster = 8;
constexpr int kVerSubs = 8;  // parts of a warp's segment whose sums it keeps

struct VerArgs {
    int B, L, V;
    const float *p, *q;  // [B, L + 1, V]; [B, L, V] or null: the drafter put all its mass on the drafted token
    const int32_t *draft, *len;
    const float *u, *us;
    int32_t *tokens, *n_accepted;
};

// The row the next token is drawn from: max(p - q, 0), non-finite entries 0.
struct VerRow {
    const float *p, *q;
    int hot;  // token whose q is 1 (q == null), -1: none
    bool pv, qv;
    __device__ void values(long long i, long long end, double (&r)[4]) const {
        mass(i, load4(p, pv, i, end), q ? load4(q, qv, i, end) : make_float4(0.f, 0.f, 0.f, 0.f), r);
    }
    __device__ void mass(long long i, const float4 &a, const float4 &b, double (&r)[4]) const {
        const float x[4] = {a.x, a.y, a.z, a.w};
        float y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (i + c == hot) y[c] = 1.f;
            const double d = (double)x[c] - (double)y[c];
            r[c] = d > 0. && d <= 3.5e38 ? d : 0.;
        }
    }
    // values i .. i + 3, those from `end` on 0
    __device__ static float4 load4(const float *s, bool vec, long long i, long long end) {
        if (vec && i + 4 <= end) return __ldg(reinterpret_cast<const float4 *>(s + i));
        float v[4] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (i + c < end) v[c] = __ldg(s + i + c);
        return make_float4(v[0], v[1], v[2], v[3]);
    }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t cluster_addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(cluster_addr) : "memory");
    return v;
}

__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerArgs a) {
    __shared__ double wsum[kVerWarps];
    __shared__ double total[2];  // this CTA's sum of the row, of p alone when the first is 0
    __shared__ int s_n, s_refused;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), b = blockIdx.x / kVerCluster;
    const int V = a.V, L = a.L;
    pdl_launch_dependents();
    pdl_wait();

    if (warp == 0) {  // the accepted length
        const int n_in = a.len ? min(max(__ldg(a.len + b), 0), L) : L;
        int n = n_in, refused = 0;
        for (int i0 = 0; i0 < n_in; i0 += 32) {
            const int i = i0 + lane;
            bool stop = false, ref = false;
            if (i < n_in) {
                const int tok = __ldg(a.draft + (size_t)b * L + i);
                if (tok < 0 || tok >= V) {
                    stop = true;  // the block ends here
                } else {
                    const double px = __ldg(a.p + ((size_t)b * (L + 1) + i) * V + tok);
                    const double qx = a.q ? (double)__ldg(a.q + ((size_t)b * L + i) * V + tok) : 1.;
                    ref = stop = !((double)__ldg(a.u + (size_t)b * L + i) * qx < px);
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, stop);
            if (m) {
                const int f = __ffs(m) - 1;
                n = i0 + f;
                refused = __shfl_sync(0xffffffffu, (int)ref, f);
                break;
            }
        }
        if (lane == 0) {
            s_n = n;
            s_refused = refused;
        }
    }
    __syncthreads();
    const int n = s_n;
    VerRow row;
    row.p = a.p + ((size_t)b * (L + 1) + n) * V;
    row.q = s_refused && a.q ? a.q + ((size_t)b * L + n) * V : nullptr;
    row.hot = s_refused && !a.q ? __ldg(a.draft + (size_t)b * L + n) : -1;
    row.pv = (reinterpret_cast<uintptr_t>(row.p) & 15u) == 0;
    row.qv = (reinterpret_cast<uintptr_t>(row.q) & 15u) == 0;

    // this warp's segment: multiples of 128 values (one float4 per lane)
    const long long per = (((long long)V + kVerCluster * kVerWarps - 1) / (kVerCluster * kVerWarps) + 127) / 128 * 128;
    const long long s0 = min((long long)V, (rank * kVerWarps + warp) * per), s1 = min((long long)V, s0 + per);
    const long long sub = (per / 128 + kVerSubs - 1) / kVerSubs * 128;  // and its eighths
    double tot[kVerCluster], all = 0., sums[kVerSubs] = {};
    for (int pass = 0; pass < 2; ++pass) {
        double s = 0.;
        if (sub == 128 && s0 + per <= V && row.pv && (!row.q || row.qv)) {
            // a whole segment, aligned: one float4 per lane and eighth, four eighths in flight
            const float4 *p4 = reinterpret_cast<const float4 *>(row.p + s0) + lane;
            const float4 *q4 = reinterpret_cast<const float4 *>((row.q ? row.q : row.p) + s0) + lane;
            const int n = (int)(per / 128);
#pragma unroll
            for (int k0 = 0; k0 < kVerSubs; k0 += 4) {
                if (k0 >= n) break;
                float4 pf[4], qf[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // behind the segment: its last eighth again, not counted
                    pf[k] = __ldg(p4 + min(k0 + k, n - 1) * 32);
                    qf[k] = __ldg(q4 + min(k0 + k, n - 1) * 32);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    double r[4];
                    row.mass(s0 + (k0 + k) * 128 + lane * 4, pf[k], row.q ? qf[k] : make_float4(0.f, 0.f, 0.f, 0.f), r);
                    sums[k0 + k] = k0 + k < n ? (r[0] + r[1]) + (r[2] + r[3]) : 0.;
                }
            }
        } else {
#pragma unroll 1
            for (int k = 0; k < kVerSubs; ++k) {
                const long long e0 = min(s1, s0 + k * sub), e1 = min(s1, e0 + sub);
                double t = 0.;
#pragma unroll 4
                for (long long i = e0 + lane * 4; i < e1; i += 128) {
                    double r[4];
                    row.values(i, s1, r);
                    t += (r[0] + r[1]) + (r[2] + r[3]);
                }
#pragma unroll
                for (int c = 0; c < kVerSubs; ++c)
                    if (c == k) sums[c] = t;
            }
        }
#pragma unroll
        for (int k = 0; k < kVerSubs; ++k) s += sums[k];
        s = warp_sum(s);
        if (lane == 0) wsum[warp] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            double t = 0.;
            for (int w = 0; w < kVerWarps; ++w) t += wsum[w];
            total[pass] = t;
        }
        cluster_sync();
        all = 0.;
#pragma unroll
        for (int c = 0; c < kVerCluster; ++c) {
            tot[c] = ld_cluster_f64(mapa(smem_u32(&total[pass]), c));
            all += tot[c];
        }
        if (all > 0. || (!row.q && row.hot < 0)) break;
        // p <= q everywhere (rounded probabilities): draw from p itself
        row.q = nullptr;
        row.hot = -1;
        __syncthreads();  // wsum is rewritten
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA reads no peer's memory any more

    // the CTA, then the warp, whose range holds u total (rounding past the end: the last with mass)
    float us = __ldg(a.us + b);
    if (!(us > 0.f)) us = 0.f;
    const double target = (double)us * all;
    double before = 0.;
    int own = -1;
    double own_before = 0.;
    bool found = false;
#pragma unroll
    for (int c = 0; c < kVerCluster; ++c) {
        if (!found && tot[c] > 0.) {
            own = c;
            own_before = before;
            found = before + tot[c] > target;
        }
        before += tot[c];
    }
    int32_t *out = a.tokens + (size_t)b * (L + 1);
    if (rank == 0) {
        for (int i = threadIdx.x; i <= L; i += kVerThreads)
            if (i != n || own < 0) out[i] = i < n ? __ldg(a.draft + (size_t)b * L + i) : -1;
        if (threadIdx.x == 0) a.n_accepted[b] = n;
    }
    if (rank == own) {
        int ow = -1;
        double wb = 0., bw = own_before;
        bool wf = false;
        for (int w = 0; w < kVerWarps; ++w) {
            if (!wf && wsum[w] > 0.) {
                ow = w;
                wb = bw;
                wf = bw + wsum[w] > target;
            }
            bw += wsum[w];
        }
        if (warp == ow) {
            // the eighth of the segment (rounding past the end: the last with mass)
            double run = wb, bs = wb;
            long long tok = -1, last = -1, e0 = s0, e1 = s1;
            bool sf = false;
            if (per > 2 * 128) {  // (two eighths are as quickly read as summed)
#pragma unroll
                for (int k = 0; k < kVerSubs; ++k) {
                    const double t = warp_sum(sums[k]);
                    if (!sf && t > 0.) {
                        e0 = s0 + k * sub;
                        run = bs;
                        sf = bs + t > target;
                    }
                    bs += t;
                }
                e1 = min(s1, e0 + sub);
            }
            for (long long i0 = e0; i0 < e1 && tok < 0; i0 += 128) {
                const long long i = i0 + lane * 4;
                double r[4] = {};
                if (i < e1) row.values(i, s1, r);
                const double mine = (r[0] + r[1]) + (r[2] + r[3]);
                double incl = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += o;
                }
                // this lane's first passing value, and its last with mass
                double at = run + (incl - mine);
                int hit = -1, pos = -1;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    at += r[c];
                    if (r[c] > 0.) {
                        pos = c;
                        if (hit < 0 && at > target) hit = c;
                    }
                }
                const unsigned mh = __ballot_sync(0xffffffffu, hit >= 0), mp = __ballot_sync(0xffffffffu, pos >= 0);
                if (mh) {
                    const int f = __ffs(mh) - 1;
                    tok = i0 + f * 4 + __shfl_sync(0xffffffffu, hit, f);
                } else if (mp) {
                    const int f = 31 - __clz(mp);
                    last = i0 + f * 4 + __shfl_sync(0xffffffffu, pos, f);
                }
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) out[n] = (int32_t)(tok >= 0 ? tok : last);
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace

cudaError_t launch_verify(int B, int L, int V, const float *p, const float *q, const int32_t *draft,
                          const int32_t *len, const float *u, const float *us, int32_t *tokens, int32_t *n_accepted,
                          cudaStream_t st) {
    const VerArgs a{B, L, V, p, q, draft, len, u, us, tokens, n_accepted};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * kVerCluster);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kVerCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a);
}

}  // namespace moe
