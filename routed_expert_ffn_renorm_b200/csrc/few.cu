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
// Bound: every weight of the experts in use crosses HBM once; with at most 16
// tokens the arithmetic is a few percent of that time.  So the kernel is one
// weight stream.  A cooperative grid, one CTA per SM, walks three lists of row
// blocks of 128 weight rows -- the shared expert's gate/up (64 channels: 64 gate
// and 64 up rows), the routed experts' gate/up, the down projection -- each list
// cut into equal contiguous shares, so that all SMs stream until the end whatever
// the sizes.  A share's ends fall inside row blocks: those blocks' sums go to the
// workspace as fp32 partials, and the last CTA to arrive adds them in CTA order
// (the same bits on every run).
//
// Measured in a graph of calls (bf16): 256 experts, 8 tokens, 5.06 GB of weights in
// 766 us, 6.6 TB/s; the drafter layer (16 x 1024 experts, shared 2048), 7 tokens,
// 369 MB in 69 to 72 us, of which about 12 us are the fill, the wait for h between
// the gate/up and the down projection, and the last row blocks' partials.
// Block-scaled weights are paced by the consumers' instructions, half of them
// decoding (about 2 a cycle): MXFP8 4.5 TB/s, NVFP4 1.9 TB/s.
//
// Roles: one producer warp streams the weights into a shared-memory ring by TMA,
// two chunks of the K axis in a 3-D box (one thread's copies cost 75 ns each:
// with one chunk a box the issue, not HBM, set the pace at 4.7 TB/s), running
// ahead over everything the weights do not depend on -- the shared expert's while
// the tokens are still being routed, the down projection's while h is still being
// made; a second one loads the matching token operand (x, or h after the grid
// barrier) for the same ring slots; 16 consumer warps multiply: 4 groups, each a
// quarter of a step's columns, of 4 warps with 32 weight rows, so that a warp's
// token fragments serve two row tiles; 2 warps route beside the shared expert's
// stream.
//
// The consumers multiply with mma.sync: its 16 x 8 x 16 tile takes 16 weight rows
// by 8 tokens, so that 1..8 tokens waste no operand traffic, and the weights go
// from shared memory straight to registers; tcgen05 would pad the tokens and
// stage converted weights through tensor memory for no gain, the tensor pipe
// being idle most of the time either way.
//
// h is kept as a bf16 and its bf16 remainder (two token operands, one weight
// operand): 16 significant bits, so that the result differs from fp32
// arithmetic by its final rounding only.
#include <atomic>
#include <type_traits>

#include "few.cuh"
#include "front.cuh"
#include "quant_codec.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {
using namespace tc;

constexpr int kFewGroups = 4;                    // consumer groups: each takes a quarter of a step's columns
constexpr int kFewConsumers = kFewGroups * 128;  // 4 warps of 32 weight rows per group
constexpr int kFewRouters = 64;                  // routing threads beside a shared expert's phase
constexpr int kFewThreads = kFewConsumers + 64 + kFewRouters;  // + weight producer, token producer
constexpr int kFewMaxSlots = kFewMaxTokens * kMaxTopK;
constexpr int kFewMaxSms = 160;
constexpr int kFewSmem = 227 * 1024;

struct FewRouting {
    int32_t idx[kFewMaxSlots];
    float w[kFewMaxSlots];
    int32_t keff[kFewMaxTokens];
    uint32_t mask[kMaxExperts];  // tokens of each expert
    float agg[kMaxExperts];
    uint16_t list[kFewMaxSlots];  // experts in use, ascending
    int nu;
};

// Arrive on a grid barrier (one thread, after a CTA barrier of the writers), and
// wait for all of the grid.  `which` names the wait: 0 the logits, 1 h, 2 the picks.
__device__ __forceinline__ void grid_arrive(int32_t *ctr) { add_release(ctr, 1); }
__device__ __forceinline__ bool grid_wait(const FewArgs &a, int which, int32_t *ctr, int arrivals,
                                          volatile int *abort_flag) {
    const unsigned long long t0 = globaltimer();
    while (ld_acquire(ctr) < arrivals + (a.stall_wait == which)) {
        if (*abort_flag) return false;
        if (globaltimer() - t0 > a.wait_limit_ns) {
            *abort_flag = 1;
            atomicOr(a.status, MOE_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void consumers_sync() { named_bar_sync(1, kFewConsumers); }

// K splits of the projection: the grid over groups of 8 experts, a split no
// narrower than one 64-wide block per warp.
constexpr int kFewMaxSplits = 8;
__device__ __forceinline__ int few_splits(const FewArgs &a) {
    const int blocks = (a.H / 64 + kFewConsumers / 32 - 1) / (kFewConsumers / 32);
    return max(1, min(min((int)gridDim.x / ((a.E + 7) / 8), blocks), kFewMaxSplits));
}

// Four bytes from global (L2) to shared memory; visible to this thread after cp.async.wait_all.
__device__ __forceinline__ void copy_async4(float *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Route token t (one warp): the decisions of route_token, written as short loops
// over a row of keys in shared memory, as this code runs once per token and cold.
// Lane l owns experts l + 32 i, so the row needs no barrier.  splits > 1: the
// logits are that many partials at `lpart`.  `row`: kFewRowWords words, the keys
// and a stage for the loads, so that a round trip to L2 (1 to 2 us beside the
// weight stream) fetches 32 values per lane.
constexpr int kFewRowWords = 2 * kMaxExperts;
__device__ __forceinline__ void few_route_one(int t, const FewArgs &a, FewRouting &r, int splits, const float *lpart,
                                           uint32_t *row, bool keep, int lane) {
    const int E = a.E, k = a.k;
    const float *src = splits > 1 ? lpart + (size_t)t * E : a.logits + (size_t)t * E;
    const int slots = (E + 31) >> 5;
    // slots per round trip: a power of two, at most 32 loads
    int lg = 0;
    while ((1 << lg) < slots && (splits << (lg + 1)) <= 32) ++lg;
    const int nj = 1 << lg;
    float *stage = reinterpret_cast<float *>(row + kMaxExperts) + lane;
    uint32_t km = 0;
#pragma unroll 1
    for (int j0 = 0; j0 < slots; j0 += nj) {
#pragma unroll 1
        for (int f = 0; f < splits << lg; ++f) {
            const int e = lane + 32 * (j0 + (f & (nj - 1)));
            copy_async4(stage + f * 32, src + (f >> lg) * a.T * E + min(e, E - 1));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
        for (int j = 0; j < min(nj, slots - j0); ++j) {
            float s = 0.f;
#pragma unroll 1
            for (int i = 0; i < splits; ++i) s += stage[((i << lg) + j) * 32];
            const int e = lane + 32 * (j0 + j);
            if (e < E) {
                const uint32_t key = max(float_order_key(s), 1u);  // 0 marks a chosen expert; only the NaN of all ones has it
                km = max(km, key);
                row[e] = key;
                if (keep && splits > 1) a.logits[(size_t)t * E + e] = s;
            }
        }
    }
    const float m = order_key_float(__reduce_max_sync(0xffffffffu, km));
    float s = 0.f;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) s += expf(order_key_float(row[e]) - m);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    // k rounds of the largest key, the lowest id among equal ones.  Each lane holds
    // its two best; it looks through its row again when both are gone.
    uint32_t best = 0u, at = 0xffffffffu, second = 0u, at2 = 0xffffffffu;
    auto scan = [&] {
        best = second = 0u;
        at = at2 = 0xffffffffu;
#pragma unroll 4
        for (int e = lane; e < E; e += 32) {
            const uint32_t key = row[e];
            if (key > best) {
                second = best;
                at2 = at;
                best = key;
                at = e;
            } else if (key > second) {
                second = key;
                at2 = e;
            }
        }
    };
    scan();
    int my_idx = -1;
    uint32_t my_key = 0u;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        const uint32_t kmax = __reduce_max_sync(0xffffffffu, best);
        const int win = (int)__reduce_min_sync(0xffffffffu, best == kmax ? at : 0xffffffffu);
        if (lane == j) {
            my_idx = win;
            my_key = kmax;
        }
        if ((win & 31) == lane) {
            row[win] = 0u;
            best = second;
            at = at2;
            second = 0u;
            if (best == 0u) scan();
        }
    }
    float p = lane < k ? expf(order_key_float(my_key) - m) / s : 0.f;
    auto normalise = [&](int n) {  // by the sum of the first n, in slot order
        float sum = 0.f;
#pragma unroll 1
        for (int j = 0; j < n; ++j) sum += __shfl_sync(0xffffffffu, p, j);
        p = p / sum;
    };
    if (a.norm_topk) normalise(k);
    int c = k;  // kept slots
    if (a.topp > 0.f && a.topp < 1.f) {
        float mass = __shfl_sync(0xffffffffu, p, 0);  // the same in every lane
        for (c = 1; c < k && mass < a.topp; ++c) mass += __shfl_sync(0xffffffffu, p, c);
        if (a.norm_topk && c < k) normalise(c);
    }
    if (lane < k) {
        r.idx[t * k + lane] = lane < c ? my_idx : -1;
        r.w[t * k + lane] = lane < c ? p : 0.f;
    }
    if (lane == 0) r.keff[t] = c;
    __syncwarp();
}

// Every token routed by this CTA, a warp each.
__device__ __forceinline__ void few_route_all(const FewArgs &a, FewRouting &r, int splits, const float *lpart,
                                              uint32_t *rows, int warp, int lane) {
    for (int t = warp; t < a.T; t += kFewConsumers / 32)
        few_route_one(t, a, r, splits, lpart, rows + warp * kFewRowWords, blockIdx.x == 0, lane);
}

// Every token routed by one CTA of the grid and read by all (64 threads): `picks`
// holds [T] kept counts, [T k] experts, [T k] weights; `ctr` counts the tokens.
__device__ __forceinline__ void few_route_shared(const FewArgs &a, FewRouting &r, int splits, const float *lpart, uint32_t *row,
                                              int32_t *picks, int32_t *ctr, int tid, volatile int *abort_flag) {
    const int lane = tid & 31, Tk = a.T * a.k;
    if (a.T == 1) {  // one token: every CTA routes it, 1.5 us sooner than reading another's picks
        if (tid < 32) few_route_one(0, a, r, splits, lpart, row, blockIdx.x == 0, lane);
        named_bar_sync(5, kFewRouters);
        return;
    }
    if (tid < 32)
        for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
            few_route_one(t, a, r, splits, lpart, row, true, lane);
            for (int s = lane; s < a.k; s += 32) {
                __stcg(picks + a.T + t * a.k + s, r.idx[t * a.k + s]);
                __stcg(picks + a.T + Tk + t * a.k + s, __float_as_int(r.w[t * a.k + s]));
            }
            if (lane == 0) __stcg(picks + t, r.keff[t]);
            __syncwarp();
            if (lane == 0) add_release(ctr, 1);
        }
    if (tid == 0) grid_wait(a, 2, ctr, a.T, abort_flag);
    named_bar_sync(5, kFewRouters);
    // after a wait that gave up the picks are whatever the scratch held: no index comes
    // from them unchecked
    for (int s = tid; s < Tk; s += kFewRouters) {
        const int e = __ldcg(picks + a.T + s);
        r.idx[s] = (unsigned)e < (unsigned)a.E ? e : -1;
        r.w[s] = __int_as_float(__ldcg(picks + a.T + Tk + s));
    }
    if (tid < a.T) r.keff[tid] = min(max(__ldcg(picks + tid), 0), a.k);
}

// Apply the budget to the routed tokens and list the experts in use: threads
// tid < nthr that meet on barrier `bar`.
__device__ __forceinline__ void few_choose(const FewArgs &a, FewRouting &r, int tid, int nthr, int bar) {
    const int lane = tid & 31, Tk = a.T * a.k;
    auto sync = [&] { named_bar_sync(bar, nthr); };
    auto list = [&] {  // the experts with tokens, ascending
        if (tid < 32) {
            int n = 0;
            for (int e0 = 0; e0 < a.E; e0 += 32) {
                const bool in = e0 + lane < a.E && r.mask[e0 + lane] != 0;
                const unsigned b = __ballot_sync(0xffffffffu, in);
                if (in) r.list[n + __popc(b & ((1u << lane) - 1u))] = (uint16_t)(e0 + lane);
                n += __popc(b);
            }
            if (lane == 0) r.nu = n;
        }
        sync();
    };
    for (int e = tid; e < a.E; e += nthr) r.mask[e] = 0;
    sync();
    for (int s = tid; s < Tk; s += nthr)
        if (r.idx[s] >= 0 && r.idx[s] < a.E) atomicOr(&r.mask[r.idx[s]], 1u << (s / a.k));
    sync();
    list();
    const int nu = r.nu;
    if (a.budget > 0 && nu > a.budget) {
        // the sum of the weights routed to each expert, tokens then slots ascending
        for (int u = tid; u < nu; u += nthr) {
            const int e = r.list[u];
            float s = 0.f;
#pragma unroll 4
            for (int i = 0; i < Tk; ++i) s += r.idx[i] == e ? r.w[i] : 0.f;
            r.agg[u] = s;
        }
        sync();
        // rank in (sum descending, id ascending); the others leave
        for (int u = tid; u < nu; u += nthr) {
            int rank = 0;
            const float mine = r.agg[u];
#pragma unroll 4
            for (int o = 0; o < nu; ++o) {
                const float other = r.agg[o];
                rank += (other > mine) | ((other == mine) & (o < u));
            }
            if (rank >= a.budget) r.mask[r.list[u]] = 0;
        }
        sync();
        for (int t = tid >> 5; t < a.T; t += nthr >> 5) {  // a warp per token: the kept picks move up
            const int valid = r.keff[t];
            const int e = lane < valid ? r.idx[t * a.k + lane] : 0;
            float w = lane < valid ? r.w[t * a.k + lane] : 0.f;
            const unsigned kept = __ballot_sync(0xffffffffu, lane < valid && e >= 0 && r.mask[e] != 0);
            const int c = __popc(kept), at = __popc(kept & ((1u << lane) - 1u));
            if (a.norm_topk && c > 0 && c < valid) {
                float sum = 0.f;  // in slot order
                for (unsigned m = kept; m; m &= m - 1) sum += __shfl_sync(0xffffffffu, w, __ffs(m) - 1);
                w = w / sum;
            }
            if (kept >> lane & 1u) {
                r.idx[t * a.k + at] = e;
                r.w[t * a.k + at] = w;
            }
            if (lane >= c && lane < a.k) {
                r.idx[t * a.k + lane] = -1;
                r.w[t * a.k + lane] = 0.f;
            }
            if (lane == 0) r.keff[t] = c;
        }
        list();
    }
    if (blockIdx.x == 0) {  // the routing's optional outputs
        for (int s = tid; s < Tk; s += nthr) {
            if (a.idx) a.idx[s] = r.idx[s];
            if (a.w) a.w[s] = r.w[s];
        }
        for (int t = tid; t < a.T; t += nthr)
            if (a.keff) a.keff[t] = r.keff[t];
        if (a.budget > 0 && a.kept)
            for (int e = tid; e < a.E; e += nthr) a.kept[e] = r.mask[e] != 0;
        if (a.budget > 0 && a.n_dropped && tid == 0) *a.n_dropped = nu - r.nu;
    }
}

__device__ __forceinline__ float few_weight(const FewArgs &a, const FewRouting &r, int t, int e) {
    for (int j = 0; j < r.keff[t]; ++j)
        if (r.idx[t * a.k + j] == e) return r.w[t * a.k + j];
    return 0.f;
}


// ------------------------------------------------------------- the stream --
// A step is two chunks of the K axis (one at the end of an odd count): 128
// weight rows of 2 kK columns, their block scales, and the same columns of up to
// 2 Tp token rows.  A ring slot holds one step:
//   weights [half][chunk][64 rows][kRowBytes] (halves: gate and up, or the two
//   64-row halves of the down projection), scales [half][chunk][64][per],
//   tokens [64-column box][rows][128 bytes].
template <int FMT, int NT>
struct FewShape {
    static constexpr int kTp = 8 * NT;               // token rows (T rounded up)
    static constexpr int kK = FMT == 0 ? 64 : 128;   // K columns per chunk
    static constexpr int kRowBytes = FMT == 2 ? 64 : 128;
    static constexpr int kChunkBytes = 64 * kRowBytes;
    static constexpr int kWBytes = 4 * kChunkBytes;
    static constexpr int kRun = FMT == 0 ? 0 : FMT == 1 ? 256 : 512;  // block scales of 64 rows and one chunk
    static constexpr int kScaleBytes = 4 * kRun;
    static constexpr int kBoxes = kK / 64;           // 64-column token boxes per chunk
    static constexpr int kXBytes = 2 * kBoxes * kTp * 128;
    static constexpr int kTokOff = kWBytes + (kScaleBytes + 1023) / 1024 * 1024;
    static constexpr int kSlotBytes = kTokOff + 2 * kXBytes;
    static constexpr int kPartFloats = 256 * NT * 4;  // one row block's sums: 8 tiles of 16 rows x 32 lanes
    static constexpr int kXchFloats = kFewGroups * kPartFloats > 16 * 128 ? kFewGroups * kPartFloats : 16 * 128;
    static constexpr int kRowFloats = kFewRowWords;
    static constexpr int kFixed = 1024 + (int)sizeof(FewRouting) + (kXchFloats + kRowFloats) * 4 + 1024;
    static constexpr int kSlots = (kFewSmem - kFixed) / kSlotBytes;
    static constexpr int kSmem = kFixed + kSlots * kSlotBytes;
};

struct __align__(64) FewMaps {
    CUtensorMap gate, up, down, s_gate, s_up, s_down, x, h;
};

// Left shifts as factors (see the decoders below).
struct FewShifts {
    uint32_t by2, by4, by6, by8, by12;  // 1 << 2, ...
};

struct FewPlan {
    FewArgs a;
    FewShifts shifts;
    float *lpart;  // [kFewMaxSplits][T, E] partial logits
    int32_t *picks;  // [T] kept counts, [T k] experts, [T k] weights
    uint16_t *h;   // [2 Tp, ldh] bf16: h, then its remainder
    int ldh;
    float *part;   // [2][kFewMaxSms][2] row-block partials: the down projection's lie over the
                   // shared expert's, which the grid barrier has seen added up
    int32_t *sync; // [0], [1] grid barriers, [2] CTAs done, [3] tokens routed, [16 + phase * kFewMaxSms + cta] partial arrivals
};

// This CTA's share of a phase: steps [lo, hi) of `total`, `per` to a row block.
// Whole row blocks where that keeps no CTA busier than equal shares do by more
// than the 3 us that adding partials takes, about five steps.
constexpr int kFewSplitSteps = 5;
struct Share {
    int per, total, ctas, lo, hi;
    __device__ Share(int units, int per_unit) : per(per_unit), total(units * per_unit) {
        ctas = min((int)gridDim.x, total);
        lo = hi = 0;
        const int most = (units + (int)gridDim.x - 1) / (int)gridDim.x;  // whole units for the busiest CTA
        if (most * per <= total / (int)gridDim.x + kFewSplitSteps) {
            lo = min(units, (int)blockIdx.x * most) * per;
            hi = min(units, ((int)blockIdx.x + 1) * most) * per;
            return;
        }
        if ((int)blockIdx.x < ctas) {
            lo = (int)((long long)blockIdx.x * total / ctas);
            hi = (int)((long long)(blockIdx.x + 1) * total / ctas);
        }
    }
    // the CTA whose share holds step c
    __device__ int owner(int c) const { return (int)(((long long)(c + 1) * ctas - 1) / total); }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void lds64(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(d) : "r"(a), "r"(sel));
    return d;
}

// Sixteen codes of one row as bf16 pairs times their block's scale, exactly.
//
// E4M3: the code's sign, exponent and mantissa moved to a bf16's fields are
// the value times 2^-120 (subnormals included), so one bf16 product with
// 2^(120 + se) finishes it; codes (2i, 2i + 1) of word j give pair 2j + i.
// That factor is a bf16 while se <= 7 (weights below 2^16); a warp that meets a
// larger scale multiplies twice.
__device__ __forceinline__ void decode16_mx(uint32_t (&v)[8], const uint32_t (&c)[4], uint32_t scale, uint32_t by4) {
    const uint32_t f = (scale + 120u) * 0x00800080u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x = prmt(c[j], i ? 0xB3A2u : 0x9180u);  // a code and its sign, eight times, in each half
            v[2 * j + i] = mul_bf16x2((x * by4) & 0x87F087F0u, f);
        }
}
// E2M1: likewise the value times 2^-126; the factor holds the E4M3 block scale
// (not negative) times 2^118 -- the code's bits in a bf16's fields are s 2^-120,
// two products with 2^119 make the rest -- and the missing 2^8 goes to the matrix
// scale.  Word j's pairs are codes (i, i + 4), i = 0..3.  The integer pipe paces
// the decoding, so the shifts to the left are multiplications, on the other pipe;
// by parameters, as constants would be made shifts again.
constexpr float kNvFix = 256.f;
__device__ __forceinline__ void decode16_nv(uint32_t (&v)[8], const uint32_t (&c)[2], uint32_t scale, const FewShifts &sh) {
    constexpr uint32_t c119 = ((127u + 119u) << 7) * 0x00010001u;
    const uint32_t f = mul_bf16x2(mul_bf16x2(scale * 0x00100010u, c119), c119);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t w = c[j], w8 = w >> 8;
        const uint32_t mag[4] = {w * sh.by6, w * sh.by2, w8 * sh.by6, w8 * sh.by2};
        const uint32_t sgn[4] = {w * sh.by12, w * sh.by8, w * sh.by4, w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[4 * j + i] = mul_bf16x2((mag[i] & 0x01C001C0u) | (sgn[i] & 0x80008000u), f);
    }
}

// One warp's share of a step: 32 weight rows (tiles 2 rg and 2 rg + 1) times a
// half of chunk `sub`, 32 columns in bf16 and 64 block-scaled ones.  kDown: the
// tiles are 16 consecutive rows and the token operand is h and its remainder;
// otherwise a tile is 8 gate rows and the 8 up rows of the same channels.
template <int FMT, int NT, bool kDown>
__device__ __forceinline__ void few_step(float (&acc)[2][NT][4], uint32_t slot, int rg, int sub, int half, int lane,
                                         const FewShifts &sh) {
    using S = FewShape<FMT, NT>;
    constexpr int kParts = kDown ? 2 : 1, kBoxBytes = kParts * S::kTp * 128;
    const int g = lane >> 2, q = lane & 3;
    const uint32_t tb = slot + S::kTokOff;
    // the tile's rows 0..7 and 8..15: a half of the step's 128 rows, and a row of it
    auto row = [&](int m, int hi, int &h) -> uint32_t {
        const int tile = rg * 2 + m, rr = kDown ? tile * 16 + hi * 8 : hi * 64 + tile * 8;
        h = rr >> 6;
        return (uint32_t)(rr & 63);
    };
    if constexpr (FMT == 0) {
        const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int ks = half * 2 + s;  // of the chunk's four K16 steps
            uint32_t A[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                int h;
                const uint32_t rr = row(m, mi & 1, h) + lr;
                ldsm4(A[m], slot + (h * 2 + sub) * S::kChunkBytes + rr * 128 + (((2 * ks + (mi >> 1)) ^ lr) << 4));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t B[4];  // matrices 0, 1: x or h; 2, 3: the remainder
                const uint32_t tr = n * 8 + lr + (kDown && mi >= 2 ? S::kTp : 0);
                ldsm4(B, tb + sub * kBoxBytes + tr * 128 + (((2 * ks + (mi & 1)) ^ lr) << 4));
#pragma unroll
                for (int m = 0; m < 2; ++m) mma16816(acc[m][n], A[m][0], A[m][1], A[m][2], A[m][3], B[0], B[1]);
                if constexpr (kDown) {
#pragma unroll
                    for (int m = 0; m < 2; ++m) mma16816(acc[m][n], A[m][0], A[m][1], A[m][2], A[m][3], B[2], B[3]);
                }
            }
        }
    } else {
        // lane (g, q) takes 16 codes of rows g and g + 8 of each tile (one block scale
        // each) and the same 16 token columns
        uint32_t v[2][2][8];
        uint32_t c[2][2][FMT == 1 ? 4 : 2], sc[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                int h;
                const uint32_t rr = row(m, hi, h) + g;
                const uint32_t wb = slot + (h * 2 + sub) * S::kChunkBytes, sb = slot + S::kWBytes + (h * 2 + sub) * S::kRun;
                if constexpr (FMT == 1) {
                    lds128(c[m][hi], wb + rr * 128 + (((half * 4 + q) ^ (rr & 7)) << 4));
                    sc[m][hi] = lds8(sb + rr * 4 + half * 2 + (q >> 1));
                } else {
                    lds64(c[m][hi], wb + rr * 64 + (((half * 2 + (q >> 1)) ^ ((rr >> 1) & 3)) << 4) + (q & 1) * 8);
                    sc[m][hi] = lds8(sb + rr * 8 + half * 4 + q);
                }
            }
        if constexpr (FMT == 1) {
            if (__any_sync(0xffffffffu, max(max(sc[0][0], sc[0][1]), max(sc[1][0], sc[1][1])) > 134u)) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) {
                        const uint32_t low = min(sc[m][hi], 134u), rest = (sc[m][hi] - low + 127u) * 0x00800080u;
                        decode16_mx(v[m][hi], c[m][hi], low, sh.by4);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[m][hi][i] = mul_bf16x2(v[m][hi][i], rest);
                    }
            } else {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) decode16_mx(v[m][hi], c[m][hi], sc[m][hi], sh.by4);
            }
        } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) decode16_nv(v[m][hi], c[m][hi], sc[m][hi], sh);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                const uint32_t tr = tb + (sub * 2 + half) * kBoxBytes + (part * S::kTp + n * 8 + g) * 128;
                uint32_t b[8];
                lds128(reinterpret_cast<uint32_t(&)[4]>(b[0]), tr + (((2 * q) ^ g) << 4));
                lds128(reinterpret_cast<uint32_t(&)[4]>(b[4]), tr + (((2 * q + 1) ^ g) << 4));
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t b0 = b[2 * s], b1 = b[2 * s + 1];
                    if constexpr (FMT == 2 && !kDown) {  // the columns in the codes' pair order (h is stored in it)
                        const uint32_t lo = b[(s >> 1) * 4 + (s & 1)], hi = b[(s >> 1) * 4 + (s & 1) + 2];
                        b0 = __byte_perm(lo, hi, 0x5410);
                        b1 = __byte_perm(lo, hi, 0x7632);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        mma16816(acc[m][n], v[m][0][2 * s], v[m][1][2 * s], v[m][0][2 * s + 1], v[m][1][2 * s + 1], b0, b1);
                }
            }
    }
}

template <int FMT, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewMaps maps,
                                                             const __grid_constant__ FewPlan p) {
    using S = FewShape<FMT, NT>;
    constexpr int kTp = S::kTp, kSlots = S::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *xch = reinterpret_cast<float *>(ring + (size_t)kSlots * S::kSlotBytes);  // the groups' sums; the projection's
    FewRouting &r = *reinterpret_cast<FewRouting *>(xch + S::kXchFloats + S::kRowFloats);
    uint64_t *full = reinterpret_cast<uint64_t *>((reinterpret_cast<uintptr_t>(&r + 1) + 7) & ~uintptr_t(7));
    uint64_t *empty = full + kSlots, *routed = empty + kSlots;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(routed + 1);
    volatile int *last_flag = abort_flag + 1;
    const FewArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&full[s], 2);  // the two producers
            mbar_init(&empty[s], kFewConsumers / 32);
        }
        mbar_init(routed, 1);
        r.nu = 0;
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();

    const int kH = a.H / S::kK, kS = a.Is / S::kK, kI = a.I / S::kK;  // chunks along H, Is, I
    const int sH = (kH + 1) >> 1, sS = (kS + 1) >> 1, sI = (kI + 1) >> 1;  // steps
    // the three phases' shares; the routed ones are known once the tokens are routed
    auto share = [&](int phase) {
        return phase == 0 ? Share(a.Is / 64, sH) : phase == 1 ? Share(r.nu * (a.I / 64), sH)
                                                              : Share(a.H / 128, sS + r.nu * sI);
    };

    auto drain = [&](uint32_t issued) {  // a producer's copies in flight
        unsigned long long until = 0;
        for (uint32_t n = issued > (uint32_t)kSlots ? issued - kSlots : 0; n < issued; ++n)
            until = mbar_drain(&full[n % kSlots], (n / kSlots) & 1u, abort_flag, a.status, until);
    };
    if (warp == kFewConsumers / 32) {
        // ================= weight producer =================
        if (lane < 8) prefetch_tmap(&maps.gate + lane);  // all eight: a first use costs a microsecond otherwise
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            uint32_t st = 0, ph = 0, issued = 0;
            bool ok = true;
            // one step: chunks kcol .. kcol + n - 1 of rows y0 .. + 63 and y1 .. + 63
            auto load = [&](const CUtensorMap *m0, const CUtensorMap *m1, const uint8_t *f0, const uint8_t *f1, int y0,
                            int y1, int kcol, int cols) {
                if (issued >= (uint32_t)kSlots && !mbar_wait_fast(&empty[st], ph ^ 1u, abort_flag, a.status, true)) {
                    ok = false;
                    return;
                }
                uint8_t *dst = ring + (size_t)st * S::kSlotBytes;
                const uint32_t run = S::kRun * (uint32_t)min(2, cols - kcol);
                mbar_arrive_expect_tx(&full[st], S::kWBytes + 2 * run);
                tma_load_3d_hint(m0, &full[st], dst, 0, y0, kcol, pol);
                tma_load_3d_hint(m1, &full[st], dst + S::kWBytes / 2, 0, y1, kcol, pol);
                if constexpr (FMT != 0) {
                    bulk_load(dst + S::kWBytes, f0 + ((size_t)(y0 >> 6) * cols + kcol) * S::kRun, run, &full[st]);
                    bulk_load(dst + S::kWBytes + 2 * S::kRun, f1 + ((size_t)(y1 >> 6) * cols + kcol) * S::kRun, run,
                              &full[st]);
                }
                ++issued;
                if (++st == (uint32_t)kSlots) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            for (int phase = 0; ok && phase < 3; ++phase) {
                if (phase == 1 && !mbar_wait(routed, 0, abort_flag, a.status, true)) break;
                const Share sh = share(phase);
                int unit = sh.lo / max(sh.per, 1), at = sh.lo - unit * sh.per;
                for (int left = sh.hi - sh.lo; ok && left > 0; ++unit, at = 0) {
                    const int end = min(sh.per, at + left);
                    left -= end - at;
                    if (phase < 2) {
                        const int per = a.I / 64;
                        const int y = phase ? r.list[unit / per] * a.I + unit % per * 64 : unit * 64;
                        const CUtensorMap *m0 = phase ? &maps.gate : &maps.s_gate, *m1 = phase ? &maps.up : &maps.s_up;
                        const uint8_t *f0 = phase ? a.gate.sf : a.s_gate.sf, *f1 = phase ? a.up.sf : a.s_up.sf;
                        for (; ok && at < end; ++at) load(m0, m1, f0, f1, y, y, 2 * at, kH);
                    } else {
                        const int y = unit * 128;
                        for (; ok && at < min(end, sS); ++at)
                            load(&maps.s_down, &maps.s_down, a.s_down.sf, a.s_down.sf, y, y + 64, 2 * at, kS);
                        int u = (at - sS) / sI, in = (at - sS) - u * sI;
                        for (; ok && at < end; ++u, in = 0) {
                            const int ye = y + r.list[u] * a.H;
                            for (; ok && in < sI && at < end; ++in, ++at)
                                load(&maps.down, &maps.down, a.down.sf, a.down.sf, ye, ye + 64, 2 * in, kI);
                        }
                    }
                }
            }
            drain(issued);
        }
    } else if (warp == kFewConsumers / 32 + 1) {
        // ================= token producer =================
        if (lane == 0) {
            uint32_t st = 0, ph = 0, issued = 0;
            bool ok = true;
            for (int phase = 0; ok && phase < 3; ++phase) {
                if (phase == 1 && !mbar_wait(routed, 0, abort_flag, a.status, true)) break;
                const Share sh = share(phase);
                if (phase == 2) {
                    if (!grid_wait(a, 1, p.sync + 1, (int)gridDim.x, abort_flag)) break;
                    fence_proxy_async_global();  // h was written by ordinary stores
                }
                const CUtensorMap *map = phase == 2 ? &maps.h : &maps.x;
                const uint32_t bytes = phase == 2 ? 2 * S::kXBytes : S::kXBytes;
                int at = sh.lo % max(sh.per, 1);
                for (int c = sh.lo; ok && c < sh.hi; ++c) {
                    if (issued >= (uint32_t)kSlots && !mbar_wait_fast(&empty[st], ph ^ 1u, abort_flag, a.status, true)) {
                        ok = false;
                        break;
                    }
                    int chunk = 2 * at;
                    if (phase == 2 && at >= sS) {  // the routed channels lie behind the shared ones
                        const int u = (at - sS) / sI;
                        chunk = kS + u * kI + 2 * (at - sS - u * sI);
                    }
                    mbar_arrive_expect_tx(&full[st], bytes);
                    tma_load_3d_hint(map, &full[st], ring + (size_t)st * S::kSlotBytes + S::kTokOff, 0, 0,
                                     chunk * S::kBoxes, policy_evict_normal());
                    ++issued;
                    if (++st == (uint32_t)kSlots) {
                        st = 0;
                        ph ^= 1u;
                    }
                    if (++at == sh.per) at = 0;
                }
            }
            drain(issued);
        }
    } else if (warp >= kFewConsumers / 32 + 2) {
        // ================= routers =================
        // With a shared expert, the wait for everyone's logits and the routing hide
        // behind its gate/up stream: each token is routed by one CTA of the grid, and
        // all read the picks.  Without one the consumers, idle till then, route every
        // token in every CTA: 16 warps, a token each, and one grid barrier less.
        if (a.Is > 0) {
            const int tid = threadIdx.x - kFewConsumers - 64;
            if (a.project && tid == 0) grid_wait(a, 0, p.sync, (int)gridDim.x, abort_flag);
            named_bar_sync(5, kFewRouters);
            few_route_shared(a, r, a.project ? few_splits(a) : 1, p.lpart,
                             reinterpret_cast<uint32_t *>(xch + S::kXchFloats), p.picks,
                             p.sync + 3, tid, abort_flag);
            few_choose(a, r, tid, kFewRouters, 5);
            if (tid == 0) mbar_arrive(routed);
        }
    } else {
        // ================= consumers =================
        const int tid = threadIdx.x;
        // the shared expert's gate, one token per CTA from the grid's end
        const int gt = (int)gridDim.x - 1 - cta;
        if (a.Is > 0)
            for (int t = gt; t < a.T; t += gridDim.x) {
                float z = 0.f;
                for (int i = tid; i < a.H / 8; i += kFewConsumers) {
                    const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.H) + i);
                    const uint4 gv = __ldg(reinterpret_cast<const uint4 *>(a.gvec) + i);
                    const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, gs[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        z = fmaf(__uint_as_float(xs[q] << 16), __uint_as_float(gs[q] << 16), z);
                        z = fmaf(__uint_as_float(xs[q] & 0xffff0000u), __uint_as_float(gs[q] & 0xffff0000u), z);
                    }
                }
#pragma unroll
                for (int off = 16; off; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
                if (lane == 0) xch[warp] = z;
                consumers_sync();
                if (tid == 0) {
                    z = 0.f;
                    for (int w = 0; w < kFewConsumers / 32; ++w) z += xch[w];
                    a.sgate[t] = 1.f / (1.f + expf(-z));
                }
                consumers_sync();
            }
        const int splits = a.project ? few_splits(a) : 1;
        if (a.project) {
            // logits: eight experts (the mma's columns) and a K split per CTA, tokens its
            // rows, the warps on alternate 64-wide K blocks; lane (g, q) holds 16
            // consecutive columns 16 q of rows g and g + 8, the same permutation of K on
            // both sides
            const int g = lane >> 2, q = lane & 3, groups = (a.E + 7) / 8;
            for (int item = cta; item < groups * splits; item += gridDim.x) {
                const int o = item % groups, sp = item / groups;
                const int kb0 = a.H / 64 * sp / splits, kb1 = a.H / 64 * (sp + 1) / splits;
                const uint16_t *x0 = a.x + (size_t)min(g, a.T - 1) * a.H, *x1 = a.x + (size_t)min(g + 8, a.T - 1) * a.H;
                const uint16_t *w0 = a.w_router + (size_t)min(o * 8 + g, a.E - 1) * a.H;
                float d[4] = {};
#pragma unroll 3
                for (int kb = kb0 + warp; kb < kb1; kb += kFewConsumers / 32) {
                    const int k = kb * 64 + q * 16;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(x0 + k) + i);
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);  // tokens 8 .. 15
                        if (NT > 1) v = __ldg(reinterpret_cast<const uint4 *>(x1 + k) + i);
                        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(w0 + k) + i);
                        mma16816(d, u.x, v.x, u.y, v.y, w.x, w.y);
                        mma16816(d, u.z, v.z, u.w, v.w, w.z, w.w);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) xch[warp * 128 + (g + 8 * (i >> 1)) * 8 + 2 * q + (i & 1)] = d[i];
                consumers_sync();
                if (tid < 128) {
                    float v = 0.f;
                    for (int w = 0; w < kFewConsumers / 32; ++w) v += xch[w * 128 + tid];
                    const int t = tid >> 3, e = o * 8 + (tid & 7);
                    float *dst = splits > 1 ? p.lpart + (size_t)sp * a.T * a.E : a.logits;
                    if (t < a.T && e < a.E) dst[(size_t)t * a.E + e] = v;
                }
                consumers_sync();
            }
            if (tid == 0) grid_arrive(p.sync);
        }
        if (a.Is == 0) {
            if (a.project) {
                if (tid == 0) grid_wait(a, 0, p.sync, (int)gridDim.x, abort_flag);
                consumers_sync();
            }
            // in the ring, which is empty till the routed experts are known
            few_route_all(a, r, splits, p.lpart, reinterpret_cast<uint32_t *>(ring), warp, lane);
            fence_proxy_async_shared();
            consumers_sync();
            few_choose(a, r, tid, kFewConsumers, 1);
            if (tid == 0) mbar_arrive(routed);
        }

        const int grp = warp >> 2, rg = warp & 3, g = lane >> 2, q = lane & 3;
        const int sub = grp >> 1, half = grp & 1;  // this group's columns: a half of a chunk of the step
        bool dead = false;  // a wait for the ring gave up: go through the motions to the end
        uint32_t st = 0, ph = 0;
        float sg[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) sg[n][0] = sg[n][1] = 0.f;
        for (int phase = 0; phase < 3; ++phase) {
            // The routing is read from here on, by every warp, abort or not: the named barriers
            // below want all of them.  The routers arrive whatever happened, after two bounded
            // waits at most; hence three rounds of the limit here.  (One thread's wait and a
            // barrier instead, with a way out for all, cost 2 us of 77 at 14 NVFP4 tokens.)
            if (phase == 1 && a.Is > 0)
                for (int i = 0; i < 3 && !mbar_wait(routed, 0, abort_flag, a.status, false); ++i) {
                }
            const Share sh = share(phase);
            int unit = sh.lo / max(sh.per, 1), at = sh.lo - unit * sh.per, left = sh.hi - sh.lo;
            bool have_sg = false;
            while (left > 0) {
                const int n_steps = min(sh.per - at, left);
                float acc[2][NT][4] = {};  // two tiles of 16 rows x 8 NT tokens
                // one step; the second chunk of an odd K range's last one is not there
                auto take = [&](auto down, bool live) {
                    if (!dead) dead = !mbar_wait_fast(&full[st], ph, abort_flag, a.status, true);
                    if (live)
                        few_step<FMT, NT, decltype(down)::value>(acc, smem_u32(ring + (size_t)st * S::kSlotBytes), rg, sub, half,
                                                                 lane, p.shifts);
                    __syncwarp();
                    if (lane == 0 && !dead) mbar_arrive(&empty[st]);  // (a slot that never filled is not free)
                    if (++st == (uint32_t)kSlots) {
                        st = 0;
                        ph ^= 1u;
                    }
                };
                if (phase < 2) {
                    const int cut = sub & kH ? sH - 1 : sH;  // (sub is 0 or 1)
                    for (int i = at; i < at + n_steps; ++i) take(std::false_type(), i != cut);
                } else {
                    int i = at;
                    const int end = at + n_steps, cut = sub & kS ? sS - 1 : sS;
                    for (; i < min(end, sS); ++i) take(std::true_type(), i != cut);
                    if (i > at) {
                        // the shared expert's channels come first: their sum takes the gate before the
                        // routed ones join.  The token operand is past the grid barrier: so are the gates
                        if (!have_sg)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const int t = n * 8 + 2 * q + c;
                                    sg[n][c] = t < a.T ? __ldcg(a.sgate + t) : 0.f;
                                }
                        have_sg = true;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                acc[m][n][0] *= sg[n][0];
                                acc[m][n][1] *= sg[n][1];
                                acc[m][n][2] *= sg[n][0];
                                acc[m][n][3] *= sg[n][1];
                            }
                    }
                    int in = (i - sS) % sI;
                    const int last_in = sub & kI ? sI - 1 : sI;
                    for (; i < end; ++i) {
                        take(std::true_type(), in != last_in);
                        if (++in == sI) in = 0;
                    }
                }
                // the groups' sums
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        *reinterpret_cast<float4 *>(xch + (((grp * NT + n) * 8 + rg * 2 + m) * 32 + lane) * 4) =
                            make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
                named_bar_sync(2, kFewConsumers);
                float sum[NT][4] = {};
                if (warp < 8) {  // tile `warp` of the row block
#pragma unroll
                    for (int k = 0; k < kFewGroups; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float4 o =
                                *reinterpret_cast<const float4 *>(xch + (((k * NT + n) * 8 + warp) * 32 + lane) * 4);
                            sum[n][0] += o.x;
                            sum[n][1] += o.y;
                            sum[n][2] += o.z;
                            sum[n][3] += o.w;
                        }
                }
                named_bar_sync(3, kFewConsumers);
                if (warp < 8) {
                    const int wr = warp;
                    bool whole = n_steps == sh.per;
                    if (!whole) {
                        // a row block shared with other CTAs: the last to arrive adds the partials
                        const int first = sh.owner(unit * sh.per), last = sh.owner(unit * sh.per + sh.per - 1);
                        auto slot = [&](int c) {
                            return reinterpret_cast<float4 *>(
                                       p.part + (size_t)(((phase & 1) * kFewMaxSms + c) * 2 + (c == first)) * S::kPartFloats) +
                                   wr * 32 + lane;
                        };
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            __stcg(slot(cta) + n * 256, make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]));
                        named_bar_sync(4, 256);
                        if (tid == 0) {
                            int32_t *ctr = p.sync + 16 + phase * kFewMaxSms + first;
                            const bool is_last = (int)add_acq_rel(reinterpret_cast<uint32_t *>(ctr), 1u) == last - first;
                            if (is_last) *ctr = 0;
                            *last_flag = is_last;
                        }
                        named_bar_sync(4, 256);
                        whole = *last_flag != 0;
                        if (whole) {
#pragma unroll
                            for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.f;
                            for (int c0 = first; c0 <= last; c0 += 4) {  // four in flight, added in order
                                float4 o[4][NT];
#pragma unroll
                                for (int c = 0; c < 4; ++c)
#pragma unroll
                                    for (int n = 0; n < NT; ++n) o[c][n] = __ldcg(slot(min(c0 + c, last)) + n * 256);
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (c0 + c <= last)
#pragma unroll
                                        for (int n = 0; n < NT; ++n) {
                                            sum[n][0] += o[c][n].x;
                                            sum[n][1] += o[c][n].y;
                                            sum[n][2] += o[c][n].z;
                                            sum[n][3] += o[c][n].w;
                                        }
                            }
                        }
                    }
                    if (whole && phase < 2) {
                        // gate (rows 0..7) and up (8..15) of one channel are in one thread
                        const int per = a.I / 64, u = phase ? unit / per : 0, e = phase ? r.list[u] : 0;
                        // NVFP4: in the order of the down projection's code pairs, 0 4 1 5 2 6 3 7
                        const int at8 = FMT == 2 ? (g & 3) * 2 + (g >> 2) : g;
                        const int ch = (phase ? unit % per : unit) * 64 + wr * 8 + at8;
                        const uint32_t tokens = phase ? r.mask[e] : (1u << a.T) - 1u;
                        uint16_t *dst = p.h + (phase ? a.Is + (size_t)u * a.I : 0) + ch;
                        float tg = 1.f, tu = 1.f, td = 1.f;
                        if constexpr (FMT == 2) {
                            tg = kNvFix * __ldg((phase ? a.gate.ts : a.s_gate.ts) + e);
                            tu = kNvFix * __ldg((phase ? a.up.ts : a.s_up.ts) + e);
                            td = kNvFix * __ldg((phase ? a.down.ts : a.s_down.ts) + e);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int t = n * 8 + 2 * q + c;
                                float v = 0.f;
                                if ((tokens >> t) & 1u) {
                                    const float gv = sum[n][c] * tg;
                                    v = gv / (1.f + expf(-gv)) * (sum[n][2 + c] * tu) * td;
                                    if (phase) v *= few_weight(a, r, t, e);
                                }
                                const uint16_t hi = f32_to_bf16_bits(v);
                                const float rem = v - bf16_bits_to_f32(hi);
                                dst[(size_t)t * p.ldh] = hi;
                                // an infinite or NaN h has no remainder
                                dst[(size_t)(kTp + t) * p.ldh] = f32_to_bf16_bits(fabsf(rem) < INFINITY ? rem : 0.f);
                            }
                    } else if (whole) {
                        const int o = unit * 128 + wr * 16 + g;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int t = n * 8 + 2 * q + (c & 1);
                                if (t < a.T) a.out[(size_t)t * a.H + o + (c >> 1) * 8] = f32_to_bf16_bits(sum[n][c]);
                            }
                    }
                }
                left -= n_steps;
                at = 0;
                ++unit;
            }
            if (phase == 1 && warp < 8) {  // this CTA's part of h is written
                named_bar_sync(4, 256);
                if (tid == 0) grid_arrive(p.sync + 1);
            }
        }
    }
    // the last CTA out leaves the barriers at zero
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.sync + 2, 1) == (int)gridDim.x - 1) {
        p.sync[0] = 0;
        p.sync[1] = 0;
        p.sync[2] = 0;
        p.sync[3] = 0;
    }
}

size_t part_bytes(int tp) { return (size_t)2 * kFewMaxSms * 2 * 128 * tp * 4; }
size_t lpart_bytes(int T, int E) { return (size_t)kFewMaxSplits * T * E * 4; }
size_t picks_bytes(int T, int k) { return (size_t)T * (2 * k + 1) * 4; }
size_t route_bytes(int T, int E, int k) { return (lpart_bytes(T, E) + picks_bytes(T, k) + 255) / 256 * 256; }
int few_ldh(int T, int E, int I, int k, int Is) { return Is + std::min(E, T * k) * I; }
int few_tp(int T) { return T <= 8 ? 8 : 16; }

// Weights [rows, K] as [K / chunk][rows][chunk bytes]: a box of 64 rows and two chunks.
template <int FMT>
bool encode_weights(CUtensorMap *m, const void *base, uint64_t rows, uint64_t K) {
    return encode_3d(m, base, rows, FMT == 0 ? 2 * K : FMT == 1 ? K : K / 2, FMT == 2 ? 64 : 128, 64, 2);
}

template <int FMT, int NT>
cudaError_t launch_shape(const FewArgs &a, cudaStream_t st) {
    using S = FewShape<FMT, NT>;
    static_assert(S::kSlots >= 3 && S::kSmem <= kFewSmem, "ring");
    static_assert(S::kSlots * S::kSlotBytes >= kFewConsumers / 32 * kFewRowWords * 4, "routing rows in the ring");
    static_assert(S::kSlotBytes % 1024 == 0, "swizzled boxes need 1024-byte aligned slots");
    FewMaps m;
    const uint64_t E = a.E, I = a.I, H = a.H, Is = a.Is;
    FewPlan p;
    p.a = a;
    p.shifts = {1u << 2, 1u << 4, 1u << 6, 1u << 8, 1u << 12};
    p.ldh = few_ldh(a.T, a.E, a.I, a.k, a.Is);
    p.part = static_cast<float *>(a.h);
    p.lpart = reinterpret_cast<float *>(static_cast<uint8_t *>(a.h) + part_bytes(S::kTp));
    p.h = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(a.h) + part_bytes(S::kTp) + route_bytes(a.T, a.E, a.k));
    p.picks = reinterpret_cast<int32_t *>(p.lpart) + lpart_bytes(a.T, a.E) / 4;
    p.sync = a.sync;
    if (!encode_weights<FMT>(&m.gate, a.gate.w, E * I, H) || !encode_weights<FMT>(&m.up, a.up.w, E * I, H) ||
        !encode_weights<FMT>(&m.down, a.down.w, E * H, I) || !encode_3d(&m.x, a.x, a.T, 2 * H, 128, S::kTp, 2 * S::kBoxes) ||
        !encode_3d(&m.h, p.h, 2 * S::kTp, 2 * (uint64_t)p.ldh, 128, 2 * S::kTp, 2 * S::kBoxes))
        return cudaErrorInvalidValue;
    if (Is > 0) {
        if (!encode_weights<FMT>(&m.s_gate, a.s_gate.w, Is, H) || !encode_weights<FMT>(&m.s_up, a.s_up.w, Is, H) ||
            !encode_weights<FMT>(&m.s_down, a.s_down.w, H, Is))
            return cudaErrorInvalidValue;
    } else {
        m.s_gate = m.s_up = m.s_down = m.gate;  // not read
    }
    static std::atomic<int> attr_set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(few_kernel<FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(device_sm_count(), kFewMaxSms));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few_kernel<FMT, NT>, m, p);
}

template <int FMT>
cudaError_t launch_fmt(const FewArgs &a, cudaStream_t st) {
    return a.T <= 8 ? launch_shape<FMT, 1>(a, st) : launch_shape<FMT, 2>(a, st);
}

}  // namespace

size_t few_scratch_bytes(int T, int E, int I, int k, int Is) {
    const int tp = few_tp(T);
    return part_bytes(tp) + route_bytes(T, E, k) + (size_t)2 * tp * few_ldh(T, E, I, k, Is) * 2;
}

cudaError_t launch_few(const FewArgs &a, int fmt, cudaStream_t st) {
    return fmt == 0 ? launch_fmt<0>(a, st) : fmt == 1 ? launch_fmt<1>(a, st) : launch_fmt<2>(a, st);
}

}  // namespace moe
