// The fused linear map out = residual + act(x W^T + bias) on the
// 5th-generation tensor cores: bf16 operands, fp32 sums, one rounding of the
// result (or none, fp32 out).
//
// One kernel from one token to long prompts.  The MMA's M is output channels
// and its N tokens: a tile is 128 rows of W (256 for a CTA pair, 128 in each
// CTA) by Nt tokens, Nt the tokens rounded up to 16 (at most 256 a tile), so
// that a few tokens pay for a few columns and not for a padded row block.  K
// runs in 64-wide slices, both operands TMA-loaded into 128-byte-swizzled
// shared memory; ragged edges are zero-filled by TMA and not stored.  The fp32
// accumulator lives in TMEM, double buffered: a tile's epilogue runs under the
// next one's products.
//
// The tensor cores truncate at every addition to an accumulator, 4 per slice: at
// K = 5120 an fp32 result was 5.5e-6 off, 30 times an fp32 sum's error.  fp32 out
// therefore sums segments of 512 columns in TMEM and the segments in registers,
// rounded to nearest (4.8e-7; segments of 256 columns 2.4e-7, and 74 us would be 86 at
// 1000 x 5120 x 5120); for bf16 out the rounding hides the rest.
//
// Bound: few tokens stream W from HBM (one CTA per SM, single tiles: 7 x 131072 x
// 5120 in 218 us, 6.2 TB/s); from about 200 tokens on the tensor cores bind, and a
// pair halves each CTA's share of the token operand (8191 x 7168 x 7168 in 740 to 755
// us, 1.12 PFLOP/s, under the power cap, 80 us of it the epilogue's).  Pairs against
// single CTAs at 5120 x 17408, us: 38 and 37 at 16 tokens, 39 and 37 at 64, 45 and 46
// at 128, 60 and 71 at 224; hence pairs above 64 tokens.
//
// Tiles go to the grid in whole waves, in bands of 8 row tiles so that a wave's
// operands stay in L2; the tiles that would make up a last, partial wave have
// their K range cut into equal contiguous shares over the whole grid.  Shares of
// a tile leave fp32 partials in the workspace, which are added in share order
// (the same bits on every run) by the warps that are there when all have arrived:
// left to the last one, the adding took 18 us at 224 x 5120 x 17408.
//
// Roles: warps 0 and 1 TMA producers of W and of the tokens (one lane each),
// warp 2 TMEM allocation and MMA issue (one lane), warps 3..10 epilogue (two to
// each TMEM lane quarter, on alternate 32-column blocks), warp 11 the copies of
// the staged epilogue.  A lane holds one output channel, so a warp's direct store
// of one token covers 32 consecutive channels.  Every wait is bounded: past the
// limit the kernel sets MOE_STATUS_TIMEOUT, every role of the CTA or pair stops, and
// what it has under way gets 10 ms to land.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "linear.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {
using namespace tc;

constexpr int kLinEpi = 256;                   // epilogue threads
constexpr int kLinThreads = 96 + kLinEpi + 32;
constexpr int kLinSliceA = 128 * 128;          // 128 rows of W x 64 columns
constexpr int kLinRing = 216 * 1024;           // at most
constexpr int kLinAccStride = 256;             // TMEM columns between the two accumulators
constexpr int kLinSegment = 8;                 // K slices summed in TMEM for fp32 out
constexpr int kLinBand = 8;                    // row tiles of a band
constexpr int kLinMaxStages = 16;
constexpr int kLinStagedSlices = 32;           // staged epilogue up to this many K slices
constexpr int kLinBlockBytes = 32 * 128 * 2;   // staged epilogue: 32 tokens x 128 channels, 8 blocks a tile
constexpr int kLinMaxSplit = 12;               // shares of a tile, and two for unaligned ends
constexpr unsigned long long kLinLingerNs = 30000;  // wait for a tile's other shares to help adding them

struct __align__(64) LinMaps {
    CUtensorMap w;  // [N, K], box 64 x 128
    CUtensorMap x;  // [T, K], box 64 x Nt (pair: Nt / 2)
    CUtensorMap r, r16;  // residual [T, N], box 128 x 32 and 128 x 16 (staged epilogue)
    CUtensorMap o, o16;  // out [T, N], the same
};

struct LinPlan {
    LinearArgs a;
    int Nt, nk;         // tokens of a tile (the MMA's N), K slices
    int rt, tt;         // row tiles, token tiles
    int waves;          // whole waves of tiles
    int rest, sharers;  // tiles left, workers that share their K slices (== rest: a tile each)
    int stages;
    int staged;         // whole tiles' residual and output pass through shared memory
};

// The tiles of worker w (a CTA or a pair): its tile of every wave, then its share of the rest.
struct LinWalk {
    int w, workers, nk, waves, i, lo, hi, base;
    __device__ LinWalk(const LinPlan &p, int worker, int n) : w(worker), workers(n), nk(p.nk), waves(p.waves), i(0) {
        base = waves * workers;
        lo = hi = 0;
        if (w < p.sharers) {
            const long long total = (long long)p.rest * nk;
            lo = (int)(w * total / p.sharers);
            hi = (int)((w + 1) * total / p.sharers);
        }
    }
    __device__ bool next(int &tile, int &k0, int &k1) {
        if (i < waves) {
            tile = i * workers + w;
            k0 = 0;
            k1 = nk;
            ++i;
            return true;
        }
        if (lo >= hi) return false;
        const int t = lo / nk;
        tile = base + t;
        k0 = lo - t * nk;
        k1 = min(nk, k0 + hi - lo);
        lo += k1 - k0;
        return true;
    }
    __device__ bool finished() const { return i >= waves && lo >= hi; }
};

__device__ __forceinline__ void lin_tile(const LinPlan &p, int tile, int &r, int &j) {
    const int band = tile / (kLinBand * p.tt), in = tile - band * kLinBand * p.tt;
    const int rows = min(kLinBand, p.rt - band * kLinBand);
    j = in / rows;
    r = band * kLinBand + in - j * rows;
}

// The residual of channel n (clamped to the last) and 32 tokens from t0 (behind
// the last: the last's).  Without a condition on the loads: 32 conditional ones
// ran one after the other, 14 us a block instead of 1.
__device__ __forceinline__ void lin_residual(const LinearArgs &a, int t0, int n, uint32_t (&res)[32]) {
    if (!a.residual) return;
    const uint16_t *src = a.residual + min(n, a.N - 1);
    if (t0 + 32 <= a.T) {
        src += (size_t)t0 * a.N;
#pragma unroll
        for (int i = 0; i < 32; ++i) res[i] = src[(size_t)i * a.N];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) res[i] = src[(size_t)min(t0 + i, a.T - 1) * a.N];
    }
}

// Channel n of `count` tokens from t0: the epilogue of the sums v, in fp32, rounded once.
template <bool kF32, bool kFull>
__device__ __forceinline__ void lin_store32(const LinearArgs &a, int t0, int count, int n, const float (&v)[32]) {
    const size_t o = (size_t)t0 * a.N + n, ld = a.N;
    if (kF32) {
        float *out = static_cast<float *>(a.out) + o;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (kFull || i < count) out[i * ld] = v[i];
    } else {
        uint16_t *out = static_cast<uint16_t *>(a.out) + o;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (kFull || i < count) out[i * ld] = f32_to_bf16_bits(v[i]);
    }
}
template <bool kF32>
__device__ __forceinline__ void lin_activate(const LinearArgs &a, float bias, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += bias;
    if (a.act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = linear_act<MOE_ACT_RELU, kF32>(v[i]);
    } else if (a.act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = linear_act<MOE_ACT_GELU, kF32>(v[i]);
    } else if (a.act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = linear_act<MOE_ACT_SILU, kF32>(v[i]);
    }
}
template <bool kF32>
__device__ __forceinline__ void lin_epilogue(const LinearArgs &a, int t0, int count, int n, float bias,
                                             const uint32_t (&res)[32], float (&v)[32]) {
    lin_activate<kF32>(a, bias, v);
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(res[i] << 16);
    }
    if (n >= a.N) return;
    if (count >= 32) lin_store32<kF32, true>(a, t0, 32, n, v);
    else lin_store32<kF32, false>(a, t0, count, n, v);
}

// v += the partials of shares first .. last in order, 4 kVecs columns each, kShares
// of them in flight (behind the last: the last's again, not added).
template <int kShares, int kVecs, typename Part>
__device__ __forceinline__ void lin_add(float (&v)[32], int first, int last, Part part) {
    for (int w0 = first; w0 <= last; w0 += kShares) {
        float4 o[kShares][kVecs];
#pragma unroll
        for (int w = 0; w < kShares; ++w) {
            const float4 *src = part(min(w0 + w, last));
#pragma unroll
            for (int c = 0; c < kVecs; ++c) o[w][c] = __ldcg(src + c * 128);
        }
#pragma unroll
        for (int w = 0; w < kShares; ++w)
            if (w0 + w <= last)
#pragma unroll
                for (int c = 0; c < kVecs; ++c) {
                    v[4 * c] += o[w][c].x;
                    v[4 * c + 1] += o[w][c].y;
                    v[4 * c + 2] += o[w][c].z;
                    v[4 * c + 3] += o[w][c].w;
                }
    }
}

// Stores of the staged epilogue: bulk groups, one per block.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {  // all but the newest N groups have been read out of shared memory
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Bounded wait for a barrier (kCl: one that the other CTA of a pair arrives on).
// False: the limit passed or a role has given up; in a pair both CTAs learn of it.
template <bool kPair>
__device__ __noinline__ bool lin_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *status,
                                           unsigned long long limit_ns) {
    const unsigned long long t0 = globaltimer();
    for (uint32_t it = 1; !mbar_try_wait<kPair>(bar, parity); ++it) {
        if ((it & 63u) != 0) continue;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > limit_ns) {
            *abort_flag = 1;
            if (kPair) st_cluster_u32(mapa(smem_u32(const_cast<const int *>(abort_flag)), cluster_ctarank() ^ 1u), 1u);
            atomicOr(status, MOE_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}
template <bool kPair, bool kCl = kPair>
__device__ __forceinline__ bool lin_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, const LinPlan &p) {
    return mbar_try_wait<kCl>(bar, parity) || lin_wait_slow<kPair>(bar, parity, abort_flag, p.a.status, p.a.wait_limit_ns);
}

// kF32: fp32 out, the K axis summed in segments of kLinSegment slices.
template <bool kPair, bool kF32>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinPlan p) {
    constexpr int kSlices = kPair ? 1 : 2;  // K slices per stage: one barrier round trip for two small ones
    constexpr int kBlocks = kPair ? 3 : 1;  // kF32: 32-column blocks of a token tile per epilogue half
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kLinMaxStages], empty[kLinMaxStages], tfull[2], tempty[2], mma_done, rfull[8], bfull[8];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag, go_flag;
    const LinearArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const int worker = kPair ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
    const int workers = kPair ? (int)gridDim.x >> 1 : (int)gridDim.x;
    const uint32_t brows = kPair ? (uint32_t)p.Nt >> 1 : (uint32_t)p.Nt;  // token rows this CTA loads
    const uint32_t slice = kLinSliceA + (brows * 128 + 1023) / 1024 * 1024;
    uint8_t *staging = ring + (size_t)p.stages * kSlices * slice;  // the staged epilogue's 8 blocks
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], s == 0 && worker == a.stall_worker ? 3 : 2);  // the two producers
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], kPair ? 2 : 1);
        }
        mbar_init(&mma_done, 1);
        for (int i = 0; i < 8; ++i) {
            mbar_init(&rfull[i], 1);
            mbar_init(&bfull[i], 4);
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&maps.w);
        prefetch_tmap(&maps.x);
    }
    if (warp == 2) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                         "r"(2 * kLinAccStride)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                         "r"(2 * kLinAccStride)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        tc_fence_before();
    }
    if constexpr (kPair) cluster_sync();  // the other CTA's barriers exist before anything arrives on them
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_slot;
    pdl_wait();  // the operands and the workspace are ready past this point

    int tile, k0, k1;
    if (warp < 2) {
        // ================= TMA producers: W (warp 0) and tokens (warp 1) =================
        // A copy costs its issuing thread about 75 ns, a slice of a full pair's tile
        // 240 ns of MMA: one thread for both operands and the barriers held the pair at 60%.
        if (lane == 0) {
            const CUtensorMap *map = warp == 0 ? &maps.w : &maps.x;
            const uint32_t off = warp == 0 ? 0u : (uint32_t)kLinSliceA;
            const uint32_t tx = warp == 0 ? (uint32_t)kLinSliceA : brows * 128;
            // a single token tile: every weight is read once.  Otherwise the bands' repeats hit L2
            const uint64_t pol = warp == 0 && p.tt == 1 ? policy_evict_first() : policy_evict_normal();
            LinWalk walk(p, worker, workers);
            uint32_t issued = 0, ph = 0;
            int st = 0;
            bool ok = true;
            while (ok && walk.next(tile, k0, k1)) {
                int r, j;
                lin_tile(p, tile, r, j);
                const int y = warp == 0 ? (kPair ? r * 256 + (int)rank * 128 : r * 128) : j * p.Nt + (int)(rank * brows);
                for (int k = k0; k < k1; k += kSlices) {
                    const int n = min(kSlices, k1 - k);
                    if (issued >= (uint32_t)p.stages &&
                        !lin_wait<kPair>(&empty[st], ph ^ 1u, &abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = ring + (size_t)st * kSlices * slice + off;
                    if constexpr (kPair) {  // both CTAs' copies complete on CTA 0's barrier
                        if (rank == 0) mbar_arrive_expect_tx(&full[st], 2u * tx);
                        tma_load_2d_pair(map, mapa(smem_u32(&full[st]), 0), dst, k * 64, y, pol);
                    } else {
                        mbar_arrive_expect_tx(&full[st], (uint32_t)n * tx);
                        for (int u = 0; u < n; ++u)
                            tma_load_2d_hint(map, &full[st], dst + u * slice, (k + u) * 64, y, pol);
                    }
                    ++issued;
                    if (++st == p.stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // the copies still in flight (pair: released by the MMAs that read them)
            unsigned long long until = 0;
            for (uint32_t n = issued > (uint32_t)p.stages ? issued - p.stages : 0; n < issued; ++n)
                until = mbar_drain(kPair ? &empty[n % p.stages] : &full[n % p.stages], (n / p.stages) & 1u, &abort_flag,
                                   a.status, until);
        }
    } else if (warp == 2) {
        // ================= MMA issuer =================
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_bf16(p.Nt, kPair ? 256 : 128);
            const uint64_t desc0 = sw128_desc(smem_u32(ring));
            LinWalk walk(p, worker, workers);
            int st = 0;
            uint32_t ph = 0;
            bool ok = true, more = walk.next(tile, k0, k1);
            for (uint32_t it = 0; ok && more; ++it) {
                const uint32_t acc = it & 1u;
                if (!lin_wait<kPair>(&tempty[acc], ((it >> 1) & 1u) ^ 1u, &abort_flag, p)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * kLinAccStride;
                const int end = kF32 ? min(k1, k0 + kLinSegment) : k1;
                for (int k = k0; k < end; k += kSlices) {
                    const int n = min(kSlices, end - k);
                    if (!lin_wait<kPair>(&full[st], ph, &abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int u = 0; u < n; ++u) {
                        const uint64_t da = desc0 + (uint64_t)((st * kSlices + u) * slice / 16);
                        const uint64_t db = da + kLinSliceA / 16;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {  // K16 steps: 32 bytes each
                            if constexpr (kPair)
                                umma_bf16_pair(d, da + 2 * kk, db + 2 * kk, idesc, k + u > k0 || kk > 0);
                            else
                                umma_bf16(d, da + 2 * kk, db + 2 * kk, idesc, k + u > k0 || kk > 0);
                        }
                    }
                    if constexpr (kPair) umma_commit_pair(&empty[st]);
                    else umma_commit(&empty[st]);
                    if (++st == p.stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if constexpr (kPair) umma_commit_pair(&tfull[acc]);
                else umma_commit(&tfull[acc]);
                k0 = end;
                if (k0 >= k1) more = walk.next(tile, k0, k1);
            }
            if constexpr (kPair) umma_commit_pair_local(&mma_done);
            else umma_commit(&mma_done);
            mbar_wait(&mma_done, 0, &abort_flag, a.status, false);
        }
    } else if (warp == kLinThreads / 32 - 1) {
        // ================= copies of the staged epilogue =================
        // Pairs, bf16 out: the residual of a whole tile arrives by TMA in 8 blocks of 32
        // tokens x 128 channels, the epilogue turns each into the output in place, and it
        // leaves by TMA in rows of 256 bytes.  As a block leaves, the next tile's residual
        // (or just the room for it) is made ready.  The direct form's 64-byte accesses and
        // their latency held 8192 x 16384 x 256 with a residual at 2.3 TB/s.
        if (kPair && !kF32 && p.staged && lane == 0) {
            LinWalk walk(p, worker, workers);
            uint32_t bpar = 0;
            struct Place {
                int n0, t0, tile_end, end;  // first channel and token, the tile's end in tokens, and the rows'
            };
            auto place = [&](int tile) {
                int r, j;
                lin_tile(p, tile, r, j);
                const int n0 = r * 256 + (int)rank * 128, tile_end = (j + 1) * p.Nt;
                return Place{n0, j * p.Nt, tile_end, n0 < a.N ? min(tile_end, a.T) : 0};
            };
            // tokens of a block: 0, 16 or 32 (also 32 where the rows end: TMA stops there)
            auto tokens = [&](const Place &at, int blk) {
                const int t = at.t0 + 32 * blk;
                return t >= at.end ? 0 : t + 16 < at.tile_end ? 32 : 16;
            };
            auto make_ready = [&](const Place &at, int blk) {
                const int rows = tokens(at, blk);
                if (rows == 0) return;
                if (a.residual) {
                    mbar_arrive_expect_tx(&rfull[blk], rows * 256);
                    tma_load_2d(rows == 32 ? &maps.r : &maps.r16, &rfull[blk], staging + blk * kLinBlockBytes, at.n0,
                                at.t0 + 32 * blk);
                } else {
                    mbar_arrive(&rfull[blk]);
                }
            };
            bool more = walk.next(tile, k0, k1) && k1 - k0 == p.nk, ok = true;
            Place now{}, next = more ? place(tile) : now;
            for (int blk = 0; more && blk < 8; ++blk) make_ready(next, blk);
            // the two blocks that left last and whether the next tile (or this one) wants them
            int qa = -1, qb = -1;
            bool qa_next = false, qb_next = false;
            auto flush = [&](int q, bool to_next) {
                if (q >= 0) make_ready(to_next ? next : now, q);
            };
            while (more && ok) {
                now = next;
                qa_next = qb_next = false;
                more = walk.next(tile, k0, k1) && k1 - k0 == p.nk;
                if (more) next = place(tile);
                for (int blk = 0; blk < 8; ++blk) {
                    if (blk == qa || blk == qb) {  // narrow tiles: wanted already
                        bulk_wait_read<0>();
                        flush(qa, qa_next);
                        flush(qb, qb_next);
                        qa = qb = -1;
                    }
                    const int rows = tokens(now, blk);
                    if (rows == 0) {
                        if (more) make_ready(next, blk);  // not used by this tile
                        continue;
                    }
                    ok = lin_wait<kPair, false>(&bfull[blk], (bpar >> blk) & 1u, &abort_flag, p);
                    if (!ok) break;
                    bpar ^= 1u << blk;
                    tma_store_2d(rows == 32 ? &maps.o : &maps.o16, staging + blk * kLinBlockBytes, now.n0,
                                 now.t0 + 32 * blk);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    bulk_wait_read<2>();
                    flush(qa, qa_next);
                    qa = qb;
                    qa_next = qb_next;
                    qb = more ? blk : -1;
                    qb_next = true;
                }
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            if (!ok)  // residuals may be on their way
                for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < kDrainNs;) {
                }
        }
    } else {
        // ================= epilogue =================
        const int q = warp & 3, half = (warp - 3) >> 2, row = q * 32 + lane;
        const bool elected = threadIdx.x == 96;
        auto release = [&](uint32_t acc) {
            if (kPair && rank != 0) mbar_arrive_cluster(mapa(smem_u32(&tempty[acc]), 0));
            else mbar_arrive(&tempty[acc]);
        };
        constexpr bool kCanStage = kPair && !kF32;
        uint32_t rpar = 0;  // parity of the half's four block barriers
        LinWalk walk(p, worker, workers);
        for (uint32_t it = 0; walk.next(tile, k0, k1);) {
            int r, j;
            lin_tile(p, tile, r, j);
            const int n = (kPair ? r * 256 + (int)rank * 128 : r * 128) + row;
            const int t0 = j * p.Nt, cols = min(p.Nt, a.T - t0);
            const bool whole = k1 - k0 == p.nk;
            const float bias = a.bias && n < a.N ? bf16_bits_to_f32(__ldg(a.bias + n)) : 0.f;
            uint32_t next[32];  // the coming block's residual, read ahead of its sums
            const bool staged = kCanStage && p.staged && whole;
            if (!kF32 && !staged && whole && half * 32 < cols) lin_residual(a, t0 + half * 32, n, next);
            // the sums: in TMEM, or (kF32) of all segments but the last in registers
            float sum[kF32 ? kBlocks : 1][32];
            uint32_t acc = 0, tbase = 0;
            bool go = true;
#pragma unroll 1
            for (int k = k0; k < k1; k += kF32 ? kLinSegment : k1 - k0, ++it) {
                acc = it & 1u;
                tbase = tmem_base + acc * kLinAccStride + ((uint32_t)(q * 32) << 16);
                if (elected) go_flag = lin_wait<kPair>(&tfull[acc], (it >> 1) & 1u, &abort_flag, p);
                named_bar_sync(1, kLinEpi);
                go = go_flag;
                if (!go) break;
                tc_fence_after();
                if constexpr (kF32) {
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b)
                        if (half * 32 + 64 * b < p.Nt) {
                            float v[32];
                            tmem_ld32(tbase + (uint32_t)(half * 32 + 64 * b), v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) sum[b][i] = k == k0 ? v[i] : sum[b][i] + v[i];
                        }
                    tc_fence_before();
                    named_bar_sync(1, kLinEpi);
                    if (elected) release(acc);
                }
            }
            if (!go) break;
            auto done = [&] {  // the accumulator is read
                if constexpr (!kF32) {
                    tc_fence_before();
                    named_bar_sync(1, kLinEpi);
                    if (elected) release(acc);
                }
            };
            if constexpr (kCanStage) {
                if (staged) {
                    const int n0 = n - row, nb = n0 < a.N ? (cols - half * 32 + 63) / 64 : 0;  // this half's blocks
                    for (int b = 0; b < nb; ++b) {
                        const int c0 = half * 32 + 64 * b, blk = 2 * b + half;
                        uint16_t *buf = reinterpret_cast<uint16_t *>(staging + blk * kLinBlockBytes) + row;
                        float v[32];
                        tmem_ld32(tbase + (uint32_t)c0, v);
                        lin_activate<kF32>(a, bias, v);
                        lin_wait<kPair, false>(&rfull[blk], (rpar >> b) & 1u, &abort_flag, p);
                        rpar ^= 1u << b;
                        if (a.residual) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] += bf16_bits_to_f32(buf[i * 128]);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) buf[i * 128] = f32_to_bf16_bits(v[i]);
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bfull[blk]);
                    }
                    done();
                    continue;
                }
            }
            if (whole) {
                if constexpr (kF32) {
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        const int c0 = half * 32 + 64 * b;
                        if (c0 < cols) {
                            lin_residual(a, t0 + c0, n, next);
                            lin_epilogue<kF32>(a, t0 + c0, cols - c0, n, bias, next, sum[b]);
                        }
                    }
                } else {
                    for (int c0 = half * 32; c0 < cols; c0 += 64) {
                        uint32_t res[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) res[i] = next[i];
                        if (c0 + 64 < cols) lin_residual(a, t0 + c0 + 64, n, next);
                        float v[32];
                        tmem_ld32(tbase + (uint32_t)c0, v);
                        lin_epilogue<kF32>(a, t0 + c0, cols - c0, n, bias, res, v);
                    }
                }
                done();
                continue;
            }
            // a share of the tile: its sums to the workspace, [column / 4][128 rows] float4
            const long long s0 = (long long)(tile - workers * p.waves) * p.nk, total = (long long)p.rest * p.nk;
            const int first = (int)(((s0 + 1) * p.sharers - 1) / total);
            const int last = (int)(((s0 + p.nk) * p.sharers - 1) / total);
            const int blocks = (p.Nt + 31) / 32;
            auto part = [&](int w) {
                const int slot = ((w * 2 + (w == first)) << kPair) + (int)rank;
                return reinterpret_cast<float4 *>(a.scratch + (size_t)slot * 128 * 32 * blocks) + row;
            };
            auto put = [&](int c0, const float (&v)[32]) {
                float4 *dst = part(worker) + c0 / 4 * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    __stcg(dst + c * 128, make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]));
            };
            if constexpr (kF32) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
                    if (half * 32 + 64 * b < p.Nt) put(half * 32 + 64 * b, sum[b]);
            } else {
                for (int c0 = half * 32; c0 < p.Nt; c0 += 64) {
                    float v[32];
                    tmem_ld32(tbase + (uint32_t)c0, v);
                    put(c0, v);
                }
            }
            done();
            if constexpr (kF32) named_bar_sync(1, kLinEpi);  // (done() has one otherwise)
            // Once all shares are in, the tile's 32-column blocks are added up in share
            // order by whichever warps of its sharers (of the same lane quarter) are there
            // to take one: the last to arrive, and those that wait for it at the end of
            // their walk.  Nobody has to wait: what is not taken the last one does.
            const uint32_t shares = (uint32_t)(last - first + 1);
            uint32_t *word = reinterpret_cast<uint32_t *>(a.sync) + ((first << kPair) + (int)rank) * 4 + q;
            int ready = 0;  // word: shares in, blocks taken << 8, warps gone << 16
            if (lane == 0 && (half == 0 || blocks > 1)) {
                uint32_t v = 0;
                if (half == 0) {
                    v = add_acq_rel(word, 1u) + 1u;  // releases all of the CTA's partial: a barrier lies before
                } else {
                    v = (uint32_t)ld_acquire(reinterpret_cast<const int32_t *>(word));
                }
                if (blocks > 1 && walk.finished()) {
                    const unsigned long long t0 = globaltimer();
                    while ((v & 255u) < shares && !abort_flag && globaltimer() - t0 < kLinLingerNs)
                        v = (uint32_t)ld_acquire(reinterpret_cast<const int32_t *>(word));
                }
                ready = (v & 255u) == shares;
            }
            ready = __shfl_sync(0xffffffffu, ready, 0);
            __syncwarp();  // lane 0's acquire lies before the other lanes' loads of the partials
            while (ready) {
                int blk = 0;
                if (blocks > 1) {
                    if (lane == 0) blk = (int)(atomicAdd(word, 1u << 8) >> 8 & 255u);
                    blk = __shfl_sync(0xffffffffu, blk, 0);
                    if (blk >= blocks) break;
                }
                const int c0 = 32 * blk;
                float v[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = 0.f;
                if (c0 < cols) lin_residual(a, t0 + c0, n, next);
                if (!kPair && p.Nt <= 16) lin_add<4, 4>(v, first, last, [&](int w) { return part(w) + c0 / 4 * 128; });
                else lin_add<kF32 && kPair ? 1 : 2, 8>(v, first, last, [&](int w) { return part(w) + c0 / 4 * 128; });
                if (c0 < cols) lin_epilogue<kF32>(a, t0 + c0, cols - c0, n, bias, next, v);
                if (blocks == 1) break;
            }
            // the last warp to go (of one block: the one that added it) leaves the word at zero
            if (lane == 0 && (blocks > 1 ? (atomicAdd(word, 1u << 16) >> 16 & 255u) == 2 * shares - 1 : ready))
                atomicExch(word, 0u);
        }
    }

    __syncthreads();
    if constexpr (kPair) cluster_sync();  // the other CTA is done with the shared TMEM allocation and our barriers
    if (warp == 2) {
        tc_fence_after();
        if constexpr (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(2 * kLinAccStride)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(2 * kLinAccStride)
                         : "memory");
    }
}

// Single CTAs up to this many tokens, pairs above (figures at the top).
constexpr int kLinSingleTokens = 64;

// Token tile: the tokens in as few tiles of at most 256 (fp32 out: 192, whose sums a
// thread holds in 96 registers; 128 took 800 us for 8000 x 6000 x 6000, 192 takes 630 to
// 675) as hold them, rounded up to 16.
constexpr int kLinMaxTile = 256;
int lin_token_tile(int T, bool f32) {
    const int most = f32 ? 192 : kLinMaxTile, tiles = (T - 1) / most + 1;
    return ((T - 1) / tiles + 16) / 16 * 16;
}

template <bool kPair, bool kF32>
cudaError_t launch_shape(const LinearArgs &a, int sms, cudaStream_t st) {
    constexpr int kSlices = kPair ? 1 : 2;
    LinPlan p{};
    p.a = a;
    p.Nt = lin_token_tile(a.T, kF32);
    p.nk = (a.K + 63) / 64;
    p.rt = (a.N - 1) / (kPair ? 256 : 128) + 1;
    p.tt = (a.T - 1) / p.Nt + 1;
    const long long tiles = (long long)p.rt * p.tt;
    if (tiles >= (1ll << 30)) return cudaErrorInvalidValue;
    int workers = kPair ? sms / 2 : sms;
    p.waves = (int)(tiles / workers);
    p.rest = (int)(tiles % workers);
    // the rest's K slices over the whole grid, unless that shortens it by fewer slices
    // (0.3 us each) than adding the partials costs: about 4 us for 16 tokens, 13 us for
    // 256.  2000 x 8192 x 1024 took 41 us in whole tiles and 70 us shared; 224 x 5120 x
    // 17408 97 us in whole tiles and 47 us shared
    p.sharers = p.rest;
    if (p.rest > 0) {
        const int split = std::min(kLinMaxSplit, std::max(1, (int)std::sqrt(p.nk)));
        const int s = std::min(workers, p.rest * std::min(split, std::max(1, p.nk / 4)));
        if ((long long)(s - p.rest) * p.nk >= (12ll + p.Nt / 8) * s) p.sharers = s;
    }
    if (p.waves == 0) workers = p.sharers;
    const int brows = kPair ? p.Nt / 2 : p.Nt;
    const int stage = kSlices * (kLinSliceA + (brows * 128 + 1023) / 1024 * 1024);
    // Whole tiles of pairs with bf16 out go through shared memory where TMA can take
    // their rows (a stride of whole 16 bytes) and K is short, so that the epilogue
    // counts: 8192 x 16384 x 256 with a residual 228 us direct and 161 us staged, 2000 x
    // 8192 x 1024 41 and 36; 1000 x 5120 x 5120 51 and 53 (a shorter ring).
    p.staged = kPair && !kF32 && p.waves > 0 && a.N % 8 == 0 && p.nk <= kLinStagedSlices;
    const int staging = p.staged ? 8 * kLinBlockBytes : 0;
    p.stages = std::min(kLinMaxStages, (kLinRing - staging) / stage);
    LinMaps m;
    if (!encode_2d(&m.w, a.w, a.N, a.K, 128) || !encode_2d(&m.x, a.x, a.T, a.K, brows)) return cudaErrorInvalidValue;
    m.r = m.r16 = m.o = m.o16 = m.x;  // not read
    if (p.staged && (!encode_rows(&m.o, a.out, a.T, a.N, 128, 32) || !encode_rows(&m.o16, a.out, a.T, a.N, 128, 16)))
        return cudaErrorInvalidValue;
    if (p.staged && a.residual &&
        (!encode_rows(&m.r, a.residual, a.T, a.N, 128, 32) || !encode_rows(&m.r16, a.residual, a.T, a.N, 128, 16)))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + (size_t)p.stages * stage + staging;
    static std::atomic<int> attr_set[64];  // per device: opted in to the ring's shared memory
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(linear_kernel<kPair, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kLinRing);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPair ? 2 * workers : workers);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<kPair, kF32>, m, p);
}

}  // namespace

size_t linear_scratch_bytes(int T, int N, int K) {
    (void)N;
    (void)K;
    // two partials per CTA of the widest token tile that T or fewer tokens have (tiles
    // are narrower again at 257 tokens than at 256), so that a workspace serves fewer too
    return (size_t)kLinMaxSms * 2 * 128 * ((std::min(T, kLinMaxTile) + 31) / 32 * 32) * 4;
}

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t st) {
    const int sms = std::min(device_sm_count(), kLinMaxSms);
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (a.T <= kLinSingleTokens || sms < 2)
        return a.out_f32 ? launch_shape<false, true>(a, sms, st) : launch_shape<false, false>(a, sms, st);
    return a.out_f32 ? launch_shape<true, true>(a, sms, st) : launch_shape<true, false>(a, sms, st);
}

}  // namespace moe
