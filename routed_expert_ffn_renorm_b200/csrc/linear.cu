// The fused linear map out = residual + act(x W^T + bias): bf16 operands,
// fp32 sums, one rounding of the result (or none, fp32 out).
//
// One 64 x 64 output tile per CTA from 16-wide K slices in shared memory,
// 4 x 4 outputs per thread.
#include "linear.cuh"

namespace moe {

namespace {

constexpr int kTile = 64, kSlice = 16;

__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
    __shared__ float xs[kSlice][kTile + 1], wsh[kSlice][kTile + 1];
    const int t0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kSlice) {
        for (int i = threadIdx.x; i < kTile * kSlice; i += 256) {
            const int r = i / kSlice, c = i % kSlice, k = k0 + c;
            xs[c][r] = t0 + r < a.T && k < a.K ? bf16_bits_to_f32(a.x[(size_t)(t0 + r) * a.K + k]) : 0.f;
            wsh[c][r] = n0 + r < a.N && k < a.K ? bf16_bits_to_f32(a.w[(size_t)(n0 + r) * a.K + k]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kSlice; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[c][ty * 4 + i], wsh[c][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + ty * 4 + i, n = n0 + tx + 16 * j;
            if (t < a.T && n < a.N) linear_store(a, t, n, acc[i][j]);
        }
}

}  // namespace

size_t linear_scratch_bytes(int, int, int) { return 0; }

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t st) {
    const dim3 grid((a.N + kTile - 1) / kTile, (a.T + kTile - 1) / kTile);
    linear_kernel<<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
