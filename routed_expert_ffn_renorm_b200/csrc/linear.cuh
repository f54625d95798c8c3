// Argument block, epilogue and launch of the fused linear map (linear.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {

struct LinearArgs {
    int T, N, K;
    const uint16_t *x, *w;            // [T, K], [N, K]
    const uint16_t *bias, *residual;  // [N], [T, N]; null: none
    int act;                          // MOE_ACT_*
    void *out;                        // [T, N], bf16 or (out_f32) fp32; may be `residual` itself when bf16
    int out_f32;
    int32_t *status, *sync;
    float *scratch;
};

__device__ __forceinline__ float linear_act(float v, int act) {
    if (act == MOE_ACT_RELU) return v < 0.f ? 0.f : v;  // a NaN stays
    if (act == MOE_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);  // no cancellation for v < 0
    if (act == MOE_ACT_SILU) return v / (1.f + expf(-v));
    return v;
}

// The epilogue of one output: everything in fp32, rounded once.
__device__ __forceinline__ void linear_store(const LinearArgs &a, int t, int n, float v) {
    if (a.bias) v += bf16_bits_to_f32(__ldg(a.bias + n));
    v = linear_act(v, a.act);
    const size_t o = (size_t)t * a.N + n;
    if (a.residual) v += bf16_bits_to_f32(a.residual[o]);
    if (a.out_f32)
        static_cast<float *>(a.out)[o] = v;
    else
        static_cast<uint16_t *>(a.out)[o] = f32_to_bf16_bits(v);
}

size_t linear_scratch_bytes(int T, int N, int K);
cudaError_t launch_linear(const LinearArgs &a, cudaStream_t st);

}  // namespace moe
