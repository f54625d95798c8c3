// Argument block, activations and launch of the fused linear map (linear.cu).
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
    unsigned long long wait_limit_ns;  // of the pipeline's waits, and a worker whose first
    int stall_worker;                  // ring slot never fills (wait_hooks)
};

// kExact: results that stay fp32.
template <int kAct, bool kExact>
__device__ __forceinline__ float linear_act(float v) {
    if (kAct == MOE_ACT_RELU) return v < 0.f ? 0.f : v;  // a NaN stays
    if (kAct == MOE_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);  // no cancellation for v < 0
    if (kAct == MOE_ACT_SILU) {
        if (kExact) return v / (1.f + expf(-v));
        // Before a rounding to bf16: the approximate exponential, whose error grows to
        // 2 + 1.17 |v| ulps (1.2e-5 at v = -80, where bf16 keeps 3.9e-3), and reciprocal.
        // 13 us less of 650 for 59M outputs
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-v)));
        return v * r;
    }
    return v;
}

constexpr int kLinMaxSms = 160;  // no device has more SMs (workspace sizing)
// Ints of the workspace head the kernel counts in (zero between launches).
constexpr int kLinSyncInts = 4 * kLinMaxSms;
size_t linear_scratch_bytes(int T, int N, int K);
cudaError_t launch_linear(const LinearArgs &a, cudaStream_t st);

}  // namespace moe
