// Argument block and launch of the few-token layer (few.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kFewMaxTokens = MOE_FEW_MAX_TOKENS;

// One projection's weights in any of the three formats: bf16 values, or codes
// with packed block scales (and, NVFP4, fp32 matrix scales).
struct FewMatrix {
    const void *w;
    const uint8_t *sf;
    const float *ts;
};

struct FewArgs {
    int T, H, E, I, k, Is;
    int norm_topk, budget;
    float topp;
    const uint16_t *x, *w_router, *gvec;
    float *logits;  // given, or where the projection puts them
    int project;    // 1: logits = x . w_router^T first
    FewMatrix gate, up, down, s_gate, s_up, s_down;
    int32_t *idx;   // outputs, null when not wanted
    float *w;
    float *sgate;   // [T], always set when Is > 0
    int32_t *keff;
    uint8_t *kept;
    int32_t *n_dropped;
    uint16_t *out;
    void *h;        // scratch: row-block partials, then the gate/up activations
    int32_t *status, *sync;
    unsigned long long wait_limit_ns;  // of the grid's waits, and the one that stalls
    int stall_wait;                    // (wait_hooks)
};

// Ints of the workspace head the kernel's counters take (zero between launches).
constexpr int kFewSyncInts = 16 + 3 * 160;
size_t few_scratch_bytes(int T, int E, int I, int k, int Is);
// fmt: 0 bf16, 1 MXFP8, 2 NVFP4.
cudaError_t launch_few(const FewArgs &a, int fmt, cudaStream_t st);

}  // namespace moe
