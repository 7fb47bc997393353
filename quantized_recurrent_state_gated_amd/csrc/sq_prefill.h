// sq_prefill.h -- internal interface between the host code (sq_serve_api.hip)
// and the kernels of the prompt form (sq_prefill.hip).  Not installed, not
// part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sqk {

struct PrefillArgs {
    const void *q, *k, *v;       // [N][k_heads][dk] (q, k), [N][heads][dv]; tokens *_stride apart
    int64_t q_stride, k_stride, v_stride;
    const float *alpha, *beta;   // [N][heads]
    const int32_t *cu;           // [n_seq + 1]
    int32_t n_seq, n_tokens, heads, per_k;  // per_k = heads / k_heads
    int32_t dk, dv;
    const float *S0;             // [n_seq][heads][dk][dv] or null
    void *o;                     // [N][heads][dv]
    float *S;                    // [n_seq][heads][dk][dv] or null; may be S0
    uint8_t *ws;                 // workspace of the segments, if any
    int32_t seg = 0;             // chunks per segment, and where the workspace's states
    int64_t seg_pad = 0;         // start, in floats (both set by the launcher)
};

// Workspace for every call with at most these sizes, and what one call needs.
uint64_t prefill_workspace(int32_t n_seq, int32_t n_tokens, int32_t heads, int32_t dk, int32_t dv,
                           bool bf16, bool delta);
uint64_t prefill_needs(const PrefillArgs &a, bool bf16, bool delta);
hipError_t launch_prefill(const PrefillArgs &a, bool bf16, bool delta, hipStream_t st);

}  // namespace sqk
