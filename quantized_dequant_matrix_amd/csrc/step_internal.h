// Host-side internal interface between the C ABI of qmv_step.h (step_api.cpp)
// and its kernel translation units.  Arguments reaching these functions have
// already been validated.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qmv_step.h"

namespace qmv {

hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* k, int64_t ldk, const float* v,
                           int64_t ldv, hipStream_t stream);
hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_batch& b, float* k, int64_t ldk, float* v, int64_t ldv,
                          hipStream_t stream);

// The workspace's size depends on the descriptors' numbers and q_heads only.
size_t attn_ws_bytes(const qmv_kv_cache& c, const qmv_kv_batch& b, int q_heads);
hipError_t launch_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* q, int64_t ldq, float* out,
                       int64_t ldo, int q_heads, float scale, int window, void* ws, hipStream_t stream);

// q == nullptr: y float32; else the codes and scales.  z and r may be null.
hipError_t launch_rmsnorm(const float* x, const float* r, const float* w, float* z, float* y, int8_t* q, float* d,
                          int64_t K, int64_t M, float eps, hipStream_t stream);

// Step 2 of qmm_q4_0_q8act on row-major codes and scales (qmm.hip).
hipError_t launch_qmm_q8(const void* W, const int8_t* q, const float* d, float* y, int64_t N, int64_t K, int64_t M,
                         void* ws, hipStream_t stream);

struct DraftArgs {
    const float* target;
    const float* draft;
    const int32_t* draft_tokens;
    const int32_t* n_draft;
    const float* u;
    int32_t* accepted;
    int32_t* tokens;
    int64_t ldt, ldd, V, B;
    int G;
    float temperature, softcap;
};
size_t draft_ws_bytes(int64_t B, int G, int64_t V);
hipError_t launch_draft_verify(const DraftArgs& a, void* ws, hipStream_t stream);

}  // namespace qmv
