// Host-side internal interface between the C ABI of qmv_serve.h
// (serve_api.cpp) and its kernel translation units.  Arguments reaching these
// functions have already been validated.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qmv_serve.h"

namespace qmv {

struct PlanArgs {
    const int32_t* kv_len;
    const int32_t* keep;  // or null
    const int32_t* n_new;
    const int32_t* free_count;
    int32_t* new_len;
    int32_t* new_count;
    int32_t* row_start;
    int32_t* position;  // or null
    int64_t* slot;      // or null
    int32_t* status;
    int64_t T;
};
size_t plan_ws_bytes(int B);
hipError_t launch_kv_plan(const qmv_kv_pool& pool, const PlanArgs& a, void* ws, hipStream_t stream);

// fmt: 0 Q4_0, 1 Q8_0, 2 Q4_K, 3 Q6_K, as in launch_gemv.
hipError_t launch_embed(int fmt, const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M,
                        float scale, hipStream_t stream);

struct LoraArgs {
    const int32_t* adapter;
    const int32_t* row_start;
    const float* x;
    const float* base;  // or null
    float* y;
    int64_t ldx, ldb, ldy, B, T;
};
size_t lora_ws_bytes(const qmv_lora& l, int64_t B, int64_t T);
hipError_t launch_lora(const qmv_lora& l, const LoraArgs& a, void* ws, hipStream_t stream);

struct DrawArgs {
    const float* logits;
    const float* temperature;
    const int32_t* top_k;  // or null, as the next two
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* token;
    int32_t* kept;  // or null
    int64_t ldl, V, M;
    float softcap;
};
size_t draw_ws_bytes(int64_t V, int64_t M);
hipError_t launch_logits_draw(const DrawArgs& a, void* ws, hipStream_t stream);

}  // namespace qmv
