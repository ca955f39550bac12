// C ABI of qmv_serve.h: argument checking and dispatch, by the rules of
// qmv_api.cpp (every check on the host before anything is enqueued; on any
// error nothing is launched).
#include "../../include/qmv_serve.h"

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "serve_internal.h"

namespace {

constexpr int64_t kMaxInt = (int64_t{1} << 31) - 1;
// one workgroup of 256 threads a row: a grid holds fewer than 2^32 threads
constexpr int64_t kMaxT = (int64_t{1} << 24) - 1;
// softcap: tanh is taken to 2^-42, so that a level is off by 2^-26 at most
constexpr float kMaxCap = 65536.0f;
constexpr float kMaxFloat = 3.4028234663852886e38f;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

int launched(hipError_t e) { return e == hipSuccess ? QMV_OK : QMV_ERR_LAUNCH; }

int check_pool_shape(const qmv_kv_pool& p) {
    if (p.num_pages < 1 || p.num_pages > kMaxInt || p.B < 1 || p.B > 65535 || p.max_pages < 1) return QMV_ERR_SHAPE;
    if (p.page_size < 16 || p.page_size > 1024 || (p.page_size & (p.page_size - 1)) != 0) return QMV_ERR_SHAPE;
    if (static_cast<int64_t>(p.max_pages) * p.page_size > (int64_t{1} << 30)) return QMV_ERR_SHAPE;
    return QMV_OK;
}

int check_lora_shape(const qmv_lora& l, int64_t B, int64_t T) {
    if (l.format != QMV_LORA_F16 && l.format != QMV_LORA_BF16) return QMV_ERR_ARG;
    if (l.K < 8 || l.K > kMaxT || l.K % 8 != 0 || l.N < 1 || l.N > kMaxT) return QMV_ERR_SHAPE;
    if (l.max_rank < 8 || l.max_rank > 256 || l.max_rank % 8 != 0) return QMV_ERR_SHAPE;
    if (l.slots < 1 || l.slots >= (1 << 20)) return QMV_ERR_SHAPE;
    if (B < 1 || B > 65535 || T < 1 || T > kMaxT) return QMV_ERR_SHAPE;
    return QMV_OK;
}

// T rows of `width` float32 elements, ld apart.
int check_rows(const void* p, int64_t ld, int64_t width, int64_t T) {
    int64_t t;
    if (ld < width || !mul_ok(ld, T, &t) || !mul_ok(t, 4, &t)) return QMV_ERR_SHAPE;
    return aligned(p, 4) ? QMV_OK : QMV_ERR_ALIGN;
}

int embed(int fmt, const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
          hipStream_t stream) {
    if (!W || !tokens || !y) return QMV_ERR_NULL;
    if (N < 1 || N > kMaxInt || M < 1 || M > kMaxT || K < 1 || K > kMaxInt) return QMV_ERR_SHAPE;
    if (K % (fmt >= 2 ? 256 : 32) != 0) return QMV_ERR_SHAPE;  // the byte counts of N and M rows fit then
    if (!(scale >= -kMaxFloat) || !(scale <= kMaxFloat)) return QMV_ERR_ARG;
    if (!aligned(W, 16) || !aligned(tokens, 4) || !aligned(y, 4)) return QMV_ERR_ALIGN;
    return launched(qmv::launch_embed(fmt, W, tokens, y, N, K, M, scale, stream));
}

}  // namespace

extern "C" {

size_t kv_plan_ws_bytes(const qmv_kv_pool* pool) {
    if (!pool || check_pool_shape(*pool)) return 0;
    return qmv::plan_ws_bytes(pool->B);
}

int kv_plan(const qmv_kv_pool* pool, const int32_t* kv_len, const int32_t* keep, const int32_t* n_new,
            const int32_t* free_count, int32_t* new_len, int32_t* new_count, int32_t* row_start, int32_t* position,
            int64_t* slot, int32_t* status, int64_t T, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!pool || !pool->page_table || !pool->free_pages || !kv_len || !n_new || !free_count || !new_len || !new_count ||
        !row_start || !status || !ws)
        return QMV_ERR_NULL;
    const int rc = check_pool_shape(*pool);
    if (rc) return rc;
    if (T < 1 || T > kMaxT) return QMV_ERR_SHAPE;
    if (!aligned(pool->page_table, 4) || !aligned(pool->free_pages, 4) || !aligned(kv_len, 4) || !aligned(keep, 4) ||
        !aligned(n_new, 4) || !aligned(free_count, 4) || !aligned(new_len, 4) || !aligned(new_count, 4) ||
        !aligned(row_start, 4) || !aligned(position, 4) || !aligned(slot, 8) || !aligned(status, 4) || !aligned(ws, 16))
        return QMV_ERR_ALIGN;
    if (ws_bytes < qmv::plan_ws_bytes(pool->B)) return QMV_ERR_WORKSPACE;
    qmv::PlanArgs a;
    a.kv_len = kv_len;
    a.keep = keep;
    a.n_new = n_new;
    a.free_count = free_count;
    a.new_len = new_len;
    a.new_count = new_count;
    a.row_start = row_start;
    a.position = position;
    a.slot = slot;
    a.status = status;
    a.T = T;
    return launched(qmv::launch_kv_plan(*pool, a, ws, stream));
}

int embed_q8_0(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream) {
    return embed(1, W, tokens, y, N, K, M, scale, stream);
}

int embed_q4_0(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream) {
    return embed(0, W, tokens, y, N, K, M, scale, stream);
}

int embed_q4_k(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream) {
    return embed(2, W, tokens, y, N, K, M, scale, stream);
}

int embed_q6_k(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream) {
    return embed(3, W, tokens, y, N, K, M, scale, stream);
}

size_t lora_add_ws_bytes(const qmv_lora* lora, int64_t B, int64_t T) {
    if (!lora || check_lora_shape(*lora, B, T)) return 0;
    return qmv::lora_ws_bytes(*lora, B, T);
}

int lora_add(const qmv_lora* lora, const int32_t* adapter, const int32_t* row_start, const float* x, int64_t ldx,
             const float* base, int64_t ldb, float* y, int64_t ldy, int64_t B, int64_t T, void* ws, size_t ws_bytes,
             hipStream_t stream) {
    if (!lora || !lora->A || !lora->Bm || !lora->scale || !adapter || !row_start || !x || !y || !ws) return QMV_ERR_NULL;
    int rc = check_lora_shape(*lora, B, T);
    if (!rc) rc = check_rows(x, ldx, lora->K, T);
    if (!rc && base) rc = check_rows(base, ldb, lora->N, T);
    if (!rc) rc = check_rows(y, ldy, lora->N, T);
    if (rc) return rc;
    // in place means row by row
    if (base == y && ldb != ldy) return QMV_ERR_ARG;
    if (!aligned(lora->A, 16) || !aligned(lora->Bm, 16) || !aligned(lora->rank, 4) || !aligned(lora->scale, 4) ||
        !aligned(adapter, 4) || !aligned(row_start, 4) || !aligned(ws, 16))
        return QMV_ERR_ALIGN;
    if (ws_bytes < qmv::lora_ws_bytes(*lora, B, T)) return QMV_ERR_WORKSPACE;
    qmv::LoraArgs a;
    a.adapter = adapter;
    a.row_start = row_start;
    a.x = x;
    a.base = base;
    a.y = y;
    a.ldx = ldx;
    a.ldb = ldb;
    a.ldy = ldy;
    a.B = B;
    a.T = T;
    return launched(qmv::launch_lora(*lora, a, ws, stream));
}

size_t logits_draw_ws_bytes(int64_t V, int64_t M) {
    if (V < 1 || V > kMaxInt || M < 1 || M > 65535) return 0;
    return qmv::draw_ws_bytes(V, M);
}

int logits_draw(const float* logits, int64_t ldl, const float* temperature, const int32_t* top_k, const float* top_p,
                const float* min_p, const float* u, int32_t* token, int32_t* kept, int64_t V, int64_t M, float softcap,
                void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!logits || !temperature || !u || !token || !ws) return QMV_ERR_NULL;
    const size_t need = logits_draw_ws_bytes(V, M);
    if (need == 0) return QMV_ERR_SHAPE;
    const int rc = check_rows(logits, ldl, V, M);
    if (rc) return rc;
    if (!(softcap >= 0.0f) || !(softcap <= kMaxCap)) return QMV_ERR_ARG;
    if (!aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(u, 4) ||
        !aligned(token, 4) || !aligned(kept, 4) || !aligned(ws, 16))
        return QMV_ERR_ALIGN;
    if (ws_bytes < need) return QMV_ERR_WORKSPACE;
    qmv::DrawArgs a;
    a.logits = logits;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.kept = kept;
    a.ldl = ldl;
    a.V = V;
    a.M = M;
    a.softcap = softcap;
    return launched(qmv::launch_logits_draw(a, ws, stream));
}

}  // extern "C"
