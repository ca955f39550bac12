// C ABI of qmv_step.h: argument checking and dispatch, by the rules of
// qmv_api.cpp (every check on the host before anything is enqueued; on any
// error nothing is launched).
#include "../../include/qmv_step.h"

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "step_internal.h"

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

// The numbers of the two descriptors (the sizes, not the pointers).
int check_cache_shape(const qmv_kv_cache& c) {
    if (c.format != QMV_KV_Q8 && c.format != QMV_KV_F16) return QMV_ERR_ARG;
    if (c.num_pages < 1 || c.num_pages > kMaxInt || c.kv_heads < 1 || c.kv_heads > 65535) return QMV_ERR_SHAPE;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return QMV_ERR_SHAPE;
    if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)) != 0) return QMV_ERR_SHAPE;
    int64_t t;
    if (!mul_ok(c.num_pages, c.kv_heads, &t) || !mul_ok(t, 2 * c.page_size * c.head_dim, &t)) return QMV_ERR_SHAPE;
    return QMV_OK;
}

int check_batch_shape(const qmv_kv_cache& c, const qmv_kv_batch& b) {
    if (b.T < 1 || b.T > kMaxT || b.B < 1 || b.B > 65535 || b.max_pages < 1) return QMV_ERR_SHAPE;
    if (static_cast<int64_t>(b.max_pages) * c.page_size > (int64_t{1} << 30)) return QMV_ERR_SHAPE;
    return QMV_OK;
}

int check_kv(const qmv_kv_cache* c, const qmv_kv_batch* b) {
    if (!c || !b || !c->k || !c->v || !b->page_table || !b->row_start || !b->kv_len) return QMV_ERR_NULL;
    if (c->format == QMV_KV_Q8 && (!c->k_scale || !c->v_scale)) return QMV_ERR_NULL;
    int rc = check_cache_shape(*c);
    if (!rc) rc = check_batch_shape(*c, *b);
    if (rc) return rc;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(b->page_table, 4) || !aligned(b->row_start, 4) ||
        !aligned(b->kv_len, 4))
        return QMV_ERR_ALIGN;
    if (c->format == QMV_KV_Q8 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))) return QMV_ERR_ALIGN;
    return QMV_OK;
}

// T rows of `width` float32 elements, ld apart.
int check_rows(const void* p, int64_t ld, int64_t width, int64_t T) {
    int64_t t;
    if (ld < width || !mul_ok(ld, T, &t) || !mul_ok(t, 4, &t)) return QMV_ERR_SHAPE;
    return aligned(p, 4) ? QMV_OK : QMV_ERR_ALIGN;
}

int check_q_heads(const qmv_kv_cache& c, const qmv_kv_batch& b, int32_t q_heads) {
    if (q_heads < 1 || q_heads % c.kv_heads != 0 || q_heads / c.kv_heads > 64) return QMV_ERR_SHAPE;
    // a workgroup of 256 threads for every 16 rows of a head and every sequence
    // (one of 512 only where those fit a launch too: plan_attn)
    const int64_t tiles = b.T * (q_heads / c.kv_heads) / 16 + b.B;
    return tiles * c.kv_heads <= kMaxT ? QMV_OK : QMV_ERR_SHAPE;
}

int check_norm(const float* x, const float* r, const float* w, const float* z, int64_t K, int64_t M, float eps) {
    if (!x || !w) return QMV_ERR_NULL;
    if (K < 1 || K > kMaxInt || M < 1 || M > 65535) return QMV_ERR_SHAPE;
    if (!(eps >= 0.0f) || !(eps <= kMaxFloat)) return QMV_ERR_ARG;
    if (!aligned(x, 4) || !aligned(r, 4) || !aligned(w, 4) || !aligned(z, 4)) return QMV_ERR_ALIGN;
    return QMV_OK;
}

}  // namespace

extern "C" {

int kv_write(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const float* k, int64_t ldk, const float* v,
             int64_t ldv, hipStream_t stream) {
    if (!k || !v) return QMV_ERR_NULL;
    int rc = check_kv(cache, batch);
    const int64_t width = rc ? 0 : static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if (!rc) rc = check_rows(k, ldk, width, batch->T);
    if (!rc) rc = check_rows(v, ldv, width, batch->T);
    if (rc) return rc;
    return launched(qmv::launch_kv_write(*cache, *batch, k, ldk, v, ldv, stream));
}

int kv_read(const qmv_kv_cache* cache, const qmv_kv_batch* batch, float* k, int64_t ldk, float* v, int64_t ldv,
            hipStream_t stream) {
    if (!k || !v) return QMV_ERR_NULL;
    int rc = check_kv(cache, batch);
    const int64_t width = rc ? 0 : static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if (!rc) rc = check_rows(k, ldk, width, batch->T);
    if (!rc) rc = check_rows(v, ldv, width, batch->T);
    if (rc) return rc;
    return launched(qmv::launch_kv_read(*cache, *batch, k, ldk, v, ldv, stream));
}

size_t attn_paged_ws_bytes(const qmv_kv_cache* cache, const qmv_kv_batch* batch, int32_t q_heads) {
    if (!cache || !batch || check_cache_shape(*cache) || check_batch_shape(*cache, *batch) ||
        check_q_heads(*cache, *batch, q_heads))
        return 0;
    return qmv::attn_ws_bytes(*cache, *batch, q_heads);
}

int attn_paged(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const float* q, int64_t ldq, float* out,
               int64_t ldo, int32_t q_heads, float scale, int32_t window, void* ws, size_t ws_bytes,
               hipStream_t stream) {
    if (!q || !out || !ws) return QMV_ERR_NULL;
    int rc = check_kv(cache, batch);
    if (!rc) rc = check_q_heads(*cache, *batch, q_heads);
    const int64_t width = rc ? 0 : static_cast<int64_t>(q_heads) * cache->head_dim;
    if (!rc) rc = check_rows(q, ldq, width, batch->T);
    if (!rc) rc = check_rows(out, ldo, width, batch->T);
    if (rc) return rc;
    if (!(scale >= -kMaxFloat) || !(scale <= kMaxFloat) || window < 0) return QMV_ERR_ARG;
    if (!aligned(ws, 16)) return QMV_ERR_ALIGN;
    if (ws_bytes < attn_paged_ws_bytes(cache, batch, q_heads)) return QMV_ERR_WORKSPACE;
    return launched(qmv::launch_attn(*cache, *batch, q, ldq, out, ldo, q_heads, scale, window, ws, stream));
}

int rmsnorm_add(const float* x, const float* r, const float* w, float* z, float* y, int64_t K, int64_t M, float eps,
                hipStream_t stream) {
    if (!y) return QMV_ERR_NULL;
    const int rc = check_norm(x, r, w, z, K, M, eps);
    if (rc) return rc;
    if (!aligned(y, 4)) return QMV_ERR_ALIGN;
    return launched(qmv::launch_rmsnorm(x, r, w, z, y, nullptr, nullptr, K, M, eps, stream));
}

int rmsnorm_add_q8(const float* x, const float* r, const float* w, float* z, int8_t* q, float* d, int64_t K,
                   int64_t M, float eps, hipStream_t stream) {
    if (!q || !d) return QMV_ERR_NULL;
    const int rc = check_norm(x, r, w, z, K, M, eps);
    if (rc) return rc;
    if (K % 32 != 0) return QMV_ERR_SHAPE;
    if (!aligned(q, 4) || !aligned(d, 4)) return QMV_ERR_ALIGN;
    return launched(qmv::launch_rmsnorm(x, r, w, z, nullptr, q, d, K, M, eps, stream));
}

size_t qmm_q4_0_q8_ws_bytes(int64_t N, int64_t K, int64_t M) { return qmm_q4_0_q8act_ws_bytes(N, K, M); }

int qmm_q4_0_q8(const void* W, const int8_t* q, const float* d, float* y, int64_t N, int64_t K, int64_t M, void* ws,
                size_t ws_bytes, hipStream_t stream) {
    if (!W || !q || !d || !y || !ws) return QMV_ERR_NULL;
    const size_t need = qmm_q4_0_q8act_ws_bytes(N, K, M);
    if (need == 0) return QMV_ERR_SHAPE;
    if (!aligned(W, 16) || !aligned(q, 16) || !aligned(d, 4) || !aligned(y, 4) || !aligned(ws, 16))
        return QMV_ERR_ALIGN;
    if (ws_bytes < need) return QMV_ERR_WORKSPACE;
    return launched(qmv::launch_qmm_q8(W, q, d, y, N, K, M, ws, stream));
}

size_t draft_verify_ws_bytes(int64_t B, int32_t G, int64_t V) {
    if (B < 1 || B > 65535 || G < 1 || G > 64 || V < 1 || V > kMaxInt) return 0;
    return qmv::draft_ws_bytes(B, G, V);
}

int draft_verify(const float* target, int64_t ldt, const float* draft, int64_t ldd, const int32_t* draft_tokens,
                 const int32_t* n_draft, const float* u, int32_t* accepted, int32_t* tokens, int64_t B, int32_t G,
                 int64_t V, float temperature, float softcap, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!target || !draft || !draft_tokens || !u || !accepted || !tokens || !ws) return QMV_ERR_NULL;
    const size_t need = draft_verify_ws_bytes(B, G, V);
    if (need == 0) return QMV_ERR_SHAPE;
    int rc = check_rows(target, ldt, V, B * (G + 1));
    if (!rc) rc = check_rows(draft, ldd, V, B * G);
    if (rc) return rc;
    if (!(temperature > 0.0f) || !(temperature <= kMaxFloat)) return QMV_ERR_ARG;
    if (!(softcap >= 0.0f) || !(softcap <= kMaxCap)) return QMV_ERR_ARG;
    if (!aligned(draft_tokens, 4) || !aligned(n_draft, 4) || !aligned(u, 4) || !aligned(accepted, 4) ||
        !aligned(tokens, 4) || !aligned(ws, 16))
        return QMV_ERR_ALIGN;
    if (ws_bytes < need) return QMV_ERR_WORKSPACE;
    qmv::DraftArgs a;
    a.target = target;
    a.draft = draft;
    a.draft_tokens = draft_tokens;
    a.n_draft = n_draft;
    a.u = u;
    a.accepted = accepted;
    a.tokens = tokens;
    a.ldt = ldt;
    a.ldd = ldd;
    a.V = V;
    a.B = B;
    a.G = G;
    a.temperature = temperature;
    a.softcap = softcap;
    return launched(qmv::launch_draft_verify(a, ws, stream));
}

}  // extern "C"
