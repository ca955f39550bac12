/*
 * qmv_step.h -- C ABI of libqmv.so, second part: what a decode step does
 * around the weight products of qmv.h.
 *
 *   kv_write, kv_read        a paged key/value cache, 8-bit codes with scales
 *                            or float16, written and read back
 *   attn_paged               attention of new tokens over that cache
 *   rmsnorm_add              residual addition and root-mean-square norm
 *   rmsnorm_add_q8           the same with Q8 activation blocks as output
 *   qmm_q4_0_q8              Q4_0 weights times given Q8 activation blocks
 *   draft_verify             drafted tokens against the target's logits
 *
 * The conventions of qmv.h hold: device buffers owned by the caller, no
 * allocation, copy or synchronization, work enqueued on `stream`, every
 * argument that the host can see checked before anything is launched, and
 * the same status codes.  The descriptors below are read during the call
 * only; the buffers they point to must live until the work has run.
 * Calls are reentrant when they share neither outputs nor workspaces; two
 * calls that may run at the same time (on two streams, or captured in two
 * graphs that are replayed together) need workspaces of their own.
 * Output buffers and workspaces must not overlap any input unless said so.
 */
#ifndef QMV_STEP_H
#define QMV_STEP_H

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the paged key/value cache ----
 *
 * Keys and values of a token are kv_heads rows of head_dim elements each.
 * A page holds page_size consecutive positions of one sequence for every
 * head:
 *   k, v             [num_pages][kv_heads][page_size][head_dim] codes
 *   k_scale, v_scale [num_pages][kv_heads][page_size] float32 (QMV_KV_Q8)
 * QMV_KV_Q8:  int8 codes and one scale a row (a token's head), by the rule
 *   of the activation quantizer over the row's head_dim elements:
 *   d = max|x| / 127 (IEEE float32 division),
 *   q = clamp(round_half_away_from_zero(x / d), -127, 127), x ~ q * d;
 *   a row whose d is 0 (all zeros, or no magnitude above 63 2^-149) has q = 0.
 * QMV_KV_F16: IEEE float16 elements (k_scale and v_scale unused, NULL).
 * A row that holds a NaN or infinity (or a magnitude float16 rounds to
 * infinity) is stored as NaN in whole.  Pages filled by other means have to
 * follow this: scales not negative, finite or NaN, rows of float16 finite or
 * NaN in whole.
 * head_dim is 64, 128 or 256; page_size a power of two in [16, 1024].
 * k, v, k_scale and v_scale are 16-byte aligned. */
enum { QMV_KV_Q8 = 0, QMV_KV_F16 = 1 };

typedef struct qmv_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t num_pages;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_size;
    int32_t format;
} qmv_kv_cache;

/* A batch of sequences: rows and where they live in the cache.
 *   page_table [B][max_pages] int32: page j of sequence b holds its
 *     positions [j * page_size, (j + 1) * page_size)
 *   row_start  [B + 1] int32, not decreasing: rows row_start[b] ..
 *     row_start[b + 1] - 1 of the row buffers (T rows) belong to sequence b
 *   kv_len     [B] int32: positions of sequence b, the rows' own included
 * The n = row_start[b + 1] - row_start[b] rows are the LAST n positions of
 * their sequence: row row_start[b] + i has position kv_len[b] - n + i.
 * n may be 0, and so may kv_len; a row whose position is negative (n >
 * kv_len) has no place in the cache.  Rows at or behind row_start[B] belong
 * to no sequence.  A sequence's positions end with its table: positions
 * from max_pages * page_size on have no place.  The contents of the three
 * arrays are checked where they are used, on the device: a page number
 * outside [0, num_pages) is never followed, its positions hold nothing, and
 * row starts out of order leave some or all rows undefined.
 * 1 <= T < 2^24, 1 <= B <= 65535, max_pages * page_size <= 2^30. */
typedef struct qmv_kv_batch {
    const int32_t* page_table;
    const int32_t* row_start;
    const int32_t* kv_len;
    int64_t T;
    int32_t B;
    int32_t max_pages;
} qmv_kv_batch;

/* Quantizes new rows into the cache.  k, v: float32, row r at k + r * ldk
 * (ldk, ldv >= kv_heads * head_dim elements), heads one after the other.
 * Rows without a place are dropped.  Two rows must not have the same place
 * (pages of a shared prefix are read, not written). */
int kv_write(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const float* k, int64_t ldk, const float* v,
             int64_t ldv, hipStream_t stream);

/* Reads rows back as float32: with the batch of a kv_write its rows, with
 * row_start the running sum of kv_len whole sequences.  Rows of a sequence
 * without a place in the cache read as zeros; rows at or behind row_start[B]
 * are left as they were. */
int kv_read(const qmv_kv_cache* cache, const qmv_kv_batch* batch, float* k, int64_t ldk, float* v, int64_t ldv,
            hipStream_t stream);

/* Attention of the batch's rows over the cache (their own keys and values
 * written before).  For query head h of the row at position p, with the
 * key/value head h / (q_heads / kv_heads):
 *   s_j = scale * q . k_j    for the visible positions j: j <= p, and with
 *                            window > 0 also j > p - window
 *   out = sum_j exp(s_j - max s) v_j / sum_j exp(s_j - max s)
 * Row r of q at q + r * ldq, of out at out + r * ldo (ldq, ldo >= q_heads *
 * head_dim).  A row that sees nothing gets zeros; rows at or behind
 * row_start[B] are left as they were.  Positions that a row does not see
 * have no effect on it, whatever they hold.  A row that sees a key or value
 * stored as NaN gets NaN in every dimension of the heads that see it, and so
 * does a query that is not finite.
 * Accuracy: one pass over the keys, with scores, weights p, sums and results
 * in float32, but narrower operands of the products.  A query element is held
 * to 2^-22 of its row's largest magnitude (a score is off by as much of
 * scale * max|q| * sum|k_j|).  A weight is held to 2^-20 of itself (8-bit
 * values beyond [2^-14, 2^16]: 2^-18), or
 *   8-bit values:   2^-34 of the row's largest weight times value scale, so
 *     that a value which weighs nothing takes nothing from the others; weights
 *     below 2^-114 of the largest may count as zero
 *   float16 values: 2^-34 of the row's largest weight, whatever the values:
 *     each position may be off by 2^-34 |v_j|, which matters where values are
 *     seen that are 2^10 or more times those that hold the weight
 * Scores are formed from the codes before they are scaled: 8-bit keys of 2^96
 * and more may overflow there and give NaN, and a row whose scale * max|q| is
 * below 2^-104 loses accuracy (beside keys below 2^72 its scores are 0 to
 * float32 anyway).  8-bit values outside [2^-80, 2^90] lose accuracy.  A row
 * with scores beyond float32 is undefined.
 * q_heads: a multiple of kv_heads, at most 64 times as many, and
 * T * q_heads / 16 + B * kv_heads < 2^24.  scale finite; window >= 0 (0: none).
 * ws: attn_paged_ws_bytes(cache, batch, q_heads) bytes, 16-byte aligned,
 * contents overwritten; the size depends on the descriptors' numbers only,
 * not on the arrays, and is 0 for invalid ones.  So does the split of the
 * work: it takes every sequence to be as long as max_pages allows (or the
 * window), and a table cut to the longest sequence can be a third faster. */
size_t attn_paged_ws_bytes(const qmv_kv_cache* cache, const qmv_kv_batch* batch, int32_t q_heads);
int attn_paged(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const float* q, int64_t ldq, float* out,
               int64_t ldo, int32_t q_heads, float scale, int32_t window, void* ws, size_t ws_bytes,
               hipStream_t stream);

/* ---- the norm between two products ----
 *
 * z = x + r (z = x with r NULL), and y = (z * rstd) * w a row, with
 *   rstd = float32(1 / sqrt(mean(z^2) + eps)),
 * the mean and its root in 64 bits, everything else in float32, so that y is
 * the same bits whatever the order of the sum.  x, r, z, y: float32 [M][K];
 * w: float32 [K].  z may be NULL (not kept), and may be x or r (updated in
 * place); y may not overlap x, r or z.  eps finite and >= 0.  K >= 1 and M as
 * in qmv.h (rmsnorm_add_q8: K % 32 == 0). */
int rmsnorm_add(const float* x, const float* r, const float* w, float* z, float* y, int64_t K, int64_t M, float eps,
                hipStream_t stream);

/* The same with y quantized as qmm_q4_0_q8act quantizes its activations:
 * codes int8 [M][K] (4-byte aligned) and scales float32 [M][K / 32].  A
 * block that is not finite gets the scale NaN, one whose scale is 0 the codes
 * 0 (as in the cache; its products are 0 whatever the codes). */
int rmsnorm_add_q8(const float* x, const float* r, const float* w, float* z, int8_t* q, float* d, int64_t K,
                   int64_t M, float eps, hipStream_t stream);

/* y = W (q d): qmm_q4_0_q8act on activations that are already codes q int8
 * [M][K] (16-byte aligned) and scales d float32 [M][K / 32].  Kernels, grids and results
 * are those of qmm_q4_0_q8act, whose step 1 is replaced by bringing the
 * codes into the layout of step 2 (nothing to do for M == 1).  One set of
 * codes can feed several products. */
size_t qmm_q4_0_q8_ws_bytes(int64_t N, int64_t K, int64_t M);
int qmm_q4_0_q8(const void* W, const int8_t* q, const float* d, float* y, int64_t N, int64_t K, int64_t M, void* ws,
                size_t ws_bytes, hipStream_t stream);

/* ---- drafted tokens ----
 *
 * For each of B sequences with n = n_draft[b] drafted tokens t_0 .. t_{n-1}
 * (n_draft NULL: G each; values are clamped to [0, G]):
 *   p_i = softmax(cap(target[b][i]) / temperature), i <= n
 *   q_i = softmax(cap(draft[b][i]) / temperature),  i < n
 *   draft i is accepted iff u[b][i] * q_i(t_i) < p_i(t_i), up to the first
 *     that is not: accepted[b] = a
 *   the next token is drawn from max(p_a - q_a, 0) if a < n (from p_a if
 *     that is all zero), from p_n if a == n: the first index whose running
 *     sum exceeds u[b][G] times the whole sum
 *   tokens[b] = t_0 .. t_{a-1}, the drawn token, then -1
 * so that the tokens are distributed as the target's own.  Everything is
 * computed in 64 bits; an exponential is taken to 2^-42 of itself, so that
 * decisions within about that of their border may fall either way.
 * cap(y) = softcap * tanh(y / softcap), or y with softcap 0.
 * target: float32 [B][G + 1] rows of V logits, rows ldt elements apart;
 * draft: [B][G] rows, ldd apart; draft_tokens int32 [B][G]; u float32
 * [B][G + 1], each in [0, 1); accepted int32 [B]; tokens int32 [B][G + 1].
 * Logits that are NaN or -infinity weigh nothing, +infinity counts as the
 * largest float32.  A drafted token outside [0, V) is not accepted.  Where
 * p_a has no weight at all the drawn token is -1.
 * 1 <= B <= 65535, 1 <= G <= 64, 1 <= V < 2^31, temperature > 0 and finite,
 * softcap in [0, 65536] (its tanh is taken to 2^-42 of softcap; a larger cap
 * would lose the logits' last bits, and 0 means none).
 * ws: draft_verify_ws_bytes(B, G, V) bytes, 16-byte aligned, overwritten. */
size_t draft_verify_ws_bytes(int64_t B, int32_t G, int64_t V);
int draft_verify(const float* target, int64_t ldt, const float* draft, int64_t ldd, const int32_t* draft_tokens,
                 const int32_t* n_draft, const float* u, int32_t* accepted, int32_t* tokens, int64_t B, int32_t G,
                 int64_t V, float temperature, float softcap, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_STEP_H */
