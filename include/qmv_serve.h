/*
 * qmv_serve.h -- C ABI of libqmv.so, third part: the two ends of a serving
 * step, and the adapters in its middle.
 *
 *   kv_plan                  cache pages, row starts, positions and slots of
 *                            a step, from the sequences' lengths
 *   embed_q8_0, embed_q4_0,  rows of a quantized embedding table, scaled
 *   embed_q4_k, embed_q6_k
 *   lora_add                 each sequence's own low-rank adapter added to a
 *                            shared projection's output
 *   logits_draw              temperature, top-k, top-p and min-p of each row
 *                            over the whole vocabulary, and a draw
 *
 * With them a decode loop (plan, embed, norms, products and adapters, cache,
 * attention, logits, draw) needs nothing from the host between two tokens and
 * can be captured in a graph.
 *
 * The conventions of qmv.h and qmv_step.h hold: device buffers owned by the
 * caller, no allocation, copy or synchronization, work enqueued on `stream`,
 * every argument that the host can see checked before anything is launched,
 * the same status codes.  Descriptors are read during the call only.  Calls
 * are reentrant when they share neither outputs nor workspaces; two calls
 * that may run at the same time need workspaces of their own.  Outputs and
 * workspaces must not overlap any input unless said so.
 */
#ifndef QMV_SERVE_H
#define QMV_SERVE_H

#include "qmv_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- planning a step ----
 *
 * The pages of a paged cache (qmv_step.h) that belong to sequences, and those
 * that are free:
 *   page_table [B][max_pages] int32: page j of sequence b; the first
 *     P(length) entries of a row are its pages, P(x) = ceil(x / page_size),
 *     the others hold anything
 *   free_pages [num_pages] int32: a stack; its first *free_count entries are
 *     the free pages, the last of them on top
 * 1 <= B <= 65535, 1 <= num_pages < 2^31, page_size a power of two in
 * [16, 1024], max_pages * page_size <= 2^30. */
typedef struct qmv_kv_pool {
    int32_t* page_table;
    int32_t* free_pages;
    int64_t num_pages;
    int32_t B;
    int32_t max_pages;
    int32_t page_size;
} qmv_kv_pool;

/* Every sequence is cut to keep[b] of its kv_len[b] positions and grows by
 * n_new[b] rows: new_len[b] = keep[b] + n_new[b] (keep NULL: nothing is cut).
 * A sequence that goes on decoding has keep = kv_len; after rejected drafts
 * keep is smaller; one that ends has keep = n_new = 0, and a new one kv_len =
 * 0.  In the order of the sequences, and of positions within one:
 *   - pages that a sequence no longer needs, P(new_len) .. P(kv_len) - 1 of
 *     its table, are pushed onto the stack,
 *   - then pages that it needs, P(kv_len) .. P(new_len) - 1, are popped from
 *     the stack into its table (a sequence does one or the other).
 * A page is moved as the number that it is: a table that holds -1 gives back
 * -1.  Outputs:
 *   new_len   [B] int32 (may be kv_len or keep)
 *   new_count [1] int32 (may be free_count): free pages after the step
 *   row_start [B + 1] int32: the running sum of n_new
 *   position  [T] int32 (or NULL): row row_start[b] + i has keep[b] + i
 *   slot      [T] int64 (or NULL): page * page_size + position % page_size,
 *             the row's place in one plane of a head, -1 where the page is
 *             outside [0, num_pages)
 *   status    [2] int32: 0 and 0, or why nothing was done, as a sum of
 *     QMV_PLAN_PAGES  the stack has too few pages; status[1] how many
 *     QMV_PLAN_ROWS   more than T rows
 *     QMV_PLAN_LENGTH a number is negative, keep is larger than kv_len, or
 *                     kv_len or new_len larger than max_pages * page_size
 *     QMV_PLAN_STACK  free_count is outside [0, num_pages], or with the pages
 *                     given back it would be
 * row_start, new_len (and the tables) are what qmv_kv_batch takes next.  The
 * step is done in whole or not at all: with status[0] != 0 new_len is kv_len
 * and new_count free_count, every row start is 0 (so that what follows has no
 * rows), and tables and stack are as they were.  A sequence whose length is
 * out of range counts for nothing here, and pages are not counted with
 * QMV_PLAN_STACK.  Rows from row_start[B] on are left as they
 * were, and so are table entries behind the new length; stack entries from
 * new_count on are unspecified.
 * 1 <= T < 2^24.
 * ws: kv_plan_ws_bytes(pool) bytes, 16-byte aligned, contents overwritten. */
enum { QMV_PLAN_PAGES = 1, QMV_PLAN_ROWS = 2, QMV_PLAN_LENGTH = 4, QMV_PLAN_STACK = 8 };
size_t kv_plan_ws_bytes(const qmv_kv_pool* pool);
int kv_plan(const qmv_kv_pool* pool, const int32_t* kv_len, const int32_t* keep, const int32_t* n_new,
            const int32_t* free_count, int32_t* new_len, int32_t* new_count, int32_t* row_start, int32_t* position,
            int64_t* slot, int32_t* status, int64_t T, void* ws, size_t ws_bytes, hipStream_t stream);

/* ---- embedding rows ----
 *
 * y[m] = scale * W[tokens[m]], W: N rows of K weights in the layouts of
 * qmv.h (the table of a tied logit projection serves both), tokens int32 [M],
 * y float32 [M][K].  A weight is formed in float32 as qmv.h defines it (exact
 * but for Q4_K, whose difference is rounded once) and multiplied by scale.  A
 * token outside [0, N) gives zeros.  1 <= N < 2^31, 1 <= M < 2^24, K a
 * positive number of whole blocks below 2^31, scale finite, W 16-byte
 * aligned. */
int embed_q8_0(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream);
int embed_q4_0(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream);
int embed_q4_k(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream);
int embed_q6_k(const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M, float scale,
               hipStream_t stream);

/* ---- low-rank adapters ----
 *
 * `slots` adapters of one projection, K inputs and N outputs:
 *   A     [slots][max_rank][K], Bm [slots][N][max_rank]: float16 or bfloat16
 *   rank  [slots] int32 or NULL (max_rank each): only the first rank[s] rows
 *         of A and columns of Bm count, whatever the others hold; values are
 *         clamped to [0, max_rank]
 *   scale [slots] float32
 * max_rank a multiple of 8 in [8, 256], K a multiple of 8, K, N < 2^24,
 * slots < 2^20; A and Bm are 16-byte aligned. */
enum { QMV_LORA_F16 = 0, QMV_LORA_BF16 = 1 };

typedef struct qmv_lora {
    const void* A;
    const void* Bm;
    const int32_t* rank;
    const float* scale;
    int64_t K;
    int64_t N;
    int32_t slots;
    int32_t max_rank;
    int32_t format;
} qmv_lora;

/* y_r = base_r + scale[s] * Bm[s] (A[s] x_r) for the rows r of sequence b
 * (row_start[b] .. row_start[b + 1] - 1, as in qmv_kv_batch) with s =
 * adapter[b]; y_r = base_r where adapter[b] is outside [0, slots).
 * x float32, row r at x + r * ldx (ldx >= K); base (or NULL: zeros) and y
 * likewise with N.  base may be y, with ldb = ldy: then the product's output is
 * updated in place, and rows without an adapter are not touched.  Rows before
 * row_start[0] (of a part of a batch) and at or behind row_start[B] are left as
 * they were.  Weights enter as they are, x and all sums are float32.  row_start and adapter are checked where they are used:
 * row starts out of order leave rows undefined.
 * 1 <= B <= 65535, 1 <= T < 2^24.
 * ws: lora_add_ws_bytes(lora, B, T) bytes, 16-byte aligned, overwritten.  They do
 * not fall as B or T grows: what serves a batch serves every smaller one. */
size_t lora_add_ws_bytes(const qmv_lora* lora, int64_t B, int64_t T);
int lora_add(const qmv_lora* lora, const int32_t* adapter, const int32_t* row_start, const float* x, int64_t ldx,
             const float* base, int64_t ldb, float* y, int64_t ldy, int64_t B, int64_t T, void* ws, size_t ws_bytes,
             hipStream_t stream);

/* ---- a filtered draw ----
 *
 * For each of M rows of V logits z (row m at logits + m * ldl), ordered by
 * larger logit first and equal ones by the lower index:
 *   w_i = exp((cap(z_i) - cap(z_0)) / temperature[m])   (w_0 = 1)
 *   the first n are kept, n the smallest of
 *     top_k[m], if positive,
 *     the smallest count whose sum of w reaches top_p[m] times the sum over
 *       the first top_k, if top_p[m] < 1,
 *     the number with w_i >= min_p[m], if positive,
 *     the number of logits that can be kept at all,
 *   but at least 1
 *   token[m] = the first whose running sum exceeds u[m] times the sum of
 *     the n kept;  kept[m] = n
 * temperature[m] = 0 (or anything not above 0) takes the first, n = 1.
 * top_k, top_p, min_p (float32; top_k int32) may each be NULL: no such filter;
 * kept may be NULL.  cap(y) = softcap * tanh(y / softcap), or y with softcap 0.
 * u float32 in [0, 1) (from 1 on the last kept one with weight, below 0 the
 * first).  Logits that are NaN or -infinity weigh nothing and are not kept,
 * +infinity counts as the largest float32.  A row without any other logit has
 * token -1, kept 0.
 * Weights are rounded to whole multiples of 2^-q, 2^q the largest power of two
 * up to 2^51 with V 2^q <= 2^62 (q = 44 for 262,144), and sums of them are exact:
 * the result does not depend on the order of a sum.  An exponential is taken to 2^-42 of itself
 * (tanh to 2^-42 of softcap), so that decisions within about that of their
 * border may fall either way.
 * 1 <= M <= 65535, 1 <= V < 2^31, softcap in [0, 65536].
 * ws: logits_draw_ws_bytes(V, M) bytes, 16-byte aligned, overwritten.  They do
 * not fall as V or M grows: what serves a batch serves every smaller one. */
size_t logits_draw_ws_bytes(int64_t V, int64_t M);
int logits_draw(const float* logits, int64_t ldl, const float* temperature, const int32_t* top_k, const float* top_p,
                const float* min_p, const float* u, int32_t* token, int32_t* kept, int64_t V, int64_t M, float softcap,
                void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_SERVE_H */
