// Verification of drafted tokens against the target's logits.
//
//   p_i, q_i = softmax(cap(logits) / T) of the target's and the drafter's row i
//   draft i is accepted iff u_i q_i(t_i) < p_i(t_i); at the first that is not
//   (row a) the token is drawn from max(p_a - q_a, 0), else from row n.
//
// A draw is "the first index whose running sum exceeds u times the whole
// sum": among 262,144 borders, sums that are off by 1e-7 would move one past
// the drawn point every few calls.  So weights and sums are taken in 64 bits
// (gfx950's float64 FMA rate equals its float32 rate without packing), and
// neither the order of a sum nor the split over workgroups changes a token.
//
// Three launches:
//   stats  one workgroup per (chunk of a row, row, sequence): maximum and sum
//          of weights of the chunk.  Reads every logit once: this is the
//          traffic.
//   pick   one workgroup per (chunk, sequence): joins the rows' chunks, makes
//          the accept tests, and sums its chunk of the row to draw from.
//   draw   one workgroup a sequence: the chunk that holds the drawn point,
//          then the element.
#include <stdint.h>

#include "qmv_device.h"
#include "qmv_internal.h"
#include "step_internal.h"

namespace qmv {
namespace {

constexpr int kChunk = 4096;                          // logits of one workgroup
constexpr int kPer = kChunk / kBlockThreads;          // 16 a thread
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kNegInf = -__builtin_inff();

// 2^t for t <= 0 (also for t somewhat above): t = n + f with n whole and
// |f| <= 1/2, 2^f by its Taylor series (ln 2)^k / k! up to k = 11, whose next
// term is below 7e-15 of the result.  -infinity gives 0.
__device__ __forceinline__ double exp2_f64(double t) {
    t = fmax(t, -1100.0);
    const double n = rint(t);
    const double f = (t - n) * 0.69314718055994530942;
    double p = 1.0 / 39916800.0;
    p = fma(p, f, 1.0 / 3628800.0);
    p = fma(p, f, 1.0 / 362880.0);
    p = fma(p, f, 1.0 / 40320.0);
    p = fma(p, f, 1.0 / 5040.0);
    p = fma(p, f, 1.0 / 720.0);
    p = fma(p, f, 1.0 / 120.0);
    p = fma(p, f, 1.0 / 24.0);
    p = fma(p, f, 1.0 / 6.0);
    p = fma(p, f, 0.5);
    p = fma(p, f, 1.0);
    p = fma(p, f, 1.0);
    return ldexp(p, static_cast<int>(n));
}

// 1 / x for x in [1, 2^200]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp_f64(double x) {
    double r = __builtin_amdgcn_rcp(x);
    r = fma(fma(-x, r, 1.0), r, r);
    return fma(fma(-x, r, 1.0), r, r);
}

struct Weights {
    double cap;    // softcap, 0: none
    double k;      // log2(e) / temperature
    double twice;  // 2 log2(e) / softcap
    // cap(y) in units of log2: the exponent of a weight up to the row's maximum
    __device__ __forceinline__ double level(float y) const {
        const double v = static_cast<double>(y);
        if (cap == 0.0) return v * k;
        // tanh z = 1 - 2 / (1 + e^(2 z)); beyond |z| = 20 it is +-1 in 64 bits
        const double e = exp2_f64(fmin(fmax(v * twice, -64.0), 64.0));
        return (1.0 - 2.0 * rcp_f64(1.0 + e)) * (cap * k);
    }
    // weight relative to the level `top` of the row's (or chunk's) maximum
    __device__ __forceinline__ double weight(float y, double top) const {
        return y == kNegInf ? 0.0 : exp2_f64(level(y) - top);
    }
};

// NaN weighs nothing; +infinity is the largest float.
__device__ __forceinline__ float clean(float y) { return y == y ? fminf(y, 3.4028234663852886e38f) : kNegInf; }

struct Stat {
    double sum;
    float top;  // largest logit of the chunk, -infinity if none weighs anything
    float pad;
};

struct DraftView {
    DraftArgs a;
    Weights w;
    int chunks;
    Stat* stats;       // [B][2 G + 1][chunks]: target rows 0 .. G, then draft rows
    double* rest;      // [B][chunks]: sums of max(p - q, 0) (or of p for the bonus row)
    double* whole;     // [B][chunks]: sums of p
    __device__ __forceinline__ int drafts(int64_t b) const {
        const int n = a.n_draft ? a.n_draft[b] : a.G;
        return n < 0 ? 0 : (n > a.G ? a.G : n);
    }
    __device__ __forceinline__ const float* row(int64_t b, int r) const {
        return r <= a.G ? a.target + (b * (a.G + 1) + r) * a.ldt : a.draft + (b * a.G + (r - a.G - 1)) * a.ldd;
    }
};

__device__ __forceinline__ float wave_max(float v) {
    for (int o = kWave / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

__device__ __forceinline__ double wave_add(double v) {
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

__device__ __forceinline__ double block_add(double v, double* lds) {
    v = wave_add(v);
    if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kWavesPerBlock; ++i) s += lds[i];
    return s;
}

__global__ __launch_bounds__(kBlockThreads)
void draft_stats_kernel(DraftView D) {
    __shared__ float mx[kWavesPerBlock];
    __shared__ double sm[kWavesPerBlock];
    const int c = blockIdx.x, r = blockIdx.y;
    const int64_t b = blockIdx.z;
    const int n = D.drafts(b);
    if (r <= D.a.G ? r > n : r - D.a.G - 1 >= n) return;  // a row that no draft uses
    const float* y = D.row(b, r);
    const int64_t base = static_cast<int64_t>(c) * kChunk + threadIdx.x;
    float v[kPer];
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t at = base + i * kBlockThreads;
        v[i] = at < D.a.V ? clean(y[at]) : kNegInf;
        top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    if ((threadIdx.x & (kWave - 1)) == 0) mx[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWavesPerBlock; ++i) top = fmaxf(top, mx[i]);
    const double level = D.w.level(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += D.w.weight(v[i], level);
    sum = block_add(sum, sm);
    if (threadIdx.x == 0) {
        Stat* s = D.stats + (b * (2 * D.a.G + 1) + r) * D.chunks + c;
        s->sum = sum;
        s->top = top;
    }
}

// The level of a row's maximum and its sum of weights, joined by one wave.
__device__ __forceinline__ void join_row(const DraftView& D, int64_t b, int r, double* level, double* sum) {
    const Stat* s = D.stats + (b * (2 * D.a.G + 1) + r) * D.chunks;
    const int lane = threadIdx.x & (kWave - 1);
    float top = kNegInf;
    for (int c = lane; c < D.chunks; c += kWave) top = fmaxf(top, s[c].top);
    top = wave_max(top);
    *level = D.w.level(top);
    double z = 0.0;
    for (int c = lane; c < D.chunks; c += kWave)
        if (s[c].top != kNegInf) z += s[c].sum * exp2_f64(D.w.level(s[c].top) - *level);
    *sum = wave_add(z);
}

__device__ __forceinline__ double probability(const DraftView& D, float y, double level, double sum) {
    return sum > 0.0 ? D.w.weight(clean(y), level) / sum : 0.0;
}

// What the draw of a sequence looks at.
struct Pick {
    double p_level, p_sum, q_level, q_sum;
    int accepted;
    int residual;
};

__device__ void pick_row(const DraftView& D, int64_t b, Pick* lds, int* yes) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int n = D.drafts(b), G = D.a.G;
    for (int i = wave; i < n; i += kWavesPerBlock) {
        double pl, ps, ql, qs;
        join_row(D, b, i, &pl, &ps);
        join_row(D, b, G + 1 + i, &ql, &qs);
        const int t = D.a.draft_tokens[b * G + i];
        bool ok = false;
        if (t >= 0 && t < D.a.V) {
            const double p = probability(D, D.row(b, i)[t], pl, ps);
            const double q = probability(D, D.row(b, G + 1 + i)[t], ql, qs);
            ok = static_cast<double>(D.a.u[b * (G + 1) + i]) * q < p;
        }
        if (lane == 0) yes[i] = ok;
    }
    __syncthreads();
    if (wave == 0) {
        const bool no = lane < n && !yes[lane < n ? lane : 0];
        const uint64_t nos = __ballot(no);
        const int a = nos ? __ffsll(static_cast<unsigned long long>(nos)) - 1 : n;
        Pick P;
        P.accepted = a;
        P.residual = a < n;
        join_row(D, b, a, &P.p_level, &P.p_sum);
        P.q_level = P.q_sum = 0.0;
        if (a < n) join_row(D, b, G + 1 + a, &P.q_level, &P.q_sum);
        if (lane == 0) *lds = P;
    }
    __syncthreads();
}

// Weights of 16 consecutive logits of the row to draw from: thread t of the
// workgroup has elements 16 t .. 16 t + 15 of the chunk.  rest: max(p - q, 0)
// (p for the bonus row), whole: p.
__device__ __forceinline__ void weights_of(const DraftView& D, int64_t b, int c, const Pick& P, double (&rest)[kPer],
                                           double (&whole)[kPer]) {
    const float* yp = D.row(b, P.accepted);
    const float* yq = P.residual ? D.row(b, D.a.G + 1 + P.accepted) : yp;
    const int64_t base = static_cast<int64_t>(c) * kChunk + threadIdx.x * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t at = base + i;
        double p = 0.0, q = 0.0;
        if (at < D.a.V) {
            p = probability(D, yp[at], P.p_level, P.p_sum);
            if (P.residual) q = probability(D, yq[at], P.q_level, P.q_sum);
        }
        whole[i] = p;
        rest[i] = fmax(p - q, 0.0);
    }
}

__global__ __launch_bounds__(kBlockThreads)
void draft_pick_kernel(DraftView D) {
    __shared__ Pick P;
    __shared__ int yes[64];
    __shared__ double sa[kWavesPerBlock], sb[kWavesPerBlock];
    const int c = blockIdx.x;
    const int64_t b = blockIdx.y;
    pick_row(D, b, &P, yes);
    double rest[kPer], whole[kPer];
    weights_of(D, b, c, P, rest, whole);
    double x = 0.0, y = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        x += rest[i];
        y += whole[i];
    }
    x = block_add(x, sa);
    y = block_add(y, sb);
    if (threadIdx.x == 0) {
        D.rest[b * D.chunks + c] = x;
        D.whole[b * D.chunks + c] = y;
    }
}

__global__ __launch_bounds__(kBlockThreads)
void draft_draw_kernel(DraftView D) {
    __shared__ Pick P;
    __shared__ int yes[64];
    __shared__ double scan[kBlockThreads];
    __shared__ int found, last;
    const int64_t b = blockIdx.x;
    const int t = threadIdx.x, G = D.a.G;
    pick_row(D, b, &P, yes);
    // the chunk, by one thread: the running sum in index order
    __shared__ int chunk, from_whole;
    __shared__ double target, before;
    if (t == 0) {
        double total = 0.0;
        for (int c = 0; c < D.chunks; ++c) total += D.rest[b * D.chunks + c];
        from_whole = !(total > 0.0);
        const double* s = from_whole ? D.whole + b * D.chunks : D.rest + b * D.chunks;
        if (from_whole) {
            total = 0.0;
            for (int c = 0; c < D.chunks; ++c) total += s[c];
        }
        target = static_cast<double>(D.a.u[b * (G + 1) + G]) * total;
        double run = 0.0;
        chunk = -1;
        before = 0.0;
        for (int c = 0; c < D.chunks; ++c) {
            if (s[c] > 0.0) {
                chunk = c;  // the last chunk with weight, should none pass the point
                before = run;
                if (run + s[c] > target) break;
            }
            run += s[c];
        }
        found = kChunk;
        last = -1;
    }
    __syncthreads();
    int token = -1;
    if (chunk >= 0) {
        double rest[kPer], whole[kPer];
        weights_of(D, b, chunk, P, rest, whole);
        double mine = 0.0;
        int tail = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (from_whole) rest[i] = whole[i];
            mine += rest[i];
            if (rest[i] > 0.0) tail = t * kPer + i;
        }
        scan[t] = mine;
        __syncthreads();
        for (int o = 1; o < kBlockThreads; o <<= 1) {
            const double v = t >= o ? scan[t - o] : 0.0;
            __syncthreads();
            scan[t] += v;
            __syncthreads();
        }
        double run = before + (t ? scan[t - 1] : 0.0);
        int hit = kChunk;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            run += rest[i];
            if (hit == kChunk && rest[i] > 0.0 && run > target) hit = t * kPer + i;
        }
        if (hit < kChunk) atomicMin(&found, hit);
        if (tail >= 0) atomicMax(&last, tail);
        __syncthreads();
        const int at = found < kChunk ? found : last;
        token = at < 0 ? -1 : static_cast<int>(static_cast<int64_t>(chunk) * kChunk + at);
    }
    const int a = P.accepted;
    if (t == 0) D.a.accepted[b] = a;
    for (int i = t; i <= G; i += kBlockThreads)
        D.a.tokens[b * (G + 1) + i] = i < a ? D.a.draft_tokens[b * G + i] : (i == a ? token : -1);
}

int64_t chunks_of(int64_t V) { return (V + kChunk - 1) / kChunk; }
size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t draft_ws_bytes(int64_t B, int G, int64_t V) {
    const size_t n = static_cast<size_t>(B) * static_cast<size_t>(chunks_of(V));
    return align256(n * static_cast<size_t>(2 * G + 1) * sizeof(Stat)) + 2 * align256(n * sizeof(double));
}

hipError_t launch_draft_verify(const DraftArgs& a, void* ws, hipStream_t stream) {
    DraftView D;
    D.a = a;
    D.w.cap = a.softcap;
    D.w.k = kLog2e / static_cast<double>(a.temperature);
    D.w.twice = a.softcap > 0.0f ? 2.0 * kLog2e / static_cast<double>(a.softcap) : 0.0;
    D.chunks = static_cast<int>(chunks_of(a.V));
    const size_t n = static_cast<size_t>(a.B) * static_cast<size_t>(D.chunks);
    char* p = static_cast<char*>(ws);
    D.stats = reinterpret_cast<Stat*>(p);
    p += align256(n * static_cast<size_t>(2 * a.G + 1) * sizeof(Stat));
    D.rest = reinterpret_cast<double*>(p);
    D.whole = reinterpret_cast<double*>(p + align256(n * sizeof(double)));
    const unsigned ch = static_cast<unsigned>(D.chunks), B = static_cast<unsigned>(a.B);
    hipLaunchKernelGGL(draft_stats_kernel, dim3(ch, static_cast<unsigned>(2 * a.G + 1), B), dim3(kBlockThreads), 0,
                       stream, D);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draft_pick_kernel, dim3(ch, B), dim3(kBlockThreads), 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draft_draw_kernel, dim3(B), dim3(kBlockThreads), 0, stream, D);
    return hipGetLastError();
}

}  // namespace qmv
