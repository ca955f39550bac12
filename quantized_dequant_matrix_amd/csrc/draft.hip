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
//   stats  one workgroup per (chunk of 4096 logits, row, sequence): maximum
//          and sum of weights of the chunk.  Reads every logit once: this is
//          the traffic.
//   pick   one workgroup per (part, sequence): joins the rows' chunks, makes
//          the accept tests, and sums groups of 256 weights of the row to draw
//          from, a wave each.  A part is 2048 logits or a few times that.
//   draw   one workgroup a sequence: the group that holds the drawn point,
//          then the element.
#include <stdint.h>

#include "qmv_device.h"
#include "qmv_internal.h"
#include "step_device.h"
#include "step_internal.h"

namespace qmv {
namespace {

constexpr int kStatThreads = 256, kStatWaves = kStatThreads / kWave;
constexpr int kChunk = 4096;                     // logits of a workgroup of the stats kernel
constexpr int kPickThreads = 512, kPickWaves = kPickThreads / kWave;
constexpr int kStep = 2048;                      // logits of one step of a workgroup of the pick kernel
constexpr int kGroup = kStep / kPickWaves;       // 256: a wave's share of a step
constexpr int kDrawThreads = kGroup, kDrawWaves = kDrawThreads / kWave;
constexpr int kHeld = 4;
constexpr int kMaxRows = 2 * 64 + 1;        // rows of a sequence: G + 1 target rows, G draft rows
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kNegInf = -__builtin_inff();

// 2^(j / 256), j < 256, in LDS: filled by the first 256 threads of a
// workgroup before its first barrier.
__shared__ double exp_table[256];

__device__ __forceinline__ void fill_exp_table() {
    if (threadIdx.x < 256) {
        // (ln 2 / 256) j by the series up to the 17th power: below 2^-54 left
        const double x = static_cast<double>(threadIdx.x) * (0.69314718055994530942 / 256.0);
        double p = 1.0;
#pragma unroll
        for (int k = 17; k >= 1; --k) p = fma(p * x, 1.0 / k, 1.0);
        exp_table[threadIdx.x] = p;
    }
}

// 2^t for t <= 64: t = n + j / 256 + f, |f| <= 1/512, with n + j / 256
// rounded off by an addition of 1.5 2^44 (whose last place is 1/256),
// 2^(j / 256) from the table and 2^f by its series up to the third power,
// whose next term is below 2e-13.  Below 2^-1020 the result is 0 (the row's
// maximum is 2^0).  About 23 instructions a weight with the sum, no branch: with
// 31 (a longer series, a table of 64) the sums of 371 MB of logits took 104 us,
// now 81-90.
__device__ __forceinline__ double exp2_f64(double t, bool none = false) {
    none |= t < -1020.0;
    t = fmax(t, -1020.0);
    constexpr double kShift = 26388279066624.0, kLn2 = 0.69314718055994530942;
    const double r = t + kShift;
    const uint32_t k = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, r));  // 256 n + j
    const double f = t - (r - kShift);
    const double q = fma(fma(kLn2 * kLn2 * kLn2 / 6.0, f, kLn2 * kLn2 / 2.0), f, kLn2);
    const double e = exp_table[k & 255u];
    const uint64_t v = __builtin_bit_cast(uint64_t, fma(q * f, e, e));
    const uint32_t hi = static_cast<uint32_t>(v >> 32) + ((k & ~255u) << 12);
    const double x = __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | static_cast<uint32_t>(v));
    return none ? 0.0 : x;
}

// 1 / x for x in [1, 2^200]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp_f64(double x) {
    double r = __builtin_amdgcn_rcp(x);
    r = fma(fma(-x, r, 1.0), r, r);
    return fma(fma(-x, r, 1.0), r, r);
}

struct Weights {
    double cap;    // softcap / temperature in units of log2, 0: none
    double k;      // log2(e) / temperature
    double twice;  // 2 log2(e) / softcap
    // What exponents are differences of: the logit, or its capped value over
    // the cap.
    template <bool CAP>
    __device__ __forceinline__ double level(float y) const {
        const double v = static_cast<double>(y);
        if constexpr (!CAP) return v;
        // tanh z = 1 - 2 / (1 + e^(2 z)); beyond |z| = 20 it is +-1 in 64 bits
        const double e = exp2_f64(fmin(fmax(v * twice, -64.0), 64.0));
        return fma(-2.0, rcp_f64(1.0 + e), 1.0);
    }
    // A weight's exponent below the level `top`, in units of log2.  The
    // difference first: of two logits it is exact, so the largest has weight 1
    // and rows that differ by a constant have the same weights, bit for bit.
    // Logits are bounded: their differences times k stay finite.
    template <bool CAP>
    __device__ __forceinline__ double below(double level, double top) const {
#pragma clang fp contract(off)
        return (level - top) * (CAP ? cap : k);
    }
    // weight relative to the level `top` of the row's (or chunk's) maximum;
    // no branches, so that a thread's weights overlap
    template <bool CAP>
    __device__ __forceinline__ double weight(float y, double top) const {
        return exp2_f64(below<CAP>(level<CAP>(y), top), CAP && y == kNegInf);
    }
};

// +infinity counts as the largest float; NaN weighs nothing: v_med3_f32 with
// a quiet NaN gives the smallest of the other two (the compiler's own median
// drops the -infinity as an identity).  A signalling NaN is quieted first:
// the median would do that itself and then drop the -infinity.
__device__ __forceinline__ float clean(float y) {
    y = __builtin_canonicalizef(y);
    float r;
    asm("v_med3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(y), "v"(kNegInf), "v"(3.4028234663852886e38f));
    return r;
}

struct Stat {
    double sum;
    float top;  // largest logit of the chunk, -infinity if none weighs anything
    float pad;
};

// What the draw of a sequence looks at.
struct Pick {
    double p_level, p_inv, q_level, q_inv;  // levels of the rows' maxima, 1 / sums (0: no weight)
    int accepted;
    int residual;  // the row is one of the drafts' (else the bonus row)
};

struct DraftView {
    DraftArgs a;
    Weights w;
    int chunks, groups;
    bool vec;      // rows of logits are 16-byte aligned
    Stat* stats;   // [B][2 G + 1][chunks]: target rows 0 .. G, then draft rows
    double* rest;  // [B][groups]: sums of max(p - q, 0) (of p for the bonus row)
    double* whole; // [B][groups]: sums of p
    Pick* picks;   // [B]
    __device__ __forceinline__ int drafts(int64_t b) const {
        const int n = a.n_draft ? a.n_draft[b] : a.G;
        return n < 0 ? 0 : (n > a.G ? a.G : n);
    }
    __device__ __forceinline__ const float* row(int64_t b, int r) const {
        return r <= a.G ? a.target + (b * (a.G + 1) + r) * a.ldt : a.draft + (b * a.G + (r - a.G - 1)) * a.ldd;
    }
};

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_max(float v) {
    const int bits = __builtin_bit_cast(int, v);
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(bits, bits, CTRL, ROW_MASK, 0xF, false)));
}

__device__ __forceinline__ float wave_max(float v) {
    v = dpp_max<0x111, 0xF>(v);
    v = dpp_max<0x112, 0xF>(v);
    v = dpp_max<0x114, 0xF>(v);
    v = dpp_max<0x118, 0xF>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), kWave - 1));
}

// PER logits a lane of the 64 PER from `base` on, 4 by 4 across the wave (a
// sum's order is free), as they are; past the row's end: no weight.
template <int PER>
__device__ __forceinline__ void load_spread(const DraftView& D, const float* y, int64_t base, float (&v)[PER]) {
    const int lane = threadIdx.x & (kWave - 1);
    if (D.vec && base + PER * kWave <= D.a.V) {  // all loads first
        float4 f[PER / 4];
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) f[i] = *reinterpret_cast<const float4*>(y + base + (i * kWave + lane) * 4);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            v[4 * i] = f[i].x; v[4 * i + 1] = f[i].y; v[4 * i + 2] = f[i].z; v[4 * i + 3] = f[i].w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {  // past the end: the last one again, then taken out
            const int64_t at = base + i * kWave + lane;
            v[i] = y[at < D.a.V ? at : D.a.V - 1];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = base + i * kWave + lane < D.a.V ? v[i] : kNegInf;
    }
}

template <bool CAP>
__global__ __launch_bounds__(kStatThreads)
void draft_stats_kernel(DraftView D) {
    __shared__ float mx[kStatWaves];
    __shared__ double sm[kStatWaves];
    constexpr int kPer = kChunk / kStatThreads;
    const int c = blockIdx.x, r = blockIdx.y;
    const int64_t b = blockIdx.z;
    const int n = D.drafts(b);
    if (r <= D.a.G ? r > n : r - D.a.G - 1 >= n) return;  // a row that no draft uses
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    float v[kPer];
    load_spread(D, D.row(b, r), static_cast<int64_t>(c) * kChunk + wave * (kPer * kWave), v);
    fill_exp_table();
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = clean(v[i]);
        top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    if (lane == 0) mx[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStatWaves; ++i) top = fmaxf(top, mx[i]);
    const double level = D.w.template level<CAP>(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += D.w.template weight<CAP>(v[i], level);
    sum = wave_add(sum);
    if (lane == 0) sm[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < kStatWaves; ++i) sum += sm[i];
        Stat* s = D.stats + (b * (2 * D.a.G + 1) + r) * D.chunks + c;
        s->sum = sum;
        s->top = top;
    }
}

// The level of a row's maximum and its sum of weights, joined by one wave.
template <bool CAP>
__device__ __forceinline__ void join_row(const DraftView& D, int64_t b, int r, double* level, double* sum) {
    const Stat* s = D.stats + (b * (2 * D.a.G + 1) + r) * D.chunks;
    const int lane = threadIdx.x & (kWave - 1);
    Stat first = {0.0, kNegInf, 0.0f};  // a wave's worth of chunks stays in registers
    if (lane < D.chunks) first = s[lane];
    float top = first.top;
    for (int c = lane + kWave; c < D.chunks; c += kWave) top = fmaxf(top, s[c].top);
    top = wave_max(top);
    *level = D.w.template level<CAP>(top);
    double z = first.top != kNegInf ? first.sum * exp2_f64(D.w.template below<CAP>(D.w.template level<CAP>(first.top), *level)) : 0.0;
    for (int c = lane + kWave; c < D.chunks; c += kWave)
        if (s[c].top != kNegInf) z += s[c].sum * exp2_f64(D.w.template below<CAP>(D.w.template level<CAP>(s[c].top), *level));
    *sum = wave_add(z);
}

__device__ __forceinline__ double inverse(double sum) { return sum > 0.0 ? 1.0 / sum : 0.0; }

// max(p - q, 0) of two weights and their rows' 1 / sums.  Both products are
// rounded before the difference: equal rows leave zero, and not the rounding
// of a product that one fused multiply-add would leave.
__device__ __forceinline__ double residual(double wp, double p_inv, double wq, double q_inv) {
#pragma clang fp contract(off)
    const double p = wp * p_inv, q = wq * q_inv;
    return fmax(p - q, 0.0);
}

template <bool CAP, int STEPS>
__global__ __launch_bounds__(kPickThreads)
void draft_pick_kernel(DraftView D) {
    __shared__ double levels[kMaxRows], inverses[kMaxRows];
    __shared__ Pick P;
    const int part = blockIdx.x;
    const int64_t b = blockIdx.y;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int n = D.drafts(b), G = D.a.G;
    // the drafted tokens' logits, by the wave that tests them
    float yp = kNegInf, yq = kNegInf, u = 0.0f;
    bool real = false;
    if (wave == 0 && lane < n) {
        const int t = D.a.draft_tokens[b * G + lane];
        u = D.a.u[b * (G + 1) + lane];
        real = t >= 0 && t < D.a.V;
        if (real) {
            yp = clean(D.row(b, lane)[t]);
            yq = clean(D.row(b, G + 1 + lane)[t]);
        }
    }
    fill_exp_table();
    __syncthreads();
    for (int i = wave; i < 2 * n + 1; i += kPickWaves) {
        const int r = i <= n ? i : G + i - n;  // target rows 0 .. n, draft rows G + 1 ..
        double level, sum;
        join_row<CAP>(D, b, r, &level, &sum);
        if (lane == 0) {
            levels[r] = level;
            inverses[r] = inverse(sum);
        }
    }
    __syncthreads();
    if (wave == 0) {
        bool no = false;
        if (lane < n) {
            const double p = D.w.template weight<CAP>(yp, levels[lane]) * inverses[lane];
            const double q = D.w.template weight<CAP>(yq, levels[G + 1 + lane]) * inverses[G + 1 + lane];
            no = !(real && static_cast<double>(u) * q < p);
        }
        const uint64_t nos = __ballot(no);
        const int a = nos ? __ffsll(static_cast<unsigned long long>(nos)) - 1 : n;
        if (lane == 0) {
            P.accepted = a;
            P.residual = a < n;
            P.p_level = levels[a];
            P.p_inv = inverses[a];
            P.q_level = a < n ? levels[G + 1 + a] : 0.0;
            P.q_inv = a < n ? inverses[G + 1 + a] : 0.0;
            if (part == 0) D.picks[b] = P;
        }
    }
    __syncthreads();
    constexpr int kPer = kGroup / kWave;
    const float* row_p = D.row(b, P.accepted);
    const float* row_q = D.row(b, P.residual ? G + 1 + P.accepted : P.accepted);
    float vp[STEPS][kPer], vq[STEPS][kPer];
    const int64_t group0 = static_cast<int64_t>(part) * STEPS * kPickWaves + wave;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {  // all loads first
        const int64_t base = (group0 + i * kPickWaves) * kGroup;
        load_spread(D, row_p, base, vp[i]);
        if (P.residual) load_spread(D, row_q, base, vq[i]);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t group = group0 + i * kPickWaves;
        double x = 0.0, y = 0.0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const double w = D.w.template weight<CAP>(clean(vp[i][e]), P.p_level);
            y += w * P.p_inv;
            if (P.residual) x += residual(w, P.p_inv, D.w.template weight<CAP>(clean(vq[i][e]), P.q_level), P.q_inv);
        }
        y = wave_add(y);
        x = P.residual ? wave_add(x) : y;
        if (lane == 0 && group < D.groups) {
            D.rest[b * D.groups + group] = x;
            D.whole[b * D.groups + group] = y;
        }
    }
}

// A running sum over the workgroup's threads, in order: the sum before this
// thread, and the whole.
__device__ __forceinline__ double block_prefix(double mine, double* lds, double* total) {
    const double upto = wave_prefix(mine);
    const int wave = threadIdx.x / kWave;
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == kWave - 1) lds[wave] = upto;
    __syncthreads();
    double before = upto - mine;
    *total = 0.0;
#pragma unroll
    for (int i = 0; i < kDrawWaves; ++i) {
        if (i < wave) before += lds[i];
        *total += lds[i];
    }
    return before;
}

template <bool CAP>
__global__ __launch_bounds__(kDrawThreads)
void draft_draw_kernel(DraftView D) {
    __shared__ double sums[kDrawWaves];
    __shared__ int found, last;
    __shared__ double before_group;
    const int64_t b = blockIdx.x;
    const int t = threadIdx.x, G = D.a.G;
    const Pick P = D.picks[b];
    const double u = static_cast<double>(D.a.u[b * (G + 1) + G]);
    fill_exp_table();
    const int per = (D.groups + kDrawThreads - 1) / kDrawThreads;
    const int g0 = min(t * per, D.groups), g1 = min(g0 + per, D.groups);
    int group = -1;
    double target = 0.0;
    bool minus = P.residual;
    // the group: the first whose running sum exceeds u times the whole, or
    // the last with any weight.  No rest anywhere: from p itself.
    for (int pass = 0; pass < 2; ++pass) {
        const double* s = (pass == 0 ? D.rest : D.whole) + b * D.groups;
        double mine = 0.0, total;
        int tail = -1;
        // a thread's first sums stay in registers for the search (all of
        // them up to 262,144 logits)
        double held[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = g0 + i < g1 ? s[g0 + i] : 0.0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            mine += held[i];
            tail = held[i] > 0.0 ? g0 + i : tail;
        }
#pragma unroll 4
        for (int g = g0 + kHeld; g < g1; ++g) {
            const double v = s[g];
            mine += v;
            tail = v > 0.0 ? g : tail;
        }
        double run = block_prefix(mine, sums, &total);
        if (!(total > 0.0)) {
            minus = false;
            continue;
        }
        target = u * total;
        if (t == 0) {
            found = INT32_MAX;
            last = -1;
        }
        __syncthreads();
        int hit = INT32_MAX;
        double from = run;
        if (run + mine > target) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                if (hit == INT32_MAX && held[i] > 0.0 && run + held[i] > target) {
                    hit = g0 + i;
                    from = run;
                }
                run += held[i];
            }
            for (int g = g0 + kHeld; g < g1 && hit == INT32_MAX; ++g) {
                const double v = s[g];
                if (v > 0.0 && run + v > target) {
                    hit = g;
                    from = run;
                }
                run += v;
            }
        }
        if (hit != INT32_MAX) atomicMin(&found, hit);
        if (tail >= 0) atomicMax(&last, tail);
        __syncthreads();
        group = found != INT32_MAX ? found : last;
        if (hit == group) before_group = from;
        // the point lies at the very end: nothing in the last group passes it
        // and its last element with weight is drawn
        if (found == INT32_MAX && t == 0) before_group = 0.0;
        __syncthreads();
        break;
    }
    int token = -1;
    if (group >= 0) {
        // thread t has element t of the group
        const int64_t at_v = static_cast<int64_t>(group) * kGroup + t;
        double weight = 0.0, total;
        if (at_v < D.a.V) {
            const float yp = clean(D.row(b, P.accepted)[at_v]);
            const float yq = minus ? clean(D.row(b, G + 1 + P.accepted)[at_v]) : 0.0f;
            const double w = D.w.template weight<CAP>(yp, P.p_level);
            weight = minus ? residual(w, P.p_inv, D.w.template weight<CAP>(yq, P.q_level), P.q_inv) : w * P.p_inv;
        }
        const double run = before_group + block_prefix(weight, sums, &total) + weight;
        if (t == 0) {
            found = kGroup;
            last = -1;
        }
        __syncthreads();
        if (weight > 0.0) {
            if (run > target) atomicMin(&found, t);
            atomicMax(&last, t);
        }
        __syncthreads();
        const int at = found < kGroup ? found : last;
        token = at < 0 ? -1 : static_cast<int>(static_cast<int64_t>(group) * kGroup + at);
    }
    const int a = P.accepted;
    if (t == 0) D.a.accepted[b] = a;
    for (int i = t; i <= G; i += kDrawThreads)
        D.a.tokens[b * (G + 1) + i] = i < a ? D.a.draft_tokens[b * G + i] : (i == a ? token : -1);
}

int64_t chunks_of(int64_t V) { return (V + kChunk - 1) / kChunk; }
int64_t groups_of(int64_t V) { return (V + kGroup - 1) / kGroup; }

template <bool CAP>
hipError_t launch_draft(const DraftView& D, hipStream_t stream) {
    const unsigned ch = static_cast<unsigned>(D.chunks), B = static_cast<unsigned>(D.a.B);
    // Every workgroup of the pick kernel joins the rows' chunks again: it
    // takes four steps where that leaves enough workgroups for all CUs.
    const int64_t steps = (D.a.V + kStep - 1) / kStep;
    const bool few = steps * D.a.B < 2048;
    const unsigned parts = static_cast<unsigned>(few ? steps : (steps + 3) / 4);
    hipLaunchKernelGGL(draft_stats_kernel<CAP>, dim3(ch, static_cast<unsigned>(2 * D.a.G + 1), B), dim3(kStatThreads), 0,
                       stream, D);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (few)
        hipLaunchKernelGGL((draft_pick_kernel<CAP, 1>), dim3(parts, B), dim3(kPickThreads), 0, stream, D);
    else
        hipLaunchKernelGGL((draft_pick_kernel<CAP, 4>), dim3(parts, B), dim3(kPickThreads), 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draft_draw_kernel<CAP>, dim3(B), dim3(kDrawThreads), 0, stream, D);
    return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t draft_ws_bytes(int64_t B, int G, int64_t V) {
    const size_t b = static_cast<size_t>(B);
    return align256(b * static_cast<size_t>(chunks_of(V)) * static_cast<size_t>(2 * G + 1) * sizeof(Stat)) +
           2 * align256(b * static_cast<size_t>(groups_of(V)) * sizeof(double)) + align256(b * sizeof(Pick));
}

hipError_t launch_draft_verify(const DraftArgs& a, void* ws, hipStream_t stream) {
    DraftView D;
    D.a = a;
    D.w.k = kLog2e / static_cast<double>(a.temperature);
    D.w.cap = static_cast<double>(a.softcap) * D.w.k;
    D.w.twice = a.softcap > 0.0f ? 2.0 * kLog2e / static_cast<double>(a.softcap) : 0.0;
    D.chunks = static_cast<int>(chunks_of(a.V));
    D.groups = static_cast<int>(groups_of(a.V));
    const size_t b = static_cast<size_t>(a.B);
    char* p = static_cast<char*>(ws);
    D.stats = reinterpret_cast<Stat*>(p);
    p += align256(b * static_cast<size_t>(D.chunks) * static_cast<size_t>(2 * a.G + 1) * sizeof(Stat));
    D.rest = reinterpret_cast<double*>(p);
    p += align256(b * static_cast<size_t>(D.groups) * sizeof(double));
    D.whole = reinterpret_cast<double*>(p);
    D.picks = reinterpret_cast<Pick*>(p + align256(b * static_cast<size_t>(D.groups) * sizeof(double)));
    D.vec = ((reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) & 15) == 0 &&
            a.ldt % 4 == 0 && a.ldd % 4 == 0;
    return a.softcap > 0.0f ? launch_draft<true>(D, stream) : launch_draft<false>(D, stream);
}

}  // namespace qmv
