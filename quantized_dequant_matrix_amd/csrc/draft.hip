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
// Three launches, chunks of 8192 logits, groups of 1024:
//   stats  one workgroup per (chunk of a row, row, sequence): maximum and sum
//          of weights of the chunk.  Reads every logit once: this is the
//          traffic.
//   pick   one workgroup per (chunk, sequence): joins the rows' chunks, makes
//          the accept tests, and sums the groups of its chunk of the row to
//          draw from, a wave each.
//   draw   one workgroup a sequence: the group that holds the drawn point,
//          then the element.
#include <stdint.h>

#include "qmv_device.h"
#include "qmv_internal.h"
#include "step_internal.h"

namespace qmv {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kChunk = 8192;                // logits of one workgroup
constexpr int kPer = kChunk / kThreads;     // 16 a thread
constexpr int kGroup = kChunk / kWaves;     // 1024: a wave's part of a chunk
constexpr int kGroupPer = kGroup / kThreads; // 2 a thread
constexpr int kMaxRows = 2 * 64 + 1;        // rows of a sequence: G + 1 target rows, G draft rows
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kNegInf = -__builtin_inff();

// 2^(j / 64), j < 64, in LDS: filled by the first wave of a workgroup before
// its first barrier.
__shared__ double exp_table[kWave];

__device__ __forceinline__ void fill_exp_table() {
    if (threadIdx.x < kWave) {
        // (ln 2 / 64) j by the series up to the 17th power: below 2^-54 left
        const double x = static_cast<double>(threadIdx.x) * (0.69314718055994530942 / 64.0);
        double p = 1.0;
#pragma unroll
        for (int k = 17; k >= 1; --k) p = fma(p * x, 1.0 / k, 1.0);
        exp_table[threadIdx.x] = p;
    }
}

// 2^t for t <= 64: t = n + j / 64 + f, |f| <= 1/128, with n + j / 64 rounded
// off by an addition of 1.5 2^46 (whose last place is 1/64), 2^(j / 64) from
// the table and 2^f by its series up to the 5th power, whose next term is
// below 4e-17.  Below 2^-1020 the result is 0 (the row's maximum is 2^0).
__device__ __forceinline__ double exp2_f64(double t) {
    const bool none = t < -1020.0;
    t = fmax(t, -1020.0);
    constexpr double kShift = 105553116266496.0;
    const double r = t + kShift;
    const int k = static_cast<int>(__builtin_bit_cast(uint64_t, r));  // 64 n + j
    const double f = (t - (r - kShift)) * 0.69314718055994530942;
    double p = fma(f, 1.0 / 120.0, 1.0 / 24.0);
    p = fma(p, f, 1.0 / 6.0);
    p = fma(p, f, 0.5);
    p = fma(p, f, 1.0);
    const double e = exp_table[k & 63];
    const uint64_t v = __builtin_bit_cast(uint64_t, fma(p * f, e, e));
    const double x = __builtin_bit_cast(double, v + (static_cast<uint64_t>(static_cast<uint32_t>(k >> 6) << 20) << 32));
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
    // cap(y) / temperature in units of log2: the exponent of a weight up to
    // the row's maximum.  Logits are bounded: y k stays finite.
    template <bool CAP>
    __device__ __forceinline__ double level(float y) const {
#pragma clang fp contract(off)
        // (the product is rounded as the row's own level was: the difference
        // of the largest logit to it is 0, however large both are)
        const double v = static_cast<double>(y);
        if constexpr (!CAP) return v * k;
        // tanh z = 1 - 2 / (1 + e^(2 z)); beyond |z| = 20 it is +-1 in 64 bits
        const double e = exp2_f64(fmin(fmax(v * twice, -64.0), 64.0));
        return fma(-2.0, rcp_f64(1.0 + e), 1.0) * cap;
    }
    // weight relative to the level `top` of the row's (or chunk's) maximum;
    // no branches, so that a thread's weights overlap
    template <bool CAP>
    __device__ __forceinline__ double weight(float y, double top) const {
#pragma clang fp contract(off)
        const double w = exp2_f64(level<CAP>(y) - top);
        return y == kNegInf ? 0.0 : w;
    }
};

// NaN weighs nothing; +infinity is the largest float.
__device__ __forceinline__ float clean(float y) { return y == y ? fminf(y, 3.4028234663852886e38f) : kNegInf; }

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
    int chunks, groups;  // groups = chunks * kWaves
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

// A double of another lane (0 where the pattern has none).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROW_MASK, 0xF, false);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

__device__ __forceinline__ double lane_f64(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// Inclusive sum over the lanes, in lane order: within rows of 16 lanes
// (row_shr 1, 2, 4, 8), then across them (row_bcast 15 and 31).
__device__ __forceinline__ double wave_prefix(double v) {
    v += dpp_f64<0x111, 0xF>(v);
    v += dpp_f64<0x112, 0xF>(v);
    v += dpp_f64<0x114, 0xF>(v);
    v += dpp_f64<0x118, 0xF>(v);
    v += dpp_f64<0x142, 0xA>(v);
    v += dpp_f64<0x143, 0xC>(v);
    return v;
}

__device__ __forceinline__ double wave_add(double v) { return lane_f64(wave_prefix(v), kWave - 1); }

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

// 16 logits of the wave's group of a chunk, 4 by 4 across the wave (a sum's
// order is free); past the row's end: no weight.
__device__ __forceinline__ void load_spread(const DraftView& D, const float* y, int c, float (&v)[kPer]) {
    const int64_t base = static_cast<int64_t>(c) * kChunk + threadIdx.x / kWave * kGroup + 4 * (threadIdx.x & (kWave - 1));
    if (D.vec && (c + 1) * static_cast<int64_t>(kChunk) <= D.a.V) {  // all loads first
        float4 f[kPer / 4];
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) f[i] = *reinterpret_cast<const float4*>(y + base + i * 4 * kWave);
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) {
            v[4 * i] = clean(f[i].x); v[4 * i + 1] = clean(f[i].y); v[4 * i + 2] = clean(f[i].z); v[4 * i + 3] = clean(f[i].w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {  // past the end: the last one again, then taken out
            const int64_t at = base + i / 4 * 4 * kWave + i % 4;
            v[i] = y[at < D.a.V ? at : D.a.V - 1];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t at = base + i / 4 * 4 * kWave + i % 4;
            v[i] = at < D.a.V ? clean(v[i]) : kNegInf;
        }
    }
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draft_stats_kernel(DraftView D) {
    __shared__ float mx[kWaves];
    __shared__ double sm[kWaves];
    const int c = blockIdx.x, r = blockIdx.y;
    const int64_t b = blockIdx.z;
    const int n = D.drafts(b);
    if (r <= D.a.G ? r > n : r - D.a.G - 1 >= n) return;  // a row that no draft uses
    float v[kPer];
    load_spread(D, D.row(b, r), c, v);
    fill_exp_table();
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = fmaxf(top, v[i]);
    top = wave_max(top);
    if ((threadIdx.x & (kWave - 1)) == 0) mx[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) top = fmaxf(top, mx[i]);
    const double level = D.w.template level<CAP>(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += D.w.template weight<CAP>(v[i], level);
    sum = wave_add(sum);
    if ((threadIdx.x & (kWave - 1)) == 0) sm[threadIdx.x / kWave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) sum += sm[i];
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
    double z = first.top != kNegInf ? first.sum * exp2_f64(D.w.template level<CAP>(first.top) - *level) : 0.0;
    for (int c = lane + kWave; c < D.chunks; c += kWave)
        if (s[c].top != kNegInf) z += s[c].sum * exp2_f64(D.w.template level<CAP>(s[c].top) - *level);
    *sum = wave_add(z);
}

__device__ __forceinline__ double inverse(double sum) { return sum > 0.0 ? 1.0 / sum : 0.0; }

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draft_pick_kernel(DraftView D) {
    __shared__ double levels[kMaxRows], inverses[kMaxRows];
    __shared__ Pick P;
    const int c = blockIdx.x;
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
    for (int i = wave; i < 2 * n + 1; i += kWaves) {
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
            if (c == 0) D.picks[b] = P;
        }
    }
    __syncthreads();
    float vp[kPer], vq[kPer];
    load_spread(D, D.row(b, P.accepted), c, vp);
    double x = 0.0, y = 0.0;
    if (P.residual) {
        load_spread(D, D.row(b, G + 1 + P.accepted), c, vq);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const double p = D.w.template weight<CAP>(vp[i], P.p_level) * P.p_inv;
            y += p;
            x += fmax(p - D.w.template weight<CAP>(vq[i], P.q_level) * P.q_inv, 0.0);
        }
        x = wave_add(x);
        y = wave_add(y);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x += D.w.template weight<CAP>(vp[i], P.p_level) * P.p_inv;
        x = y = wave_add(x);
    }
    if (lane == 0) {
        D.rest[b * D.groups + c * kWaves + wave] = x;
        D.whole[b * D.groups + c * kWaves + wave] = y;
    }
}

// The group that holds the drawn point, by one wave: the first whose running
// sum exceeds u times the whole sum, or the last with any weight (-1: none
// has).  A lane sums `per` consecutive groups, the wave their sums; then the
// lane with the point goes through its own.
__device__ __forceinline__ int find_group(const double* s, int groups, double u, double* target, double* before) {
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (groups + kWave - 1) / kWave;
    const int g0 = min(lane * per, groups), g1 = min(g0 + per, groups);
    double mine = 0.0;
    int tail = -1;
    for (int g = g0; g < g1; ++g) {
        mine += s[g];
        if (s[g] > 0.0) tail = g;
    }
    const double upto = wave_prefix(mine);
    *target = u * lane_f64(upto, kWave - 1);
    int hit = -1;
    double run = upto - mine, from = run;
    for (int g = g0; g < g1 && hit < 0; ++g) {
        from = run;
        run += s[g];
        if (s[g] > 0.0 && run > *target) hit = g;
    }
    uint64_t lanes = __ballot(hit >= 0);
    if (lanes == 0) {  // the point lies at the very end: the last group with weight
        hit = tail;
        lanes = __ballot(tail >= 0);
        if (lanes == 0) return -1;
        lanes = uint64_t{1} << (63 - __clzll(static_cast<long long>(lanes)));
        from = run;
        if (tail >= 0)
            for (int g = g1 - 1; g >= tail; --g) from -= s[g];
    }
    const int at = __ffsll(static_cast<unsigned long long>(lanes)) - 1;
    *before = lane_f64(from, at);
    return __builtin_amdgcn_readlane(hit, at);
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draft_draw_kernel(DraftView D) {
    __shared__ double sums[kWaves];
    __shared__ int found, last, group, from_whole;
    __shared__ double target, before;
    const int64_t b = blockIdx.x;
    const int t = threadIdx.x, wave = t / kWave, lane = t & (kWave - 1), G = D.a.G;
    const Pick P = D.picks[b];
    if (wave == 0) {
        const double u = static_cast<double>(D.a.u[b * (G + 1) + G]);
        double to, from;
        int g = find_group(D.rest + b * D.groups, D.groups, u, &to, &from);
        const bool all = g < 0;  // no rest anywhere: from p itself
        if (all) g = find_group(D.whole + b * D.groups, D.groups, u, &to, &from);
        if (lane == 0) {
            group = g;
            from_whole = all;
            target = to;
            before = from;
            found = kGroup;
            last = -1;
        }
    }
    fill_exp_table();
    __syncthreads();
    int token = -1;
    if (group >= 0) {
        // thread t has elements 2 t and 2 t + 1 of the group
        const float* yp = D.row(b, P.accepted);
        const bool minus = P.residual && !from_whole;
        const float* yq = minus ? D.row(b, G + 1 + P.accepted) : yp;
        const int64_t base = static_cast<int64_t>(group) * kGroup + t * kGroupPer;
        double w[kGroupPer];
        double mine = 0.0;
        int tail = -1;
#pragma unroll
        for (int i = 0; i < kGroupPer; ++i) {
            w[i] = 0.0;
            if (base + i < D.a.V) {
                w[i] = D.w.template weight<CAP>(clean(yp[base + i]), P.p_level) * P.p_inv;
                if (minus) w[i] = fmax(w[i] - D.w.template weight<CAP>(clean(yq[base + i]), P.q_level) * P.q_inv, 0.0);
            }
            mine += w[i];
            if (w[i] > 0.0) tail = t * kGroupPer + i;
        }
        const double upto = wave_prefix(mine);
        if (lane == kWave - 1) sums[wave] = upto;
        __syncthreads();
        double run = before + (upto - mine);
        for (int i = 0; i < wave; ++i) run += sums[i];
        int hit = kGroup;
#pragma unroll
        for (int i = 0; i < kGroupPer; ++i) {
            run += w[i];
            if (hit == kGroup && w[i] > 0.0 && run > target) hit = t * kGroupPer + i;
        }
        if (hit < kGroup) atomicMin(&found, hit);
        if (tail >= 0) atomicMax(&last, tail);
        __syncthreads();
        const int at = found < kGroup ? found : last;
        token = at < 0 ? -1 : static_cast<int>(static_cast<int64_t>(group) * kGroup + at);
    }
    const int a = P.accepted;
    if (t == 0) D.a.accepted[b] = a;
    for (int i = t; i <= G; i += kThreads)
        D.a.tokens[b * (G + 1) + i] = i < a ? D.a.draft_tokens[b * G + i] : (i == a ? token : -1);
}

int64_t chunks_of(int64_t V) { return (V + kChunk - 1) / kChunk; }

template <bool CAP>
hipError_t launch_draft(const DraftView& D, hipStream_t stream) {
    const unsigned ch = static_cast<unsigned>(D.chunks), B = static_cast<unsigned>(D.a.B);
    hipLaunchKernelGGL(draft_stats_kernel<CAP>, dim3(ch, static_cast<unsigned>(2 * D.a.G + 1), B), dim3(kThreads), 0,
                       stream, D);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draft_pick_kernel<CAP>, dim3(ch, B), dim3(kThreads), 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draft_draw_kernel<CAP>, dim3(B), dim3(kThreads), 0, stream, D);
    return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t draft_ws_bytes(int64_t B, int G, int64_t V) {
    const size_t n = static_cast<size_t>(B) * static_cast<size_t>(chunks_of(V));
    return align256(n * static_cast<size_t>(2 * G + 1) * sizeof(Stat)) + 2 * align256(n * kWaves * sizeof(double)) +
           align256(static_cast<size_t>(B) * sizeof(Pick));
}

hipError_t launch_draft_verify(const DraftArgs& a, void* ws, hipStream_t stream) {
    DraftView D;
    D.a = a;
    D.w.k = kLog2e / static_cast<double>(a.temperature);
    D.w.cap = static_cast<double>(a.softcap) * D.w.k;
    D.w.twice = a.softcap > 0.0f ? 2.0 * kLog2e / static_cast<double>(a.softcap) : 0.0;
    D.chunks = static_cast<int>(chunks_of(a.V));
    D.groups = D.chunks * kWaves;
    const size_t n = static_cast<size_t>(a.B) * static_cast<size_t>(D.chunks);
    char* p = static_cast<char*>(ws);
    D.stats = reinterpret_cast<Stat*>(p);
    p += align256(n * static_cast<size_t>(2 * a.G + 1) * sizeof(Stat));
    D.rest = reinterpret_cast<double*>(p);
    p += align256(n * kWaves * sizeof(double));
    D.whole = reinterpret_cast<double*>(p);
    D.picks = reinterpret_cast<Pick*>(p + align256(n * kWaves * sizeof(double)));
    D.vec = ((reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) & 15) == 0 &&
            a.ldt % 4 == 0 && a.ldd % 4 == 0;
    return a.softcap > 0.0f ? launch_draft<true>(D, stream) : launch_draft<false>(D, stream);
}

}  // namespace qmv
