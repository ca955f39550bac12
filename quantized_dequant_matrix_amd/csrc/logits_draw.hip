// A token of each row of logits, by temperature, top-k, top-p and min-p.
//
// The filters keep a prefix of the row in the order "larger logit first,
// equal ones by index", and the draw takes an element of it by a running sum
// in the same order.  So everything asks one kind of question: which element
// of the order is the first whose running count, or running sum of weights,
// reaches a number?  Nothing has to be sorted for that but the elements around
// the answer:
//   - counts and sums of weights in 4096 bins of the distance from the largest
//     logit say which bins hold the answers.  The first answer (the k-th
//     element) decides where the next is asked for (the sum over the first k),
//     but within the bounds that its bin gives, so that a few bins are known
//     to hold all answers;
//   - their elements are collected (up to 4096), sorted, and give the answers
//     exactly.
// Rows with a top-k of up to 2048 need no sums: the bins count, and the first
// k are collected whole.  Rows of temperature 0 end with the first step.
//
// Weights are whole multiples of 2^-q of the row's largest: their sums are
// exact in 64-bit integers in any order, so bins can be summed by atomics and
// a row may be split over workgroups in any way.
//
// A row whose answers lie among more elements than that (thousands of equal
// logits, or nearly) is resolved digit by digit of a 64-bit key (order code of
// the logit, then the index from below) instead: slower, whatever the row.
#include <stdint.h>

#include "qmv_device.h"
#include "serve_internal.h"
#include "sort_device.h"
#include "step_device.h"
#include "weights_device.h"

namespace qmv {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int kBins = 4096, kBinsPer = kBins / kThreads;
constexpr int kMostCands = 4096, kCandsPer = kMostCands / kThreads;
constexpr int kMostCounted = 2048;  // largest top-k that is collected whole
constexpr int kDigitBins = 2048;
constexpr int kMaxParts = kWave;  // a lane a part when they are joined
constexpr float kMaxLogit = 3.4028234663852886e38f;

struct Sum {
    uint64_t mass;
    uint32_t count;
};

__device__ __forceinline__ bool weighs(float y) { return y > kNegInf; }  // false for NaN

// Larger logits have larger codes; -0 ranks with +0.
__device__ __forceinline__ uint32_t code_of(float y) {
    const float v = fminf(y, kMaxLogit);
    const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float logit_of(uint32_t code) {
    return __uint_as_float((code & 0x80000000u) ? (code ^ 0x80000000u) : ~code);
}

__device__ __forceinline__ uint64_t key_of(float y, int64_t i) {
    return (static_cast<uint64_t>(code_of(y)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}

__device__ __forceinline__ int32_t index_of(uint64_t key) {
    return static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

// What a part of a row says about it.
struct Part {
    uint64_t best;   // key of its first element, 0: none
    float sum;       // of logits of ordinary size, and how many they are
    uint32_t count;
};

// Bins that hold the answers, and what else the parts add up.
struct Head {
    uint64_t above_mass;  // elements that pass min_p
    uint32_t above_count;
    uint32_t collected;
    int32_t k_bin, p_lo, p_hi, u_lo, u_hi;
    uint32_t cands;  // elements of these bins
};

struct DrawView {
    DrawArgs a;
    double twice;  // 2 log2(e) / softcap
    int q;
    int parts;
    int64_t part_len;  // a multiple of 4
    bool vec;          // rows are 16-byte aligned
    Part* part;        // [M][parts]
    Head* head;        // [M]
    uint32_t* count;   // [M][kBins]
    uint64_t* mass;    // [M][kBins]
    uint64_t* cand;    // [M][kMostCands]
};

enum Mode { kFirst, kCounted, kSummed };

// A row's parameters, the same in every thread.
template <bool CAP>
struct Row {
    const float* y;
    uint64_t best;
    Weights w;
    double level, unit;  // of the largest logit (level_of_top); 2^q
    double min_exponent;
    float top, per_bin, top_p, u;
    int32_t top_k;
    bool has_min;
    Mode mode;

    // Before the first exponent, behind a barrier after fill_exp_table().
    __device__ __forceinline__ void level_of_top() { level = w.template level<CAP>(top); }
    __device__ __forceinline__ double exponent(float v) const {
        return w.template below<CAP>(w.template level<CAP>(fminf(v, kMaxLogit)), level);
    }
    // weight * 2^q, rounded to nearest by an addition of 2^52
    __device__ __forceinline__ uint64_t mass_of(double e) const {
        const double r = fma(exp2_f64(e), unit, 4503599627370496.0);
        return __builtin_bit_cast(uint64_t, r) & 0xFFFFFFFFFFFFFull;
    }
    // Bins follow the order.  1 + distance * per_bin has 512 bins an octave, 8
    // octaves: equal steps near the largest logit, then steps in proportion to
    // the distance, so that neither the temperature nor the spread of the
    // logits matters much.
    __device__ __forceinline__ int bin_of(float v) const {
        const float t = fminf(top - fminf(v, kMaxLogit), kMaxLogit);
        const uint32_t b = (__float_as_uint(fmaf(t, per_bin, 1.0f)) - 0x3f800000u) >> 14;
        return static_cast<int>(b < kBins ? b : kBins - 1);
    }
    // Sums that the answers have to reach.
    __device__ __forceinline__ uint64_t need_p(uint64_t mass) const {
        const double border = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(mass));
        const uint64_t need = static_cast<uint64_t>(border);
        return need > mass ? mass : need;
    }
    __device__ __forceinline__ uint64_t need_u(uint64_t mass) const {
        const double f = fmin(fmax(static_cast<double>(u), 0.0), 1.0);  // NaN: 0
        const uint64_t need = static_cast<uint64_t>(f * static_cast<double>(mass)) + 1;
        return need > mass ? mass : need;
    }
};

__device__ __forceinline__ uint64_t at_least_1(uint64_t v) { return v < 1 ? 1 : v; }

template <bool CAP>
__device__ __forceinline__ Row<CAP> row_of(const DrawView& D, int64_t m, uint64_t best, float sum, uint32_t count) {
    Row<CAP> R;
    R.y = D.a.logits + m * D.a.ldl;
    R.best = best;
    const float T = D.a.temperature[m];
    R.mode = kFirst;
    if (best == 0 || !(T > 0.0f)) return R;
    R.top_k = D.a.top_k ? D.a.top_k[m] : 0;
    R.top_p = D.a.top_p ? D.a.top_p[m] : 1.0f;
    R.u = D.a.u[m];
    const float min_p = D.a.min_p ? D.a.min_p[m] : 0.0f;
    R.has_min = min_p > 0.0f;
    R.min_exponent = R.has_min ? log2(static_cast<double>(min_p)) : 0.0;
    R.w.k = kLog2e / static_cast<double>(T);
    R.w.cap = static_cast<double>(D.a.softcap) * R.w.k;
    R.w.twice = D.twice;
    R.unit = static_cast<double>(uint64_t{1} << D.q);
    R.top = logit_of(static_cast<uint32_t>(best >> 32));
    // the first octave ends at the nearer of eight powers of two of weight and
    // an eighth of the mean distance
    const float mean = count ? fmaxf(R.top - sum / static_cast<float>(count), 0.0f) : 0.0f;
    R.per_bin = fminf(fmaxf(mean > 0.0f ? 8.0f / mean : 0.0f, static_cast<float>(fmin(R.w.k, 1e30)) * 0.125f), 1e30f);
    R.mode = R.top_k > 0 && R.top_k <= kMostCounted ? kCounted : kSummed;
    return R;
}

// f(logit, index) for the logits of [lo, hi), 16 a thread and step; -infinity
// past the end.  lo is a multiple of 4.
template <class F>
__device__ __forceinline__ void for_logits(const float* y, int64_t lo, int64_t hi, bool vec, F&& f) {
    constexpr int kU = 4;
    for (int64_t base = lo + 4 * threadIdx.x; base < hi; base += kU * 4 * kThreads) {
        float v[kU][4];
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            const int64_t at = base + j * 4 * kThreads;
            if (vec && at + 4 <= hi) {
                const float4 x = *reinterpret_cast<const float4*>(y + at);
                v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][e] = at + e < hi ? y[at + e] : kNegInf;
            }
        }
#pragma unroll
        for (int j = 0; j < kU; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) f(v[j][e], base + j * 4 * kThreads + e);
    }
}

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int d) {
    const uint32_t lo = __shfl_up(static_cast<uint32_t>(v), d, kWave), hi = __shfl_up(static_cast<uint32_t>(v >> 32), d, kWave);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ Part join(Part p) {  // over the wave, in every lane
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint64_t o = shfl_xor64(p.best, d);
        p.best = o > p.best ? o : p.best;
        p.sum += __shfl_xor(p.sum, d, kWave);
        p.count += __shfl_xor(p.count, d, kWave);
    }
    return p;
}

struct Scan {
    uint64_t mass[kWaves];
    uint32_t count[kWaves];
};

// Sums before this thread in thread order, and the total.
__device__ __forceinline__ Sum block_before(Scan& S, Sum mine, Sum* total) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    Sum upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint64_t m = shfl_up64(upto.mass, d);
        const uint32_t c = __shfl_up(upto.count, d, kWave);
        if (lane >= d) {
            upto.mass += m;
            upto.count += c;
        }
    }
    __syncthreads();
    if (lane == kWave - 1) {
        S.mass[wave] = upto.mass;
        S.count[wave] = upto.count;
    }
    __syncthreads();
    Sum before = {upto.mass - mine.mass, upto.count - mine.count};
    *total = {0, 0};
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i < wave) {
            before.mass += S.mass[i];
            before.count += S.count[i];
        }
        total->mass += S.mass[i];
        total->count += S.count[i];
    }
    return before;
}

// An element (or bin) where a running count or sum reaches a number, with the
// sums before and with it.
struct Hit {
    Sum before, upto;
    int at;
};

__device__ __forceinline__ bool reaches(const Sum& before, const Sum& upto, bool mass, uint64_t need) {
    return mass ? before.mass < need && upto.mass >= need : before.count < need && upto.count >= need;
}

// ------------------------------------------------------------ digit by digit

struct Digits {
    uint64_t mass[kDigitBins];
    uint32_t count[kDigitBins];
    Scan scan;
    Hit hit;
};

struct Found {
    uint64_t key;
    Sum upto;  // sums up to and with the element
};

// The first element of the order whose running count (mass: running sum)
// reaches `need`, 1 <= need <= the row's.
template <bool CAP>
__device__ Found find(Digits& S, const DrawView& D, const Row<CAP>& R, bool mass, uint64_t need) {
    uint64_t prefix = 0;
    Sum before = {0, 0}, upto = {0, 0};
    const int t = threadIdx.x;
    constexpr int kLow[6] = {53, 42, 32, 21, 10, 0};
    for (int d = 0; d < 6; ++d) {
        const int low = kLow[d], high = d == 0 ? 64 : kLow[d - 1];
        const uint32_t digits = (1u << (high - low)) - 1u;
        __syncthreads();
        for (int i = t; i < kDigitBins; i += kThreads) {
            S.mass[i] = 0;
            S.count[i] = 0;
        }
        __syncthreads();
        for_logits(R.y, 0, D.a.V, D.vec, [&](float v, int64_t i) {
            if (!weighs(v)) return;
            const uint64_t key = key_of(v, i);
            if (d > 0 && (key >> high) != (prefix >> high)) return;
            const uint32_t bin = digits - (static_cast<uint32_t>(key >> low) & digits);  // bin 0: first in the order
            atomicAdd(&S.count[bin], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&S.mass[bin]),
                      static_cast<unsigned long long>(R.mass_of(R.exponent(v))));
        });
        __syncthreads();
        const Sum two[2] = {{S.mass[2 * t], S.count[2 * t]}, {S.mass[2 * t + 1], S.count[2 * t + 1]}};
        Sum total;
        Sum run = block_before(S.scan, {two[0].mass + two[1].mass, two[0].count + two[1].count}, &total);
        run.mass += before.mass;
        run.count += before.count;
        for (int j = 0; j < 2; ++j) {
            const Sum next = {run.mass + two[j].mass, run.count + two[j].count};
            if (reaches(run, next, mass, need)) S.hit = {run, next, 2 * t + j};
            run = next;
        }
        __syncthreads();
        before = S.hit.before;
        upto = S.hit.upto;
        prefix |= static_cast<uint64_t>(digits - static_cast<uint32_t>(S.hit.at)) << low;
    }
    return {prefix, upto};
}

// token and count of a row of any kind
template <bool CAP>
__device__ void draw_by_digits(Digits& S, const DrawView& D, const Row<CAP>& R, int32_t* token, int32_t* n) {
    Sum mine = {0, 0}, above = {0, 0}, total, kept;
    for_logits(R.y, 0, D.a.V, D.vec, [&](float v, int64_t) {
        if (!weighs(v)) return;
        const double e = R.exponent(v);
        const uint64_t w = R.mass_of(e);
        mine.mass += w;
        mine.count += 1;
        if (e >= R.min_exponent) {
            above.mass += w;
            above.count += 1;
        }
    });
    block_before(S.scan, above, &kept);
    block_before(S.scan, mine, &total);
    if (!R.has_min) kept = total;
    if (kept.count == 0) kept = {static_cast<uint64_t>(R.unit), 1};
    Sum of_k = total;
    if (R.top_k > 0 && static_cast<uint32_t>(R.top_k) < total.count)
        of_k = find(S, D, R, false, static_cast<uint64_t>(R.top_k)).upto;
    if (of_k.count < kept.count) kept = of_k;
    if (R.top_p < 1.0f) {
        const Sum of_p = find(S, D, R, true, at_least_1(R.need_p(of_k.mass))).upto;
        if (of_p.count < kept.count) kept = of_p;
    }
    *n = static_cast<int32_t>(kept.count);
    *token = index_of(find(S, D, R, true, at_least_1(R.need_u(kept.mass))).key);
}

// ------------------------------------------------------------ by bins

// The bins of a row with their running sums: thread t holds bins 4 t .. 4 t + 3.
struct Bins {
    Sum bin[kBinsPer];
    Sum before, total;
};

struct Ask {
    Scan scan;
    Hit hit[5];
    uint32_t cands;
};

__device__ __forceinline__ Bins load_bins(Ask& S, const uint32_t* count, const uint64_t* mass, bool summed) {
    Bins B;
    Sum mine = {0, 0};
#pragma unroll
    for (int j = 0; j < kBinsPer; ++j) {
        B.bin[j].count = count[kBinsPer * threadIdx.x + j];
        B.bin[j].mass = summed ? mass[kBinsPer * threadIdx.x + j] : 0;
        mine.mass += B.bin[j].mass;
        mine.count += B.bin[j].count;
    }
    B.before = block_before(S.scan, mine, &B.total);
    return B;
}

// The thread whose bin reaches `need` says so in hit[slot].
__device__ __forceinline__ void ask_bins(Ask& S, const Bins& B, int slot, bool mass, uint64_t need) {
    Sum run = B.before;
#pragma unroll
    for (int j = 0; j < kBinsPer; ++j) {
        const Sum next = {run.mass + B.bin[j].mass, run.count + B.bin[j].count};
        if (reaches(run, next, mass, need)) S.hit[slot] = {run, next, kBinsPer * static_cast<int>(threadIdx.x) + j};
        run = next;
    }
}

// Bins that hold the answers, in every thread.
template <bool CAP>
__device__ __forceinline__ Head choose_bins(Ask& S, const Row<CAP>& R, const Bins& B, Sum above) {
    Head H = {above.mass, above.count, 0, -1, 0, -1, 0, -1, 0};
    const uint32_t kk = R.top_k > 0 && static_cast<uint32_t>(R.top_k) < B.total.count ? R.top_k : B.total.count;
    if (threadIdx.x == 0) S.cands = 0;
    if (R.mode == kCounted) {
        ask_bins(S, B, 0, false, kk);
        __syncthreads();
        H.u_hi = S.hit[0].at;  // the first kk whole
        H.cands = S.hit[0].upto.count;
        return H;
    }
    uint64_t k_lo = B.total.mass, k_hi = B.total.mass;
    if (kk < B.total.count) {
        ask_bins(S, B, 0, false, kk);
        __syncthreads();
        const Hit h = S.hit[0];
        k_lo = k_hi = h.upto.mass;
        if (h.upto.count != kk) {
            H.k_bin = h.at;
            k_lo = h.before.mass;
        }
    }
    uint64_t lo = k_lo, hi = k_hi;
    if (R.top_p < 1.0f) {
        ask_bins(S, B, 1, true, at_least_1(R.need_p(k_lo)));
        ask_bins(S, B, 2, true, at_least_1(R.need_p(k_hi)));
        __syncthreads();
        H.p_lo = S.hit[1].at;
        H.p_hi = S.hit[2].at;
        lo = min(lo, S.hit[1].before.mass);
        hi = min(hi, S.hit[2].upto.mass);
    }
    if (R.has_min) {
        const uint64_t m = above.count ? above.mass : static_cast<uint64_t>(R.unit);
        lo = min(lo, m);
        hi = min(hi, m);
    }
    ask_bins(S, B, 3, true, at_least_1(R.need_u(lo)));
    ask_bins(S, B, 4, true, at_least_1(R.need_u(hi)));
    __syncthreads();
    H.u_lo = S.hit[3].at;
    H.u_hi = S.hit[4].at;
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kBinsPer; ++j) {
        const int b = kBinsPer * static_cast<int>(threadIdx.x) + j;
        if (b == H.k_bin || (b >= H.p_lo && b <= H.p_hi) || (b >= H.u_lo && b <= H.u_hi)) mine += B.bin[j].count;
    }
    if (mine) atomicAdd(&S.cands, mine);
    __syncthreads();
    H.cands = S.cands;
    return H;
}

__device__ __forceinline__ bool chosen(const Head& H, int b) {
    return b == H.k_bin || (b >= H.p_lo && b <= H.p_hi) || (b >= H.u_lo && b <= H.u_hi);
}

struct Sorter {
    uint64_t key[2 * kMostCands];
    Ask ask;
    Hit hit[3];
};

// Sorts the n <= kMostCands keys in S.key, first of the order first; thread t
// gets keys 4 t .. 4 t + 3 (0 past the end).
__device__ __forceinline__ void sort_cands(Sorter& S, uint32_t n, uint64_t (&mine)[kCandsPer]) {
    const int t = threadIdx.x, lane = t & (kWave - 1);
    __syncthreads();
    if (n <= kWave) {
        if (t < kWave) {
            uint64_t key[1] = {lane < n ? S.key[lane] : 0};
            wave_sort_desc(key);
            S.key[lane] = key[0];
        }
    } else if (n <= 4 * kWave) {
        if (t < kWave) {
            uint64_t key[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) key[j] = j * kWave + lane < n ? S.key[j * kWave + lane] : 0;
            wave_sort_desc(key);
#pragma unroll
            for (int j = 0; j < 4; ++j) S.key[j * kWave + lane] = key[j];
        }
    } else if (n <= kThreads) {
        uint64_t key[1] = {t < n ? S.key[t] : 0};
        __syncthreads();
        block_sort_desc(key, S.key);
        __syncthreads();
        S.key[t] = key[0];
    } else {
        uint64_t key[kCandsPer];
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) key[j] = j * kThreads + t < n ? S.key[j * kThreads + t] : 0;
        __syncthreads();
        block_sort_desc(key, S.key);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) S.key[j * kThreads + t] = key[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCandsPer; ++j) mine[j] = kCandsPer * t + j < n ? S.key[kCandsPer * t + j] : 0;
}

// The collected elements of a row, sorted, and the answers among them.
template <bool CAP>
__device__ __forceinline__ void draw_from_cands(Sorter& S, const Row<CAP>& R, const Bins& B, const Head& H, int32_t* token,
                                                int32_t* n) {
    uint64_t key[kCandsPer];
    sort_cands(S, H.cands, key);
    const int t = threadIdx.x;
    double e[kCandsPer];
    Sum w[kCandsPer];
    int bin[kCandsPer];
#pragma unroll
    for (int j = 0; j < kCandsPer; ++j) {
        const float v = logit_of(static_cast<uint32_t>(key[j] >> 32));
        bin[j] = key[j] ? R.bin_of(v) : -1;
        e[j] = key[j] ? R.exponent(v) : 0.0;
        w[j] = {key[j] ? R.mass_of(e[j]) : 0, key[j] ? 1u : 0u};
    }
    const uint32_t kk = R.top_k > 0 && static_cast<uint32_t>(R.top_k) < B.total.count ? R.top_k : B.total.count;
    // the element of bin `of` (of any, with -1: then from the first on) that
    // reaches `need`
    auto ask = [&](int slot, int of, Sum before, bool mass, uint64_t need) -> Hit {
        Sum own = {0, 0}, in[kCandsPer], total;
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            in[j] = of < 0 || bin[j] == of ? w[j] : Sum{0, 0};
            own.mass += in[j].mass;
            own.count += in[j].count;
        }
        Sum run = block_before(S.ask.scan, own, &total);
        run.mass += before.mass;
        run.count += before.count;
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            const Sum next = {run.mass + in[j].mass, run.count + in[j].count};
            if (reaches(run, next, mass, need)) S.hit[slot] = {run, next, kCandsPer * t + j};
            run = next;
        }
        __syncthreads();
        return S.hit[slot];
    };
    auto ask_in_bin = [&](int slot, bool mass, uint64_t need) -> Hit {
        ask_bins(S.ask, B, slot, mass, need);
        __syncthreads();
        const Hit h = S.ask.hit[slot];
        return ask(slot, h.at, h.before, mass, need);
    };
    Sum kept, of_k;
    if (R.mode == kCounted) {
        Sum mine = {0, 0}, first = {0, 0};
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            if (static_cast<uint32_t>(kCandsPer * t + j) >= kk) w[j] = {0, 0};
            first.mass += w[j].mass;
            first.count += w[j].count;
            if (w[j].count && e[j] >= R.min_exponent) {
                mine.mass += w[j].mass;
                mine.count += 1;
            }
        }
        block_before(S.ask.scan, first, &of_k);
        kept = of_k;
        if (R.has_min) block_before(S.ask.scan, mine, &kept);
    } else {
        of_k = B.total;
        if (H.k_bin >= 0) {
            of_k = ask_in_bin(0, false, kk).upto;
        } else if (kk < B.total.count) {  // the end of a bin
            ask_bins(S.ask, B, 0, false, kk);
            __syncthreads();
            of_k = S.ask.hit[0].upto;
        }
        kept = of_k;
        if (R.has_min && H.above_count < kept.count) kept = {H.above_mass, H.above_count};
    }
    if (kept.count == 0) kept = {static_cast<uint64_t>(R.unit), 1};
    if (R.top_p < 1.0f) {
        const uint64_t need = at_least_1(R.need_p(of_k.mass));
        const Sum of_p = (R.mode == kCounted ? ask(1, -1, {0, 0}, true, need) : ask_in_bin(1, true, need)).upto;
        if (of_p.count < kept.count) kept = of_p;
    }
    const uint64_t need = at_least_1(R.need_u(kept.mass));
    const Hit h = R.mode == kCounted ? ask(2, -1, {0, 0}, true, need) : ask_in_bin(2, true, need);
    *n = static_cast<int32_t>(kept.count);
    *token = index_of(S.key[h.at]);
}

template <bool CAP>
__device__ __forceinline__ void store(const DrawView& D, int64_t m, int32_t token, int32_t n) {
    if (threadIdx.x == 0) {
        D.a.token[m] = token;
        if (D.a.kept) D.a.kept[m] = n;
    }
}

// ------------------------------------------------------------ steps of a part

__device__ __forceinline__ Part first_of(const float* y, int64_t lo, int64_t hi, bool vec, Part* lds) {
    Part p = {0, 0.0f, 0};
    for_logits(y, lo, hi, vec, [&](float v, int64_t i) {
        const uint64_t key = weighs(v) ? key_of(v, i) : 0;
        p.best = key > p.best ? key : p.best;
        const bool ordinary = fabsf(v) < 1e6f;  // false for NaN
        p.sum += ordinary ? v : 0.0f;
        p.count += ordinary ? 1 : 0;
    });
    p = join(p);
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    if (lane == 0) lds[wave] = p;
    __syncthreads();
    p = lane < kWaves ? lds[lane] : Part{0, 0.0f, 0};
    return join(p);
}

// Counts (and sums) of the logits of [lo, hi) into bins in LDS, zero before.
// Returns this thread's share of those that pass min_p.
template <bool CAP>
__device__ __forceinline__ Sum fill_bins(const DrawView& D, const Row<CAP>& R, int64_t lo, int64_t hi, uint32_t* count,
                                         uint64_t* mass) {
    Sum above = {0, 0};
    if (R.mode == kCounted) {
        for_logits(R.y, lo, hi, D.vec, [&](float v, int64_t) {
            if (weighs(v)) atomicAdd(&count[R.bin_of(v)], 1u);
        });
        return above;
    }
    for_logits(R.y, lo, hi, D.vec, [&](float v, int64_t) {
        if (!weighs(v)) return;
        const double e = R.exponent(v);
        const uint64_t w = R.mass_of(e);
        const int b = R.bin_of(v);
        atomicAdd(&count[b], 1u);
        atomicAdd(reinterpret_cast<unsigned long long*>(&mass[b]), static_cast<unsigned long long>(w));
        if (e >= R.min_exponent) {
            above.mass += w;
            above.count += 1;
        }
    });
    return above;
}

// Keys of the logits of [lo, hi) in chosen bins, behind *n keys in LDS: at
// most as many as the bins count, which is at most kMostCands.
template <bool CAP>
__device__ __forceinline__ void collect(const DrawView& D, const Row<CAP>& R, const Head& H, int64_t lo, int64_t hi,
                                        uint64_t* keys, uint32_t* n) {
    for_logits(R.y, lo, hi, D.vec, [&](float v, int64_t i) {
        if (weighs(v) && chosen(H, R.bin_of(v))) keys[atomicAdd(n, 1u)] = key_of(v, i);
    });
}

// ------------------------------------------------------------ a row by one workgroup

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_row_kernel(DrawView D) {
    union Lds {
        struct {
            uint64_t mass[kBins];
            uint32_t count[kBins];
        } bins;
        Sorter sorter;
        Digits digits;
    };
    __shared__ Lds S;
    __shared__ Ask ask;
    __shared__ Part parts[kWaves];
    __shared__ uint32_t collected;
    const int64_t m = blockIdx.x;
    const int t = threadIdx.x;
    fill_exp_table();
    const Part p = first_of(D.a.logits + m * D.a.ldl, 0, D.a.V, D.vec, parts);
    Row<CAP> R = row_of<CAP>(D, m, p.best, p.sum, p.count);
    int32_t token = p.best ? index_of(p.best) : -1, n = p.best ? 1 : 0;
    if (R.mode != kFirst) {
        R.level_of_top();
        for (int i = t; i < kBins; i += kThreads) {
            S.bins.count[i] = 0;
            S.bins.mass[i] = 0;
        }
        if (t == 0) collected = 0;
        __syncthreads();
        const Sum mine = fill_bins(D, R, 0, D.a.V, S.bins.count, S.bins.mass);
        Sum above;
        block_before(ask.scan, mine, &above);  // and a barrier behind the atomics
        const Bins B = load_bins(ask, S.bins.count, S.bins.mass, R.mode == kSummed);
        const Head H = choose_bins(ask, R, B, above);
        __syncthreads();
        if (H.cands > kMostCands) {
            draw_by_digits(S.digits, D, R, &token, &n);
        } else {
            collect(D, R, H, 0, D.a.V, S.sorter.key, &collected);
            draw_from_cands(S.sorter, R, B, H, &token, &n);
        }
    }
    store<CAP>(D, m, token, n);
}

// ------------------------------------------------------------ a row by several

__global__ __launch_bounds__(kThreads)
void draw_first_kernel(DrawView D) {
    __shared__ Part parts[kWaves];
    const int64_t m = blockIdx.y, lo = blockIdx.x * D.part_len;
    const int t = threadIdx.x;
    // this part's share of the row's bins
    for (int i = blockIdx.x * kThreads + t; i < kBins; i += D.parts * kThreads) {
        D.count[m * kBins + i] = 0;
        D.mass[m * kBins + i] = 0;
    }
    const Part p = first_of(D.a.logits + m * D.a.ldl, lo, min(lo + D.part_len, D.a.V), D.vec, parts);
    if (t == 0) {
        D.part[m * D.parts + blockIdx.x] = p;
        if (blockIdx.x == 0) D.head[m] = Head{};
    }
}

// The row as its parts say, in every thread of the workgroup.
template <bool CAP>
__device__ __forceinline__ Row<CAP> row_of_parts(const DrawView& D, int64_t m) {
    const int lane = threadIdx.x & (kWave - 1);
    Part p = lane < D.parts ? D.part[m * D.parts + lane] : Part{0, 0.0f, 0};
    p = join(p);
    return row_of<CAP>(D, m, p.best, p.sum, p.count);
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_bins_kernel(DrawView D) {
    __shared__ uint64_t mass[kBins];
    __shared__ uint32_t count[kBins];
    __shared__ Scan scan;
    const int64_t m = blockIdx.y, lo = blockIdx.x * D.part_len;
    const int t = threadIdx.x;
    Row<CAP> R = row_of_parts<CAP>(D, m);
    if (R.mode == kFirst) return;
    fill_exp_table();
    for (int i = t; i < kBins; i += kThreads) {
        count[i] = 0;
        mass[i] = 0;
    }
    __syncthreads();
    R.level_of_top();
    const Sum mine = fill_bins(D, R, lo, min(lo + D.part_len, D.a.V), count, mass);
    __syncthreads();
    if (R.has_min && R.mode == kSummed) {
        Sum above;
        block_before(scan, mine, &above);
        if (t == 0 && above.count) {
            atomicAdd(&D.head[m].above_count, above.count);
            atomicAdd(reinterpret_cast<unsigned long long*>(&D.head[m].above_mass),
                      static_cast<unsigned long long>(above.mass));
        }
    }
    for (int i = t; i < kBins; i += kThreads) {
        if (count[i] == 0) continue;
        atomicAdd(&D.count[m * kBins + i], count[i]);
        if (mass[i])
            atomicAdd(reinterpret_cast<unsigned long long*>(&D.mass[m * kBins + i]),
                      static_cast<unsigned long long>(mass[i]));
    }
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_collect_kernel(DrawView D) {
    __shared__ uint64_t keys[kMostCands];
    __shared__ Ask ask;
    __shared__ uint32_t n, base;
    const int64_t m = blockIdx.y, lo = blockIdx.x * D.part_len;
    const int t = threadIdx.x;
    const Row<CAP> R = row_of_parts<CAP>(D, m);
    if (R.mode == kFirst) return;
    if (t == 0) n = 0;
    const Bins B = load_bins(ask, D.count + m * kBins, D.mass + m * kBins, R.mode == kSummed);
    Head* head = D.head + m;
    const Head H = choose_bins(ask, R, B, {head->above_mass, head->above_count});
    if (blockIdx.x == 0 && t == 0) {
        head->k_bin = H.k_bin;
        head->p_lo = H.p_lo;
        head->p_hi = H.p_hi;
        head->u_lo = H.u_lo;
        head->u_hi = H.u_hi;
        head->cands = H.cands;
    }
    if (H.cands > kMostCands) return;
    collect(D, R, H, lo, min(lo + D.part_len, D.a.V), keys, &n);
    __syncthreads();
    if (n == 0) return;
    if (t == 0) base = atomicAdd(&head->collected, n);
    __syncthreads();
    for (uint32_t i = t; i < n; i += kThreads) D.cand[m * kMostCands + base + i] = keys[i];
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_token_kernel(DrawView D) {
    union Lds {
        Sorter sorter;
        Digits digits;
    };
    __shared__ Lds S;
    const int64_t m = blockIdx.x;
    Row<CAP> R = row_of_parts<CAP>(D, m);
    int32_t token = R.best ? index_of(R.best) : -1, n = R.best ? 1 : 0;
    if (R.mode != kFirst) {
        fill_exp_table();
        __syncthreads();
        R.level_of_top();
        const Head H = D.head[m];
        if (H.cands > kMostCands) {
            draw_by_digits(S.digits, D, R, &token, &n);
        } else {
            const Bins B = load_bins(S.sorter.ask, D.count + m * kBins, D.mass + m * kBins, R.mode == kSummed);
            for (uint32_t i = threadIdx.x; i < H.cands; i += kThreads) S.sorter.key[i] = D.cand[m * kMostCands + i];
            draw_from_cands(S.sorter, R, B, H, &token, &n);
        }
    }
    store<CAP>(D, m, token, n);
}

template <bool CAP>
hipError_t launch(const DrawView& D, hipStream_t stream) {
    const dim3 rows(static_cast<unsigned>(D.a.M)), block(kThreads);
    if (D.parts == 1) {
        hipLaunchKernelGGL(draw_row_kernel<CAP>, rows, block, 0, stream, D);
        return hipGetLastError();
    }
    const dim3 grid(static_cast<unsigned>(D.parts), static_cast<unsigned>(D.a.M));
    hipLaunchKernelGGL(draw_first_kernel, grid, block, 0, stream, D);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draw_bins_kernel<CAP>, grid, block, 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draw_collect_kernel<CAP>, grid, block, 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draw_token_kernel<CAP>, rows, block, 0, stream, D);
    return hipGetLastError();
}

// Workgroups of a row: about 512 in all, 4096 logits each at least.
int parts_of(int64_t V, int64_t M) {
    const int64_t most = (V + 4095) / 4096, want = 512 / M;
    const int64_t parts = want < most ? want : most;
    return static_cast<int>(parts < 1 ? 1 : (parts > kMaxParts ? kMaxParts : parts));
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t draw_ws_bytes(int64_t V, int64_t M) {
    const int parts = parts_of(V, M);
    if (parts == 1) return 256;
    const size_t m = static_cast<size_t>(M);
    return align256(m * static_cast<size_t>(parts) * sizeof(Part)) + align256(m * sizeof(Head)) +
           m * (kBins * (sizeof(uint32_t) + sizeof(uint64_t)) + kMostCands * sizeof(uint64_t));
}

hipError_t launch_logits_draw(const DrawArgs& a, void* ws, hipStream_t stream) {
    DrawView D;
    D.a = a;
    D.twice = a.softcap > 0.0f ? 2.0 * kLog2e / static_cast<double>(a.softcap) : 0.0;
    int bits = 0;  // the smallest with V <= 2^bits
    while ((int64_t{1} << bits) < a.V) ++bits;
    D.q = 62 - bits < 51 ? 62 - bits : 51;
    D.parts = parts_of(a.V, a.M);
    D.part_len = ((a.V + D.parts - 1) / D.parts + 3) / 4 * 4;
    D.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.ldl % 4 == 0;
    const size_t m = static_cast<size_t>(a.M);
    char* p = static_cast<char*>(ws);
    D.part = reinterpret_cast<Part*>(p);
    p += align256(m * static_cast<size_t>(D.parts) * sizeof(Part));
    D.head = reinterpret_cast<Head*>(p);
    p += align256(m * sizeof(Head));
    D.mass = reinterpret_cast<uint64_t*>(p);
    p += m * kBins * sizeof(uint64_t);
    D.cand = reinterpret_cast<uint64_t*>(p);
    p += m * kMostCands * sizeof(uint64_t);
    D.count = reinterpret_cast<uint32_t*>(p);
    return a.softcap > 0.0f ? launch<true>(D, stream) : launch<false>(D, stream);
}

}  // namespace qmv
