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
// Rows with a small top-k need no sums and are read once: the largest logits of
// runs of 64 are counted in bins, the bin where k runs are reached says what the
// first k elements reach at least, and what lies there is collected whole.  Rows
// of temperature 0 end with the first step.
//
// Weights are whole multiples of 2^-q of the row's largest: their sums are
// exact in 64-bit integers in any order, so bins can be summed by atomics and
// a row may be split over workgroups in any way.
//
// A row whose answers lie among more elements than that (thousands of equal
// logits, or nearly) is resolved digit by digit of a 64-bit key (order code of
// the logit, then the index from below) instead: slower, whatever the row (one of
// 262,144 with 20,000 equal largest logits 1.2-1.3 ms).
//
// Four launches for split rows, each of which needs what the one before says of
// the whole row: first elements (and runs), bins, collected elements, answers.
// One row of 262,144 takes 33 us, which is their four chains of dependent loads
// and barriers (4.5, 8.7, 6.8, 9.4); 32 rows with mixed filters 43-49 us, 128 of
// which 97% is masked 81: the first launch reads them at 4.0 TB/s (33 us), and
// rows that need sums are read twice more, from the last-level cache (the second
// time only runs that reach the answers, where they are few).  Short rows
// are one launch, a workgroup each (256 rows of 32,000, top-k: 25 us).
#include <stdint.h>

#include <type_traits>

#include "qmv_device.h"
#include "serve_internal.h"
#include "sort_device.h"
#include "step_device.h"
#include "weights_device.h"

namespace qmv {
namespace {

// Threads of a workgroup, T below.  Besides passing over logits the kernels for
// the bins do what is the same in every thread (a row's parameters, sums to be
// reached): fewer waves of more logits each spend less on it (32 rows, top-p:
// 46 us for the two with 512 threads, 57 with 256, 62 with 1024).  The last
// kernel has a row a workgroup and few elements, and takes what it can (8-11 us;
// 10-14 with 512).
constexpr int kThreads = 1024;
constexpr int kBinThreads = 512;
constexpr int kMostWaves = kThreads / kWave;
constexpr int kBins = 4096;
constexpr float kEqualBins = 3328.0f;
constexpr float kFar = 212991.0f;    // 6 octaves on, at the end of the last bin
constexpr int kMostCands = 4096, kCandsPer = kMostCands / kThreads;
constexpr int kMostCounted = 2048;  // largest top-k that is collected whole
constexpr int kSparse = 256;        // logits of a wave's 1024 that are brought together
constexpr int kRun = 64;            // logits whose largest is kept
constexpr int kMostRuns = 4096;     // of a row by one workgroup
constexpr int kDigitBins = 2048;
constexpr int kMaxParts = kWave;  // a lane a part when they are joined
constexpr int kWorkgroups = 512;   // of a call, about
constexpr int kMostSplit = 512;    // rows that are split, each in two parts at least
constexpr float kMaxLogit = 3.4028234663852886e38f;

struct Sum {
    uint64_t mass;
    uint32_t count;
};

// Neither NaN nor -infinity, by the number's bits.  (y > -infinity says the
// same, but where lanes are counted by it the compiler makes "not equal" of it,
// which NaN is.)
__device__ __forceinline__ bool weighs(float y) {
    const uint32_t b = __float_as_uint(y), from_low = b - 0xff800000u;  // -infinity, then NaN, then 0 ..
    return (from_low & 0x7fffffffu) >= 0x00800000u || b == 0x7f800000u;
}

// The largest of four numbers, NaN dropped (NaN if all are).  The compiler makes
// v_max3_f32 of nested maxima and does not quiet what it gives it, and of a
// signalling NaN the instruction makes NaN, whatever stands beside it.
__device__ __forceinline__ float max4(const float (&v)[4]) {
    return fmaxf(fmaxf(__builtin_canonicalizef(v[0]), __builtin_canonicalizef(v[1])),
                 fmaxf(__builtin_canonicalizef(v[2]), __builtin_canonicalizef(v[3])));
}

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
    uint32_t first_k;  // of rows that are collected whole: how many the first top_k are, 0: all that are collected
};

struct DrawView {
    DrawArgs a;
    double twice;  // 2 log2(e) / softcap
    int q;
    int parts;
    int most_parts;    // with work enough for a workgroup each
    int run_parts;     // of a row by runs where it is collected
    int64_t part_len;  // of the first kernel, a multiple of 64
    bool vec;          // rows are 16-byte aligned
    int64_t runs;      // of a row
    Part* part;        // [M][parts]
    float* run;        // [M][runs]
    Head* head;        // [M]
    uint32_t* count;   // [M][kBins]
    uint64_t* mass;    // [M][kBins]
    uint64_t* cand;    // [M][kMostCands]
};

enum Mode {
    kFirst,    // the first element
    kByRuns,   // the first top_k, found by runs
    kCounted,  // the first top_k, found by counts of all elements
    kSummed
};

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
    // Bins follow the order: 3328 equal steps of the distance from the largest
    // logit, then 128 an octave, up to kFar.  *part: where in the bin, of 4096
    // parts.
    __device__ __forceinline__ int bin_of(float v, int* part = nullptr) const {
        const float x = fminf(fminf(top - fminf(v, kMaxLogit), kMaxLogit) * per_bin, kFar);
        const uint32_t past = __float_as_uint(x) - __float_as_uint(kEqualBins);
        const int e = static_cast<int>(x);
        const bool equal = x < kEqualBins;
        // 12 bits of a float below 4096 lie behind its point
        if (part) *part = equal ? static_cast<int>((x - static_cast<float>(e)) * 4096.0f) : static_cast<int>((past & 0xffffu) >> 4);
        return equal ? e : static_cast<int>(past >> 16) + static_cast<int>(kEqualBins);
    }
    // A logit below this one lies behind bin `b`: what that bin can reach, and
    // more than the roundings of bin_of below it.
    __device__ __forceinline__ float floor_of(int b) const {
        const float e = static_cast<float>(b + 1);
        const float x = e <= kEqualBins ? e
                                        : __uint_as_float(__float_as_uint(kEqualBins) +
                                                          (static_cast<uint32_t>(b + 1 - static_cast<int>(kEqualBins)) << 16));
        const float t = x / per_bin * 1.00001f;
        const float v = top - t - (fabsf(top) + t) * 1e-6f;
        // -infinity, where the bins are infinitely wide, would let masked logits in
        return b < kBins - 1 ? fmaxf(v, -kMaxLogit) : -kMaxLogit;
    }
    // A weight below this logit is below 2^-150: it adds nothing to any sum and
    // passes no min_p, so that such an element need not be collected where it is
    // known how many there are.  (After level_of_top().)
    __device__ __forceinline__ float least_weighing() const {
        double v;
        if constexpr (CAP) {
            // levels are known to 2^-42; cap = softcap * tanh backwards
            const double t = level - 152.0 / w.cap - 0x1p-38;
            if (!(t > -1.0)) return -kMaxLogit;
            v = log2((1.0 + t) / (1.0 - t)) / w.twice;
        } else {
            v = static_cast<double>(top) - 152.0 / w.k;
        }
        return fmaxf(static_cast<float>(v - fabs(v) * 0x1p-23), -kMaxLogit);  // rounded down
    }
    // Below this logit there is nothing to collect for the chosen bins.
    __device__ __forceinline__ float least_of(const Head& H) const {
        const float v = floor_of(max(H.u_hi, max(H.p_hi, H.k_bin)));
        return mode != kSummed && H.first_k ? fmaxf(v, least_weighing()) : v;
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

// A row's arguments.  They are asked for at once, before anything depends on
// one of them: a load takes most of a microsecond, and a kernel here a few.
struct Args {
    float temperature, top_p, min_p, u;
    int32_t top_k;
};

__device__ __forceinline__ Args args_of(const DrawView& D, int64_t m) {
    const float* t = D.a.temperature + m;
    Args A;
    A.temperature = *t;
    A.top_p = *(D.a.top_p ? D.a.top_p + m : t);
    A.min_p = *(D.a.min_p ? D.a.min_p + m : t);
    A.top_k = *(D.a.top_k ? D.a.top_k + m : reinterpret_cast<const int32_t*>(t));
    A.u = D.a.u[m];
    if (!D.a.top_p) A.top_p = 1.0f;
    if (!D.a.min_p) A.min_p = 0.0f;
    if (!D.a.top_k) A.top_k = 0;
    return A;
}

__device__ __forceinline__ bool by_runs(const DrawView& D, const Args& A) {
    return A.temperature > 0.0f && A.top_k > 0 && A.top_k <= kMostCounted && 4 * static_cast<int64_t>(A.top_k) <= D.runs;
}

template <bool CAP>
__device__ __forceinline__ Row<CAP> row_of(const DrawView& D, int64_t m, const Args& A, uint64_t best, float sum,
                                           uint32_t count) {
    Row<CAP> R;
    R.y = D.a.logits + m * D.a.ldl;
    R.best = best;
    const float T = A.temperature, min_p = A.min_p;
    R.mode = kFirst;
    if (best == 0 || !(T > 0.0f)) return R;
    R.top_k = A.top_k;
    R.top_p = A.top_p;
    R.u = A.u;
    R.has_min = min_p > 0.0f;
    R.min_exponent = R.has_min ? log2(static_cast<double>(min_p)) : 0.0;
    R.w.k = kLog2e / static_cast<double>(T);
    R.w.cap = static_cast<double>(D.a.softcap) * R.w.k;
    R.w.twice = D.twice;
    R.unit = static_cast<double>(uint64_t{1} << D.q);
    R.top = logit_of(static_cast<uint32_t>(best >> 32));
    // The equal steps reach to the nearer of twice the mean distance and a
    // weight of 2^-64, all bins 64 times as far: the spread of the logits then
    // matters little.  At a small temperature most of a row lies behind them, in
    // the last bin.  A top-k that ends there is not slower for it: what weighs
    // nothing is counted, not collected (see least_weighing and choose_bins; one
    // row of 262,144 with a top-k of 40 at a temperature of 0.001 25 us, 1122 when
    // it went digit by digit).
    const float mean = count ? fmaxf(R.top - sum / static_cast<float>(count), 0.0f) : 0.0f;
    R.per_bin = fminf(fmaxf(mean > 0.0f ? 0.5f * kEqualBins / mean : 0.0f,
                            static_cast<float>(fmin(R.w.k, 1e28)) * (kEqualBins / 64.0f)), 1e30f);
    // With k runs of the 4096 of 262,144 logits, hardly more than k elements
    // reach the k-th run's largest; where a run in four is asked for, about 1.15 k
    // do, and where more are, the elements are counted themselves.
    R.mode = R.top_k <= 0 || R.top_k > kMostCounted ? kSummed : (by_runs(D, A) ? kByRuns : kCounted);
    return R;
}

// 16 logits of a thread of a workgroup of T, 4 by 4; -infinity past the end.
// `from` is a multiple of 4.  WIDE: a wave's batch is 4 KB in a row (128 rows of
// 262,144 read for their first elements in 33 us, 38 with the four quads a
// workgroup's width apart); else every wave gets its share of a part that is
// less than a batch.
constexpr int kU = 4;
template <int T> constexpr int64_t kStep = kU * 4 * T;  // logits of a workgroup's batch

struct Batch {
    float v[kU][4];
};

template <int T, bool WIDE>
__device__ __forceinline__ int place_of(int j) {  // of a thread's quad j in a batch
    const int t = static_cast<int>(threadIdx.x);
    if constexpr (WIDE) return (t / kWave) * (kU * 4 * kWave) + j * (4 * kWave) + (t & (kWave - 1)) * 4;
    return (j * T + t) * 4;
}

template <int T, bool WIDE = false>
__device__ __forceinline__ Batch load_batch(const float* y, int64_t from, int64_t hi, bool vec) {
    Batch B;
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        const int64_t at = from + place_of<T, WIDE>(j);
        if (vec && at + 4 <= hi) {
            const float4 x = *reinterpret_cast<const float4*>(y + at);
            B.v[j][0] = x.x; B.v[j][1] = x.y; B.v[j][2] = x.z; B.v[j][3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) B.v[j][e] = at + e < hi ? y[at + e] : kNegInf;
        }
    }
    return B;
}

// f(four logits, index of their first) for the logits of [lo, hi); `B` is the
// first batch, and the next one is asked for before a batch is used.
template <int T, bool WIDE, class F>
__device__ __forceinline__ void for_quads(Batch B, const float* y, int64_t lo, int64_t hi, bool vec, F&& f) {
    for (int64_t from = lo; from < hi; from += kStep<T>) {
        Batch next;
        if (from + kStep<T> < hi) next = load_batch<T, WIDE>(y, from + kStep<T>, hi, vec);
#pragma unroll
        for (int j = 0; j < kU; ++j) f(B.v[j], from + place_of<T, WIDE>(j));
        B = next;
    }
}

template <int T, class F>
__device__ __forceinline__ void for_logits(const Batch& B, const float* y, int64_t lo, int64_t hi, bool vec, F&& f) {
    for_quads<T, false>(B, y, lo, hi, vec, [&](const float (&v)[4], int64_t at) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f(v[e], at + e);
    });
}

// Inclusive sums over the wave (ROWS: over each 16 lanes), in lane order, by
// row shifts and broadcasts.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ void add_lanes(Sum& v) {
    const uint32_t lo = static_cast<uint32_t>(v.mass), hi = static_cast<uint32_t>(v.mass >> 32);
    const uint32_t l = __builtin_amdgcn_update_dpp(0, static_cast<int>(lo), CTRL, ROW_MASK, 0xF, false);
    const uint32_t h = __builtin_amdgcn_update_dpp(0, static_cast<int>(hi), CTRL, ROW_MASK, 0xF, false);
    v.mass += (static_cast<uint64_t>(h) << 32) | l;
    v.count += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v.count), CTRL, ROW_MASK, 0xF, false));
}

template <bool ROWS>
__device__ __forceinline__ Sum wave_upto(Sum v) {
    add_lanes<0x111, 0xF>(v);
    add_lanes<0x112, 0xF>(v);
    add_lanes<0x114, 0xF>(v);
    add_lanes<0x118, 0xF>(v);
    if constexpr (!ROWS) {
        add_lanes<0x142, 0xA>(v);
        add_lanes<0x143, 0xC>(v);
    }
    return v;
}

__device__ __forceinline__ Sum of_lane(const Sum& v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(v.mass)), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(v.mass >> 32)), lane);
    return {(static_cast<uint64_t>(hi) << 32) | lo,
            static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v.count), lane))};
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

// Sums of the waves.  Two of them take turns, so that one barrier a scan is
// enough: who writes one of them again has passed the barrier behind its reads.
struct Scan {
    uint64_t mass[2][kMostWaves];
    uint32_t count[2][kMostWaves];
};

// Sums before this thread in thread order, and the total.
template <int T>
__device__ __forceinline__ Sum block_before(Scan& S, int& turn, Sum mine, Sum* total) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
    const Sum upto = wave_upto<false>(mine);
    turn ^= 1;
    if (lane == kWave - 1) {
        S.mass[turn][wave] = upto.mass;
        S.count[turn][wave] = upto.count;
    }
    __syncthreads();
    const Sum mine_of = lane < (T / kWave) ? Sum{S.mass[turn][lane], S.count[turn][lane]} : Sum{0, 0};
    const Sum waves = wave_upto<true>(mine_of);
    *total = of_lane(waves, (T / kWave) - 1);
    Sum before = {upto.mass - mine.mass, upto.count - mine.count};
    if (wave > 0) {
        const Sum w0 = of_lane(waves, wave - 1);
        before.mass += w0.mass;
        before.count += w0.count;
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

// One more in a bin, with a weight that depends on v alone.  Lanes that have
// the same v and bin are one addition, whose weight is kept for the next: rows
// come here for their equal logits, and additions to one place would be done one
// by one (262,144 equal logits: 4.8 ms, now 1.0).
struct Kept {
    uint32_t v;
    uint64_t weight;
};

template <class F>
__device__ __forceinline__ void add_equal(Kept& kept, float v, uint32_t bin, uint32_t* count, uint64_t* mass, F&& weight) {
    const uint32_t v0 = __builtin_amdgcn_readfirstlane(__float_as_uint(v)), b0 = __builtin_amdgcn_readfirstlane(bin);
    const uint64_t here = __ballot(1), equal = __ballot(__float_as_uint(v) == v0 && bin == b0);
    if (here == equal) {
        if (kept.v != v0) {
            kept.v = v0;
            kept.weight = weight();
        }
        const uint32_t n = static_cast<uint32_t>(__popcll(here));
        if ((threadIdx.x & (kWave - 1)) == static_cast<uint32_t>(__ffsll(static_cast<unsigned long long>(here))) - 1) {
            atomicAdd(&count[bin], n);
            atomicAdd(reinterpret_cast<unsigned long long*>(&mass[bin]), static_cast<unsigned long long>(kept.weight * n));
        }
    } else {
        atomicAdd(&count[bin], 1u);
        atomicAdd(reinterpret_cast<unsigned long long*>(&mass[bin]), static_cast<unsigned long long>(weight()));
    }
}

struct Found {
    uint64_t key;
    Sum upto;  // sums up to and with the element
};

// The first element of the order whose running count (mass: running sum)
// reaches `need`, 1 <= need <= the row's.
template <bool CAP>
__device__ __noinline__ Found find(Digits& S, int& turn, const DrawView& D, const Row<CAP>& R, bool mass, uint64_t need) {
    uint64_t prefix = 0;
    Sum before = {0, 0}, upto = {0, 0};
    const int t = threadIdx.x;
    constexpr int kLow[6] = {53, 42, 32, 21, 10, 0};
    Kept kept = {0x7fc00000u, 0};  // NaN, which does not come
    for (int d = 0; d < 6; ++d) {
        const int low = kLow[d], high = d == 0 ? 64 : kLow[d - 1];
        const uint32_t digits = (1u << (high - low)) - 1u;
        __syncthreads();
        for (int i = t; i < kDigitBins; i += kThreads) {
            S.mass[i] = 0;
            S.count[i] = 0;
        }
        __syncthreads();
        for_logits<kThreads>(load_batch<kThreads>(R.y, 0, D.a.V, D.vec), R.y, 0, D.a.V, D.vec, [&](float v, int64_t i) {
            if (!weighs(v)) return;
            const uint64_t key = key_of(v, i);
            if (d > 0 && (key >> high) != (prefix >> high)) return;
            const uint32_t bin = digits - (static_cast<uint32_t>(key >> low) & digits);  // bin 0: first in the order
            add_equal(kept, v, bin, S.count, S.mass, [&] { return R.mass_of(R.exponent(v)); });
        });
        __syncthreads();
        constexpr int kPer = kDigitBins / kThreads;
        Sum mine = {0, 0}, total;
        for (int j = 0; j < kPer; ++j) {
            mine.mass += S.mass[kPer * t + j];
            mine.count += S.count[kPer * t + j];
        }
        Sum run = block_before<kThreads>(S.scan, turn, mine, &total);
        run.mass += before.mass;
        run.count += before.count;
        for (int j = 0; j < kPer; ++j) {
            const Sum next = {run.mass + S.mass[kPer * t + j], run.count + S.count[kPer * t + j]};
            if (reaches(run, next, mass, need)) S.hit = {run, next, kPer * t + j};
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
__device__ __noinline__ void draw_by_digits(Digits& S, const DrawView& D, const Row<CAP>& R, int32_t* token, int32_t* n) {
    Sum mine = {0, 0}, above = {0, 0}, total, kept;
    int turn = 0;
    for_logits<kThreads>(load_batch<kThreads>(R.y, 0, D.a.V, D.vec), R.y, 0, D.a.V, D.vec, [&](float v, int64_t) {
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
    __syncthreads();
    block_before<kThreads>(S.scan, turn, above, &kept);
    block_before<kThreads>(S.scan, turn, mine, &total);
    if (!R.has_min) kept = total;
    if (kept.count == 0) kept = {static_cast<uint64_t>(R.unit), 1};
    Sum of_k = total;
    if (R.top_k > 0 && static_cast<uint32_t>(R.top_k) < total.count)
        of_k = find(S, turn, D, R, false, static_cast<uint64_t>(R.top_k)).upto;
    if (of_k.count < kept.count) kept = of_k;
    if (R.top_p < 1.0f) {
        const Sum of_p = find(S, turn, D, R, true, at_least_1(R.need_p(of_k.mass))).upto;
        if (of_p.count < kept.count) kept = of_p;
    }
    *n = static_cast<int32_t>(kept.count);
    *token = index_of(find(S, turn, D, R, true, at_least_1(R.need_u(kept.mass))).key);
}

// The same on copies: what the caller holds stays in registers.
template <bool CAP>
__device__ __forceinline__ void by_digits(Digits& S, const DrawView& D, const Row<CAP>& R, int32_t* token, int32_t* n) {
    const DrawView view = D;
    const Row<CAP> row = R;
    int32_t a, b;
    draw_by_digits(S, view, row, &a, &b);
    *token = a;
    *n = b;
}

// ------------------------------------------------------------ by bins

// The bins of a row with their running sums: a thread holds kPer neighbours.
template <int T>
struct Bins {
    static constexpr int kPer = kBins / T;
    Sum bin[kPer];
    Sum own, before, total;
};

struct Ask {
    Scan scan;
    Hit hit[5];
};

// The bins as they lie in memory.
template <int T>
__device__ __forceinline__ Bins<T> load_bins(const uint32_t* count, const uint64_t* mass) {
    Bins<T> B;
    constexpr int kPer = Bins<T>::kPer;
#pragma unroll
    for (int j = 0; j < Bins<T>::kPer; ++j) {
        B.bin[j].count = count[kPer * threadIdx.x + j];
        B.bin[j].mass = mass[kPer * threadIdx.x + j];
    }
    return B;
}

template <int T>
__device__ __forceinline__ void sum_bins(Ask& S, int& turn, Bins<T>& B) {
    Sum mine = {0, 0};
#pragma unroll
    for (int j = 0; j < Bins<T>::kPer; ++j) {
        mine.mass += B.bin[j].mass;
        mine.count += B.bin[j].count;
    }
    B.own = mine;
    B.before = block_before<T>(S.scan, turn, mine, &B.total);
}

// The thread whose bin reaches `need` says so in hit[slot].
template <int T>
__device__ __forceinline__ void ask_bins(Ask& S, const Bins<T>& B, int slot, bool mass, uint64_t need) {
    Sum run = B.before;
    if (!reaches(run, {run.mass + B.own.mass, run.count + B.own.count}, mass, need)) return;
#pragma unroll
    for (int j = 0; j < Bins<T>::kPer; ++j) {
        const Sum next = {run.mass + B.bin[j].mass, run.count + B.bin[j].count};
        if (reaches(run, next, mass, need)) S.hit[slot] = {run, next, Bins<T>::kPer * static_cast<int>(threadIdx.x) + j};
        run = next;
    }
}

// Bins that hold the answers, in every thread; *reach: elements up to the last
// of them.
template <bool CAP, int T>
__device__ __forceinline__ Head choose_bins(Ask& S, const Row<CAP>& R, const Bins<T>& B, Sum above, uint32_t* reach) {
    Head H = {above.mass, above.count, 0, -1, 0, -1, 0, -1, 0};
    const uint32_t kk = R.top_k > 0 && static_cast<uint32_t>(R.top_k) < B.total.count ? R.top_k : B.total.count;
    if (R.mode != kSummed) {  // the first kk whole (of runs: fewer than k may be there, then all)
        ask_bins(S, B, 0, false, kk);
        __syncthreads();
        const bool all = R.mode == kByRuns && B.total.count < static_cast<uint32_t>(R.top_k);
        H.u_hi = all ? kBins - 1 : S.hit[0].at;
        H.first_k = all ? 0 : kk;
        *reach = S.hit[0].upto.count;
        return H;
    }
    *reach = 0;
    uint64_t k_lo = B.total.mass, k_hi = B.total.mass;
    if (kk < B.total.count) {
        ask_bins(S, B, 0, false, kk);
        __syncthreads();
        const Hit h = S.hit[0];
        k_lo = k_hi = h.upto.mass;
        if (h.upto.count != kk && h.upto.mass != h.before.mass) {  // whichever of a bin of zeros are among them
            H.k_bin = h.at;
            k_lo = h.before.mass;
            *reach = h.upto.count;
        }
    }
    uint64_t lo = k_lo, hi = k_hi;
    if (R.top_p < 1.0f) {
        ask_bins(S, B, 1, true, at_least_1(R.need_p(k_lo)));
        ask_bins(S, B, 2, true, at_least_1(R.need_p(k_hi)));
        __syncthreads();
        H.p_lo = S.hit[1].at;
        H.p_hi = S.hit[2].at;
        *reach = max(*reach, S.hit[2].upto.count);
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
    *reach = max(*reach, S.hit[4].upto.count);
    return H;
}

__device__ __forceinline__ bool chosen(const Head& H, int b) {
    return b == H.k_bin || (b >= H.p_lo && b <= H.p_hi) || (b >= H.u_lo && b <= H.u_hi);
}

// The chosen bins numbered through: the three ranges follow each other, since
// what is drawn is kept, and what is kept is among the first k.
struct Chosen {
    int u_lo, u_hi, p_lo, p_hi, count, per;  // per: buckets a bin
    __device__ __forceinline__ explicit Chosen(const Head& H) {
        u_lo = H.u_lo;
        u_hi = H.u_hi;
        p_lo = max(H.p_lo, u_hi + 1);
        p_hi = max(H.p_hi, p_lo - 1);
        count = (u_hi - u_lo + 1) + (p_hi - p_lo + 1) + 1;
        per = max(kMostCands / count, 1);
    }
    __device__ __forceinline__ int bucket(int bin, int part) const {
        const int i = bin <= u_hi ? bin - u_lo : (u_hi - u_lo + 1) + (bin <= p_hi ? bin - p_lo : p_hi - p_lo + 1);
        return min(i * per + ((part * per) >> 12), kMostCands - 1);
    }
};

struct Sorter {
    uint64_t key[kMostCands], sorted[kMostCands];
    uint32_t start[kMostCands + 1];
    Ask ask;
    Hit hit[3];
    uint32_t above;
};

// Sorts n <= kMostCands keys, first of the order first: thread t has keys t,
// t + 1024, .. (anything past the n-th) and gets keys 4 t .. 4 t + 3 (0 past
// the end).  Up to 64 by exchanges in a wave; more go to 4096 buckets, equal
// parts of the chosen bins, of which most hold one or none, and are ranked in
// theirs.  (Exchanges among 1024 threads take 36 to 78 steps.)  Equal logits
// share a bucket, where each is compared with all: 1000 of them in one of 262,144
// take 73-127 us a row, 4000 780.
template <bool CAP>
__device__ __forceinline__ void sort_cands(Sorter& S, int& turn, const Row<CAP>& R, const Head& H, uint32_t n,
                                           uint64_t (&mine)[kCandsPer]) {
    const int t = threadIdx.x;
    if (n <= kWave) {
        if (t < kWave) {
            uint64_t key[1] = {t < n ? mine[0] : 0};
            wave_sort_desc(key);
            S.sorted[t] = key[0];
        }
    } else {
        const Chosen C(H);
        int bucket[kCandsPer];
        uint32_t slot[kCandsPer];
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) S.start[j * kThreads + t] = 0;
        if (t == 0) S.start[kMostCands] = n;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            if (j * kThreads + t >= n) continue;
            int part;
            const int bin = R.bin_of(logit_of(static_cast<uint32_t>(mine[j] >> 32)), &part);
            bucket[j] = C.bucket(bin, part);
            slot[j] = atomicAdd(&S.start[bucket[j]], 1u);
        }
        __syncthreads();
        uint32_t in[kCandsPer];
        Sum own = {0, 0}, total;
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            in[j] = S.start[kCandsPer * t + j];
            own.count += in[j];
        }
        uint32_t before = block_before<kThreads>(S.ask.scan, turn, own, &total).count;
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            S.start[kCandsPer * t + j] = before;
            before += in[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j)
            if (j * kThreads + t < n) S.key[S.start[bucket[j]] + slot[j]] = mine[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            if (j * kThreads + t >= n) continue;
            const uint32_t lo = S.start[bucket[j]], hi = S.start[bucket[j] + 1];
            uint32_t rank = lo;
            for (uint32_t i = lo; i < hi; ++i) rank += S.key[i] > mine[j] ? 1u : 0u;
            S.sorted[rank] = mine[j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCandsPer; ++j) mine[j] = kCandsPer * t + j < n ? S.sorted[kCandsPer * t + j] : 0;
}

// The answers among the n collected elements of a row (sort_cands says how a
// thread holds them).
template <bool CAP>
__device__ __forceinline__ void draw_from_cands(Sorter& S, int& turn, const Row<CAP>& R, const Bins<kThreads>& B, const Head& H,
                                                uint32_t n_cands, uint64_t (&key)[kCandsPer], int32_t* token, int32_t* n) {
    const int t = threadIdx.x;
    const bool whole = R.mode != kSummed;  // the first k are here
    if (t == 0) S.above = 0;
    sort_cands(S, turn, R, H, n_cands, key);
    Sum w[kCandsPer], kept, of_k;
    if (whole) {
        uint32_t above = 0;
        Sum own = {0, 0};
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            w[j] = {0, 0};
            if (key[j] && kCandsPer * t + j < R.top_k) {
                const double e = R.exponent(logit_of(static_cast<uint32_t>(key[j] >> 32)));
                w[j] = {R.mass_of(e), 1u};
                above += e >= R.min_exponent ? 1u : 0u;
            }
            own.mass += w[j].mass;
            own.count += w[j].count;
        }
        if (R.has_min && above) atomicAdd(&S.above, above);
        const Sum before = block_before<kThreads>(S.ask.scan, turn, own, &of_k);
        if (H.first_k) of_k.count = H.first_k;  // with those that weigh nothing
        auto ask = [&](int slot, bool mass, uint64_t need) {
            Sum run = before;
#pragma unroll
            for (int j = 0; j < kCandsPer; ++j) {
                const Sum next = {run.mass + w[j].mass, run.count + w[j].count};
                if (reaches(run, next, mass, need)) S.hit[slot] = {run, next, kCandsPer * t + j};
                run = next;
            }
            __syncthreads();
            return S.hit[slot];
        };
        kept = of_k;
        if (R.top_p < 1.0f) kept = ask(0, true, at_least_1(R.need_p(of_k.mass))).upto;
        if (R.has_min && S.above < kept.count) kept = ask(1, false, max(S.above, 1u)).upto;
        *n = static_cast<int32_t>(kept.count);
        *token = index_of(S.sorted[ask(2, true, at_least_1(R.need_u(kept.mass))).at]);
        return;
    }
    int bin[kCandsPer];
#pragma unroll
    for (int j = 0; j < kCandsPer; ++j) {
        bin[j] = -1;
        w[j] = {0, 0};
        if (key[j]) {
            const float v = logit_of(static_cast<uint32_t>(key[j] >> 32));
            bin[j] = R.bin_of(v);
            w[j] = {R.mass_of(R.exponent(v)), 1u};
        }
    }
    // the element that reaches `need`, in the bin that does
    auto ask = [&](int slot, bool mass, uint64_t need) -> Hit {
        ask_bins(S.ask, B, slot, mass, need);
        __syncthreads();
        const Hit of = S.ask.hit[slot];
        Sum own = {0, 0}, in[kCandsPer], total;
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            in[j] = bin[j] == of.at ? w[j] : Sum{0, 0};
            own.mass += in[j].mass;
            own.count += in[j].count;
        }
        Sum run = block_before<kThreads>(S.ask.scan, turn, own, &total);
        run.mass += of.before.mass;
        run.count += of.before.count;
#pragma unroll
        for (int j = 0; j < kCandsPer; ++j) {
            const Sum next = {run.mass + in[j].mass, run.count + in[j].count};
            if (reaches(run, next, mass, need)) S.hit[slot] = {run, next, kCandsPer * t + j};
            run = next;
        }
        __syncthreads();
        return S.hit[slot];
    };
    const uint32_t kk = R.top_k > 0 && static_cast<uint32_t>(R.top_k) < B.total.count ? R.top_k : B.total.count;
    of_k = B.total;
    if (H.k_bin >= 0) {
        of_k = ask(0, false, kk).upto;
    } else if (kk < B.total.count) {  // the end of a bin, or among zeros
        ask_bins(S.ask, B, 0, false, kk);
        __syncthreads();
        of_k = {S.ask.hit[0].upto.mass, kk};
    }
    kept = of_k;
    if (R.has_min && H.above_count < kept.count) kept = {H.above_mass, H.above_count};
    if (kept.count == 0) kept = {static_cast<uint64_t>(R.unit), 1};
    if (R.top_p < 1.0f) {
        const Sum of_p = ask(1, true, at_least_1(R.need_p(of_k.mass))).upto;
        if (of_p.count < kept.count) kept = of_p;
    }
    *n = static_cast<int32_t>(kept.count);
    *token = index_of(S.sorted[ask(2, true, at_least_1(R.need_u(kept.mass))).at]);
}

__device__ __forceinline__ void store(const DrawView& D, int64_t m, int32_t token, int32_t n) {
    if (threadIdx.x == 0) {
        D.a.token[m] = token;
        if (D.a.kept) D.a.kept[m] = n;
    }
}

// ------------------------------------------------------------ steps of a part

__device__ __forceinline__ float max16(float v) {  // over 16 lanes, in the last one
    auto step = [](float x, auto ctrl) {
        const int b = __builtin_bit_cast(int, x);
        return fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, decltype(ctrl)::value, 0xF, 0xF, false)));
    };
    v = step(v, std::integral_constant<int, 0x111>{});
    v = step(v, std::integral_constant<int, 0x112>{});
    v = step(v, std::integral_constant<int, 0x114>{});
    return step(v, std::integral_constant<int, 0x118>{});
}

// The first element of [lo, hi), and the largest logits of its runs to `run`
// (null: not wanted).  A run is what 16 lanes hold of a batch.  One logit in
// four is enough for their mean.
template <int T, bool WIDE>
__device__ __forceinline__ Part first_of(const float* y, int64_t lo, int64_t hi, bool vec, Part* lds, float* run) {
    float best = kNegInf, sum = 0.0f;
    int32_t at_best = 0;
    uint32_t count = 0;
    for_quads<T, WIDE>(load_batch<T, WIDE>(y, lo, hi, vec), y, lo, hi, vec, [&](const float (&v)[4], int64_t at) {
        // NaN is dropped; a NaN that is left is not larger than anything
        float top = fminf(max4(v), kMaxLogit);
        top = v[0] != v[0] && v[1] != v[1] && v[2] != v[2] && v[3] != v[3] ? kNegInf : top;
        at_best = top > best ? static_cast<int32_t>(at) : at_best;  // a thread goes through rising indexes
        best = fmaxf(best, top);
        const bool ordinary = fabsf(v[0]) < 1e6f;  // false for NaN
        sum += ordinary ? v[0] : 0.0f;
        count += ordinary ? 1 : 0;
        if (run) {
            top = max16(top);
            if ((threadIdx.x & 15) == 15 && at - 60 < hi) run[static_cast<uint32_t>(at) / kRun] = top;
        }
    });
    Part p = {0, sum, count};
    if (best > kNegInf) {
        int place = 3;
#pragma unroll
        for (int e = 2; e >= 0; --e) place = at_best + e < hi && y[at_best + e] >= best ? e : place;  // +infinity reaches it, NaN does not
        p.best = key_of(best, at_best + place);
    }
    p = join(p);
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    if (lane == 0) lds[wave] = p;
    __syncthreads();
    p = lane < T / kWave ? lds[lane] : Part{0, 0.0f, 0};
    return join(p);
}

// Whether the wave's batch is one number.
__device__ __forceinline__ bool all_equal(const Batch& B) {
    const uint32_t first = __builtin_amdgcn_readfirstlane(__float_as_uint(B.v[0][0]));
    bool same = true;
#pragma unroll
    for (int j = 0; j < kU; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) same = same && __float_as_uint(B.v[j][e]) == first;
    return __ballot(same) == ~uint64_t{0};
}

// Counts (and sums) of the logits of [lo, hi) into bins in LDS, zero before;
// sparse: kSparse floats a wave, of its own.
// Returns this thread's share of those that pass min_p.
template <int T, bool CAP>
__device__ __forceinline__ Sum fill_bins(const Batch& first, const DrawView& D, const Row<CAP>& R, int64_t lo, int64_t hi,
                                         uint32_t* count, uint64_t* mass, float* sparse) {
    Sum above = {0, 0};
    if (R.mode == kCounted) {
        for_quads<T, false>(first, R.y, lo, hi, D.vec, [&](const float (&v)[4], int64_t) {
            const bool same = v[0] == v[1] && v[0] == v[2] && v[0] == v[3] && weighs(v[0]) &&
                              __float_as_uint(v[0]) == __builtin_amdgcn_readfirstlane(__float_as_uint(v[0]));
            if (__ballot(same) == ~uint64_t{0}) {
                if ((threadIdx.x & (kWave - 1)) == 0) atomicAdd(&count[R.bin_of(v[0])], 4u * kWave);
                return;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (weighs(v[e])) atomicAdd(&count[R.bin_of(v[e])], 1u);
        });
        return above;
    }
    auto add = [&](float v, uint32_t n = 1) {
        const double e = R.exponent(v);
        const uint64_t w = R.mass_of(e) * n;
        const int b = R.bin_of(v);
        atomicAdd(&count[b], n);
        atomicAdd(reinterpret_cast<unsigned long long*>(&mass[b]), static_cast<unsigned long long>(w));
        if (e >= R.min_exponent) {
            above.mass += w;
            above.count += n;
        }
    };
    const int lane = threadIdx.x & (kWave - 1);
    float* mine = sparse + (threadIdx.x / kWave) * kSparse;
    Batch B = first;
    for (int64_t from = lo; from < hi; from += kStep<T>) {
        Batch next;
        if (from + kStep<T> < hi) next = load_batch<T>(R.y, from + kStep<T>, hi, D.vec);
        uint32_t n = 0;
#pragma unroll
        for (int j = 0; j < kU; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) n += static_cast<uint32_t>(__popcll(__ballot(weighs(B.v[j][e]))));
        if (n <= kSparse) {
            // mostly forbidden tokens: the others side by side, so that a
            // weight is not formed for 64 lanes where two have one
            uint32_t at = 0;
#pragma unroll
            for (int j = 0; j < kU; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t some = __ballot(weighs(B.v[j][e]));
                    if (weighs(B.v[j][e])) mine[at + __popcll(some & ((uint64_t{1} << lane) - 1))] = B.v[j][e];
                    at += static_cast<uint32_t>(__popcll(some));
                }
            __builtin_amdgcn_wave_barrier();
            for (uint32_t i = lane; i < n; i += kWave) add(mine[i]);
            __builtin_amdgcn_wave_barrier();
        } else if (n == kU * 4 * kWave && all_equal(B)) {
            if (lane == 0) add(B.v[0][0], n);  // a row that nobody uses, say
        } else {
#pragma unroll
            for (int j = 0; j < kU; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (weighs(B.v[j][e])) add(B.v[j][e]);
        }
        B = next;
    }
    return above;
}

// Keys of the logits of [lo, hi) in chosen bins, to LDS; *n counts them, also
// those for which there is no room.
template <int T, bool CAP>
__device__ __forceinline__ void collect(const Batch& first, const DrawView& D, const Row<CAP>& R, const Head& H, int64_t lo,
                                        int64_t hi, uint64_t* keys, uint32_t* n) {
    // four at a time are dropped, most of them (NaN is not above anything)
    const float least = R.least_of(H);
    for_quads<T, false>(first, R.y, lo, hi, D.vec, [&](const float (&v)[4], int64_t i) {
        if (!(max4(v) >= least)) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!(v[e] >= least) || !chosen(H, R.bin_of(v[e]))) continue;
            const uint32_t at = atomicAdd(n, 1u);
            if (at < kMostCands) keys[at] = key_of(v[e], i + e);
        }
    });
}

// Counts of the runs' largest logits in bins in LDS, zero before.
template <int T, bool CAP>
__device__ __forceinline__ void count_runs(const Row<CAP>& R, const float* run, int64_t runs, uint32_t* count) {
    const int t = threadIdx.x;
    for (int64_t i = t; i < runs; i += 8 * T) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j * T < runs ? run[i + j * T] : kNegInf;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool same = weighs(v[j]) && __float_as_uint(v[j]) == __builtin_amdgcn_readfirstlane(__float_as_uint(v[j]));
            if (__ballot(same) == ~uint64_t{0}) {
                if ((t & (kWave - 1)) == 0) atomicAdd(&count[R.bin_of(v[j])], static_cast<uint32_t>(kWave));
            } else if (weighs(v[j])) {
                atomicAdd(&count[R.bin_of(v[j])], 1u);
            }
        }
    }
}

// The same where few runs reach the bins: only those are read, by 16 threads
// each.  list: 4 T numbers in LDS; *listed and *n are 0 before, behind a barrier.
template <int T, bool CAP>
__device__ __forceinline__ void collect_runs(const DrawView& D, const Row<CAP>& R, const Head& H, const float* run, int64_t lo,
                                             int64_t hi, int32_t* list, uint32_t* listed, uint64_t* keys, uint32_t* n) {
    const int last = max(H.u_hi, max(H.p_hi, H.k_bin));
    const float least = R.least_of(H);  // drops most (and NaN) by one comparison
    const int t = threadIdx.x;
    const int64_t r0 = lo / kRun, r1 = (hi + kRun - 1) / kRun;
    for (int64_t r = r0; r < r1; r += 4 * T) {
        float top[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j] = r + j * T + t < r1 ? run[r + j * T + t] : kNegInf;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (top[j] >= least && R.bin_of(top[j]) <= last)
                list[atomicAdd(listed, 1u)] = static_cast<int32_t>(r + j * T + t - r0);
        __syncthreads();
        const uint32_t have = *listed;
        for (uint32_t i = t / 16; i < have; i += 4 * (T / 16)) {  // four at a time
            float v[4][4];
            int64_t at[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t k = i + j * (T / 16);
                at[j] = k < have ? (r0 + list[k]) * kRun + (t & 15) * 4 : hi;
                if (D.vec && at[j] + 4 <= hi) {
                    const float4 x = *reinterpret_cast<const float4*>(R.y + at[j]);
                    v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] = at[j] + e < hi ? R.y[at[j] + e] : kNegInf;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!(v[j][e] >= least) || !chosen(H, R.bin_of(v[j][e]))) continue;
                    const uint32_t to = atomicAdd(n, 1u);
                    if (to < kMostCands) keys[to] = key_of(v[j][e], at[j] + e);
                }
        }
        __syncthreads();
        if (t == 0) *listed = 0;
        __syncthreads();
    }
}

// Whether collect_runs() pays where so many elements of a row reach the bins: at
// most half the runs do, and there are enough of them.  (Top-p 0.9 of a few kept
// tokens, with this and without: 128 rows of 262,144 126 and 145 us, of 50,257 57
// and 66; in parts of 4096 a row takes 31 us and 29.)
constexpr int64_t kDirect = 32768;
__device__ __forceinline__ bool few_runs(const DrawView& D, uint32_t reach, int64_t len) {
    return len > kDirect && 2 * static_cast<int64_t>(reach) <= D.runs;
}

// ------------------------------------------------------------ a row by one workgroup

struct BinLds {
    uint64_t mass[kBins];
    uint32_t count[kBins];
    float sparse[kMostWaves * kSparse];
};

union RowLds {
    BinLds bins;
    Sorter sorter;
    Digits digits;
};

// What of a row holds the answers, by bins of all its elements: keys to
// S.sorter.key, returns how many.
template <bool CAP>
__device__ __forceinline__ uint32_t by_bins(RowLds& S, Ask& ask, uint32_t& collected, uint32_t& listed, int& turn,
                                            const DrawView& D, const Row<CAP>& R, const float* run, Bins<kThreads>& B, Head& H) {
    const int t = threadIdx.x;
    const int64_t V = D.a.V;
    for (int i = t; i < kBins; i += kThreads) {
        S.bins.count[i] = 0;
        S.bins.mass[i] = 0;
    }
    if (t == 0) collected = listed = 0;
    const Batch again = load_batch<kThreads>(R.y, 0, V, D.vec);
    __syncthreads();
    const Sum mine = fill_bins<kThreads>(again, D, R, 0, V, S.bins.count, S.bins.mass, S.bins.sparse);
    Sum above;
    block_before<kThreads>(ask.scan, turn, mine, &above);  // and a barrier behind the atomics
    B = load_bins<kThreads>(S.bins.count, S.bins.mass);
    sum_bins(ask, turn, B);  // and one behind the loads
    uint32_t reach;
    H = choose_bins(ask, R, B, above, &reach);
    if (few_runs(D, reach, V))
        collect_runs<kThreads>(D, R, H, run, 0, V, reinterpret_cast<int32_t*>(S.sorter.sorted), &listed, S.sorter.key, &collected);
    else
        collect<kThreads>(load_batch<kThreads>(R.y, 0, V, D.vec), D, R, H, 0, V, S.sorter.key, &collected);
    __syncthreads();
    return collected;
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_row_kernel(DrawView D) {
    __shared__ RowLds S;
    __shared__ Ask ask;
    __shared__ Part parts[kMostWaves];
    __shared__ float run[kMostRuns];
    __shared__ uint32_t collected, listed;
    const int64_t m = blockIdx.x, V = D.a.V;
    const int t = threadIdx.x;
    const Args A = args_of(D, m);
    fill_exp_table();
    const float* y = D.a.logits + m * D.a.ldl;
    const Part p = first_of<kThreads, true>(y, 0, V, D.vec, parts, D.runs > 0 && (V > kDirect || by_runs(D, A)) ? run : nullptr);
    Row<CAP> R = row_of<CAP>(D, m, A, p.best, p.sum, p.count);
    int32_t token = p.best ? index_of(p.best) : -1, n = p.best ? 1 : 0;
    if (R.mode != kFirst) {
        int turn = 0;
        uint32_t found = 0;
        Bins<kThreads> B;
        Head H;
        R.level_of_top();
        if (R.mode == kByRuns) {
            for (int i = t; i < kBins; i += kThreads) {
                S.bins.count[i] = 0;
                S.bins.mass[i] = 0;
            }
            if (t == 0) collected = listed = 0;
            __syncthreads();
            count_runs<kThreads>(R, run, D.runs, S.bins.count);
            __syncthreads();
            B = load_bins<kThreads>(S.bins.count, S.bins.mass);
            sum_bins(ask, turn, B);
            uint32_t reach;
            H = choose_bins(ask, R, B, {0, 0}, &reach);
            collect_runs<kThreads>(D, R, H, run, 0, V, reinterpret_cast<int32_t*>(S.sorter.sorted), &listed, S.sorter.key,
                                   &collected);
            found = collected;
            if (found > kMostCands) {  // see draw_token_kernel
                R.mode = kCounted;
                __syncthreads();  // collected is read before it is written
            }
        }
        if (R.mode != kByRuns) found = by_bins(S, ask, collected, listed, turn, D, R, run, B, H);
        if (found > kMostCands) {
            by_digits(S.digits, D, R, &token, &n);
        } else {
            uint64_t key[kCandsPer];
#pragma unroll
            for (int j = 0; j < kCandsPer; ++j) key[j] = S.sorter.key[j * kThreads + t];
            __syncthreads();
            draw_from_cands(S.sorter, turn, R, B, H, found, key, &token, &n);
        }
    }
    store(D, m, token, n);
}

// ------------------------------------------------------------ a row by several

template <bool WIDE>
__global__ __launch_bounds__(kThreads)
void draw_first_kernel(DrawView D) {
    __shared__ Part parts[kMostWaves];
    const int64_t m = blockIdx.y, lo = blockIdx.x * D.part_len;
    const int t = threadIdx.x;
    const Args A = args_of(D, m);
    // this part's share of the row's bins
    for (int i = blockIdx.x * kThreads + t; i < kBins; i += D.parts * kThreads) {
        D.count[m * kBins + i] = 0;
        D.mass[m * kBins + i] = 0;
    }
    const Part p = first_of<kThreads, WIDE>(D.a.logits + m * D.a.ldl, lo, min(lo + D.part_len, D.a.V), D.vec, parts,
                            A.temperature > 0.0f ? D.run + m * D.runs : nullptr);
    if (t == 0) {
        D.part[m * D.parts + blockIdx.x] = p;
        if (blockIdx.x == 0) D.head[m] = Head{};
    }
}

// What the parts say about a row, in every thread.
__device__ __forceinline__ Part part_of(const DrawView& D, int64_t m) {
    const int lane = threadIdx.x & (kWave - 1);
    return lane < D.parts ? D.part[m * D.parts + lane] : Part{0, 0.0f, 0};
}

// A share of the work of the bins or collect kernel: a part of a row.
struct Unit {
    int64_t m, lo, hi;
    bool some, runs;
};

struct Shares {
    uint64_t by_runs[kMostSplit / kWave], others[kMostSplit / kWave];
    int32_t row;
};

// Which rows there are is known on the device only: rows by runs need hardly
// any work in these two kernels, and rows of temperature 0 none.  The
// workgroups share out the others: every row by runs is `run_parts` units, and
// the other rows have what is left in equal parts.
__device__ __forceinline__ Unit unit_of(Shares& S, const DrawView& D, int run_parts) {
    const int t = threadIdx.x, M = static_cast<int>(D.a.M);
    Unit U = {0, 0, D.a.V, false, false};
    int part = blockIdx.x, parts = D.parts;
    if (M > 1) {
        if (t < kMostSplit) {  // whole waves
            bool runs = false, other = false;
            if (t < M) {
                const Args A = args_of(D, t);
                runs = by_runs(D, A);
                other = A.temperature > 0.0f && !runs;
            }
            const uint64_t r = __ballot(runs), o = __ballot(other);
            if ((t & (kWave - 1)) == 0) {
                S.by_runs[t / kWave] = r;
                S.others[t / kWave] = o;
            }
        }
        __syncthreads();
        int n_runs = 0, n_others = 0;
#pragma unroll
        for (int i = 0; i < kMostSplit / kWave; ++i) {
            n_runs += __popcll(S.by_runs[i]);
            n_others += __popcll(S.others[i]);
        }
        int unit = blockIdx.x, nth;
        const bool runs = unit < n_runs * run_parts;
        if (runs) {
            parts = run_parts;
        } else {
            unit -= n_runs * run_parts;
            if (n_others == 0) return U;
            // the rows are at most half the workgroups, so that this is at least 1
            parts = min((static_cast<int>(gridDim.x) - n_runs * run_parts) / n_others, D.most_parts);
        }
        nth = unit / parts;
        part = unit - nth * parts;
        if (nth >= (runs ? n_runs : n_others)) return U;
        // the thread of that row finds itself
        if (t < kMostSplit) {
            const uint64_t* mask = runs ? S.by_runs : S.others;
            int before = 0;
            for (int i = 0; i < t / kWave; ++i) before += __popcll(mask[i]);
            const uint64_t own = mask[t / kWave], bit = uint64_t{1} << (t & (kWave - 1));
            if ((own & bit) != 0 && before + __popcll(own & (bit - 1)) == nth) S.row = t;
        }
        __syncthreads();
        U.m = S.row;
        U.runs = runs;
    } else {
        U.runs = by_runs(D, args_of(D, 0));
    }
    const int64_t len = ((D.a.V + parts - 1) / parts + kRun - 1) / kRun * kRun;  // whole runs
    U.lo = part * len;
    U.hi = min(U.lo + len, D.a.V);
    U.some = U.lo < U.hi;
    return U;
}

// Bins of a part of a row.  Rows by runs: one workgroup counts their runs, and
// says which bins to collect.
template <bool CAP>
__global__ __launch_bounds__(kBinThreads)
void draw_bins_kernel(DrawView D) {
    __shared__ uint64_t mass[kBins];
    __shared__ uint32_t count[kBins];
    __shared__ float sparse[kBinThreads / kWave * kSparse];
    __shared__ Ask ask;
    __shared__ Shares shares;
    const int t = threadIdx.x;
    const Unit U = unit_of(shares, D, 1);
    if (!U.some) return;
    const int64_t m = U.m;
    Batch first;
    if (!U.runs) first = load_batch<kBinThreads>(D.a.logits + m * D.a.ldl, U.lo, U.hi, D.vec);
    Part p = part_of(D, m);
    const Args A = args_of(D, m);
    if (!(A.temperature > 0.0f) || (U.runs && U.lo > 0)) return;
    fill_exp_table();
    for (int i = t; i < kBins; i += kBinThreads) {
        count[i] = 0;
        mass[i] = 0;
    }
    p = join(p);
    Row<CAP> R = row_of<CAP>(D, m, A, p.best, p.sum, p.count);
    if (R.mode == kFirst) return;
    __syncthreads();
    int turn = 0;
    if (R.mode == kByRuns) {
        count_runs<kBinThreads>(R, D.run + m * D.runs, D.runs, count);
        __syncthreads();
        Bins<kBinThreads> B = load_bins<kBinThreads>(count, mass);
        sum_bins(ask, turn, B);
        uint32_t reach;
        const Head H = choose_bins(ask, R, B, {0, 0}, &reach);
        if (t == 0) {
            D.head[m].k_bin = H.k_bin;
            D.head[m].p_hi = H.p_hi;
            D.head[m].u_hi = H.u_hi;
            D.head[m].first_k = H.first_k;
        }
        return;
    }
    R.level_of_top();
    const Sum mine = fill_bins<kBinThreads>(first, D, R, U.lo, U.hi, count, mass, sparse);
    __syncthreads();
    if (R.has_min && R.mode == kSummed) {
        Sum above;
        block_before<kBinThreads>(ask.scan, turn, mine, &above);
        if (t == 0 && above.count) {
            atomicAdd(&D.head[m].above_count, above.count);
            atomicAdd(reinterpret_cast<unsigned long long*>(&D.head[m].above_mass),
                      static_cast<unsigned long long>(above.mass));
        }
    }
    for (int i = t; i < kBins; i += kBinThreads) {
        if (count[i] == 0) continue;
        atomicAdd(&D.count[m * kBins + i], count[i]);
        if (mass[i])
            atomicAdd(reinterpret_cast<unsigned long long*>(&D.mass[m * kBins + i]),
                      static_cast<unsigned long long>(mass[i]));
    }
}

template <bool CAP>
__global__ __launch_bounds__(kBinThreads)
void draw_collect_kernel(DrawView D) {
    __shared__ uint64_t keys[kMostCands];
    __shared__ Ask ask;
    __shared__ uint32_t n, base, listed;
    __shared__ int32_t list[4 * kBinThreads];
    __shared__ Shares shares;
    const int t = threadIdx.x;
    const Unit U = unit_of(shares, D, D.run_parts);
    if (!U.some) return;
    const int64_t m = U.m, lo = U.lo, hi = U.hi;
    Bins<kBinThreads> B = {};
    Batch first;
    if (!U.runs) {
        B = load_bins<kBinThreads>(D.count + m * kBins, D.mass + m * kBins);
        first = load_batch<kBinThreads>(D.a.logits + m * D.a.ldl, lo, hi, D.vec);
    }
    Head* head = D.head + m;
    Head H = *head;
    Part p = part_of(D, m);
    const Args A = args_of(D, m);
    if (!(A.temperature > 0.0f)) return;
    if (t == 0) n = listed = 0;
    if (CAP && A.top_k > 0 && A.top_k <= kMostCounted) fill_exp_table();  // least_weighing() asks for the level
    p = join(p);
    Row<CAP> R = row_of<CAP>(D, m, A, p.best, p.sum, p.count);
    if (R.mode == kFirst) return;
    const float* run = D.run + m * D.runs;
    if (R.mode == kByRuns) {
        __syncthreads();
        R.level_of_top();
        collect_runs<kBinThreads>(D, R, H, run, lo, hi, list, &listed, keys, &n);
    } else {
        int turn = 0;
        sum_bins(ask, turn, B);  // a barrier
        if (R.mode == kCounted) R.level_of_top();
        uint32_t reach;
        H = choose_bins(ask, R, B, {H.above_mass, H.above_count}, &reach);
        if (lo == 0 && t == 0) {
            head->k_bin = H.k_bin;
            head->p_lo = H.p_lo;
            head->p_hi = H.p_hi;
            head->u_lo = H.u_lo;
            head->u_hi = H.u_hi;
            head->first_k = H.first_k;
        }
        if (few_runs(D, reach, hi - lo))
            collect_runs<kBinThreads>(D, R, H, run, lo, hi, list, &listed, keys, &n);
        else
            collect<kBinThreads>(first, D, R, H, lo, hi, keys, &n);
    }
    __syncthreads();
    const uint32_t found = n;
    if (found == 0) return;
    if (t == 0) base = atomicAdd(&head->collected, found);
    __syncthreads();
    for (uint32_t i = t; i < found && i < kMostCands; i += kBinThreads)
        if (base + i < kMostCands) D.cand[m * kMostCands + base + i] = keys[i];
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_token_kernel(DrawView D) {
    __shared__ RowLds S;
    __shared__ Ask ask;
    __shared__ uint32_t collected, listed;
    const int64_t m = blockIdx.x;
    Part p = part_of(D, m);
    const Args A = args_of(D, m);
    Head H = D.head[m];
    uint64_t key[kCandsPer];
    const uint64_t* cand = D.cand + m * kMostCands;
    key[0] = cand[threadIdx.x];
    fill_exp_table();
    Bins<kThreads> B = {};
    if (A.temperature > 0.0f && !by_runs(D, A)) B = load_bins<kThreads>(D.count + m * kBins, D.mass + m * kBins);
#pragma unroll
    for (int j = 1; j < kCandsPer; ++j) {
        key[j] = 0;
        if (j * kThreads < H.collected) key[j] = cand[j * kThreads + threadIdx.x];
    }
    p = join(p);
    Row<CAP> R = row_of<CAP>(D, m, A, p.best, p.sum, p.count);
    int32_t token = R.best ? index_of(R.best) : -1, n = R.best ? 1 : 0;
    if (R.mode != kFirst) {
        __syncthreads();
        R.level_of_top();
        int turn = 0;
        uint32_t found = H.collected;
        if (found > kMostCands && R.mode == kByRuns) {
            // About as many runs as top_k weigh anything, or fewer: their border is
            // far down.  (One range of 57,600 allowed, top-k 1000: 78 us, 445 by
            // digits; 32 such rows 108 and 588.)
            R.mode = kCounted;
            found = by_bins(S, ask, collected, listed, turn, D, R, D.run + m * D.runs, B, H);
#pragma unroll
            for (int j = 0; j < kCandsPer; ++j) key[j] = S.sorter.key[j * kThreads + threadIdx.x];
            __syncthreads();
        }
        if (found > kMostCands) {
            by_digits(S.digits, D, R, &token, &n);
        } else {
            if (R.mode == kSummed) sum_bins(S.sorter.ask, turn, B);
            draw_from_cands(S.sorter, turn, R, B, H, found, key, &token, &n);
        }
    }
    store(D, m, token, n);
}

template <bool CAP>
hipError_t launch(const DrawView& D, hipStream_t stream) {
    const dim3 rows(static_cast<unsigned>(D.a.M)), block(kThreads);
    if (D.parts == 1) {
        hipLaunchKernelGGL(draw_row_kernel<CAP>, rows, block, 0, stream, D);
        return hipGetLastError();
    }
    const dim3 grid(static_cast<unsigned>(D.parts), static_cast<unsigned>(D.a.M));
    if (D.part_len >= kStep<kThreads>)
        hipLaunchKernelGGL(draw_first_kernel<true>, grid, block, 0, stream, D);
    else
        hipLaunchKernelGGL(draw_first_kernel<false>, grid, block, 0, stream, D);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 shares(static_cast<unsigned>(D.parts * D.a.M));
    const dim3 bin_block(kBinThreads);
    hipLaunchKernelGGL(draw_bins_kernel<CAP>, shares, bin_block, 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draw_collect_kernel<CAP>, shares, bin_block, 0, stream, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(draw_token_kernel<CAP>, rows, block, 0, stream, D);
    return hipGetLastError();
}

// Workgroups of a row: one, in one launch, for short rows, and for longer ones
// where there are many; else about 512 in all (two a CU), of 4096 logits each at
// least, in four launches.  Top-k 50 / top-p 0.9, one launch against four, us:
//   1 x 16384    15 / 23   22 / 27        128 x 65536  23 / 64   33 / 66
//   4 x 20000    17 / 30   25 / 31        256 x 65536  29 / 74   43 / 100
//   1 x 32000    17 / 35   23 / 29        300 x 65536  53 / 136  57 / 132
//   16 x 40000   19 / 44   26 / 35        256 x 131072 45 / 138  59 / 165
//   64 x 32000   19 / 38   31 / 52        300 x 262144 131 / 479 124 / 385
//   256 x 32000  23 / 45   35 / 66        512 x 262144 150 / 494 163 / 530
// Longer rows stay with four although some of these lose by it: they share the
// work out where rows differ, and one launch takes what its slowest row does.  A
// sixteenth of the rows with top-p 0.9 among ones with top-k 50 / filters drawn
// from a server's mix, one launch against four, us:
//   64 x 131072  112 / 114  43 / 47       128 x 262144 223 / 218  71 / 84
//   128 x 131072 118 / 118  54 / 62       256 x 262144 252 / 249 118 / 149
//   256 x 131072 124 / 124  71 / 98       512 x 262144 467 / 375 211 / 252
constexpr int64_t kPartLeast = 4096;
int64_t most_split(int64_t V) {  // rows of a call that are split
    return V <= 20480 ? 0 : (V <= 40960 ? 15 : (V <= 65536 ? 127 : kMostSplit));
}

int parts_of(int64_t V, int64_t M) {
    if (M > most_split(V)) return 1;
    const int64_t most = (V + kPartLeast - 1) / kPartLeast, want = M > kWorkgroups / 2 ? 2 : kWorkgroups / M;
    const int64_t parts = want < most ? want : most;
    return static_cast<int>(parts > kMaxParts ? kMaxParts : parts);
}

int64_t runs_of(int64_t V) { return (V + kRun - 1) / kRun; }

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

// What the largest batch of up to M rows needs that is split: a program that
// allocates once for its largest batch has enough for a smaller one, and for a
// longer vocabulary more.  (A row more is 80 KB for its bins and candidates, which
// what all parts of all rows say, 16 KB at most, does not outweigh.)
size_t draw_ws_bytes(int64_t V, int64_t M) {
    if (M > most_split(V)) M = most_split(V);
    if (M == 0) return 256;
    const size_t m = static_cast<size_t>(M);
    return align256(m * static_cast<size_t>(parts_of(V, M)) * sizeof(Part)) + align256(m * sizeof(Head)) +
           m * (kBins * (sizeof(uint32_t) + sizeof(uint64_t)) + kMostCands * sizeof(uint64_t)) +
           align256(m * static_cast<size_t>(runs_of(V)) * sizeof(float));
}

hipError_t launch_logits_draw(const DrawArgs& a, void* ws, hipStream_t stream) {
    DrawView D;
    D.a = a;
    D.twice = a.softcap > 0.0f ? 2.0 * kLog2e / static_cast<double>(a.softcap) : 0.0;
    int bits = 0;  // the smallest with V <= 2^bits
    while ((int64_t{1} << bits) < a.V) ++bits;
    D.q = 62 - bits < 51 ? 62 - bits : 51;
    D.parts = parts_of(a.V, a.M);
    const int64_t most = (a.V + kPartLeast - 1) / kPartLeast;
    D.most_parts = static_cast<int>(most < kMaxParts ? most : kMaxParts);
    // half the workgroups, were all rows by runs
    D.run_parts = D.parts / 2 < 16 ? (D.parts > 1 ? D.parts / 2 : 1) : 16;
    // whole runs, which are whole quads
    D.part_len = ((a.V + D.parts - 1) / D.parts + kRun - 1) / kRun * kRun;
    D.vec = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.ldl % 4 == 0;
    D.runs = D.parts > 1 || runs_of(a.V) <= kMostRuns ? runs_of(a.V) : 0;
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
    p += m * kBins * sizeof(uint32_t);
    D.run = reinterpret_cast<float*>(p);
    return a.softcap > 0.0f ? launch<true>(D, stream) : launch<false>(D, stream);
}

}  // namespace qmv
