// A token of each row of logits, by temperature, top-k, top-p and min-p.
//
// The filters keep a prefix of the row in the order "larger logit first,
// equal ones by index", and the draw takes an element of it by a running sum
// in the same order.  So everything asks one kind of question: which element
// of the order is the first whose running count, or running sum of weights,
// reaches a number?  It is answered without sorting, digit by digit of a
// 64-bit key (order code of the logit, then the index from below): count and
// sum of weights by the next digit, in bins, over the elements that share the
// digits found so far.
//
// Weights are whole multiples of 2^-q of the row's largest: their sums are
// exact, in any order, in 64-bit integers, so bins can be summed by atomics.
#include <stdint.h>

#include "qmv_device.h"
#include "serve_internal.h"
#include "step_device.h"
#include "weights_device.h"

namespace qmv {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int kBins = 2048;
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

struct DrawView {
    DrawArgs a;
    double twice;  // 2 log2(e) / softcap
    int q;
};

template <bool CAP>
struct RowWeights {
    Weights w;
    double top, unit;
    __device__ __forceinline__ double exponent(float y) const {
        return w.template below<CAP>(w.template level<CAP>(fminf(y, kMaxLogit)), top);
    }
    // weight * 2^q, rounded to nearest by an addition of 2^52
    __device__ __forceinline__ uint64_t mass(float y) const {
        const double r = fma(exp2_f64(exponent(y)), unit, 4503599627370496.0);
        return __builtin_bit_cast(uint64_t, r) & 0xFFFFFFFFFFFFFull;
    }
};

struct Shared {
    uint64_t mass[kBins];
    uint32_t count[kBins];
    uint64_t part_mass[kWaves], best[kWaves];
    uint32_t part_count[kWaves];
    uint64_t before_mass, bin_mass, key;
    uint32_t before_count, bin_count, bin;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int d) {
    const uint32_t lo = __shfl_up(static_cast<uint32_t>(v), d, kWave), hi = __shfl_up(static_cast<uint32_t>(v >> 32), d, kWave);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Sums before this thread in thread order, and the total.
__device__ __forceinline__ Sum block_before(Shared& S, Sum mine, Sum* total) {
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
        S.part_mass[wave] = upto.mass;
        S.part_count[wave] = upto.count;
    }
    __syncthreads();
    Sum before = {upto.mass - mine.mass, upto.count - mine.count};
    *total = {0, 0};
    for (int i = 0; i < kWaves; ++i) {
        if (i < wave) {
            before.mass += S.part_mass[i];
            before.count += S.part_count[i];
        }
        total->mass += S.part_mass[i];
        total->count += S.part_count[i];
    }
    return before;
}

struct Found {
    uint64_t key;
    Sum upto;  // sums up to and with the element
};

// The first element of the order whose running count (MASS: running sum)
// reaches `need`, 1 <= need <= the row's.
template <bool CAP, bool MASS>
__device__ Found find(Shared& S, const float* y, int64_t V, const RowWeights<CAP>& R, uint64_t need) {
    uint64_t prefix = 0;
    Sum before = {0, 0};
    const int t = threadIdx.x;
    constexpr int kLow[6] = {53, 42, 32, 21, 10, 0};
    for (int d = 0; d < 6; ++d) {
        const int low = kLow[d], high = d == 0 ? 64 : kLow[d - 1];
        const uint32_t digits = (1u << (high - low)) - 1u;
        __syncthreads();
        for (int i = t; i < kBins; i += kThreads) {
            S.mass[i] = 0;
            S.count[i] = 0;
        }
        __syncthreads();
        for (int64_t i = t; i < V; i += kThreads) {
            const float v = y[i];
            if (!weighs(v)) continue;
            const uint64_t key = key_of(v, i);
            if (d > 0 && (key >> high) != (prefix >> high)) continue;
            const uint32_t bin = digits - (static_cast<uint32_t>(key >> low) & digits);  // bin 0: first in the order
            atomicAdd(&S.count[bin], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&S.mass[bin]), static_cast<unsigned long long>(R.mass(v)));
        }
        __syncthreads();
        const Sum a = {S.mass[2 * t], S.count[2 * t]}, b = {S.mass[2 * t + 1], S.count[2 * t + 1]};
        Sum total;
        Sum run = block_before(S, {a.mass + b.mass, a.count + b.count}, &total);
        run.mass += before.mass;
        run.count += before.count;
        const Sum bins[2] = {a, b};
        for (int j = 0; j < 2; ++j) {
            const Sum next = {run.mass + bins[j].mass, run.count + bins[j].count};
            if (MASS ? (run.mass < need && next.mass >= need) : (run.count < need && next.count >= need)) {
                S.bin = 2 * t + j;
                S.before_mass = run.mass;
                S.before_count = run.count;
                S.bin_mass = next.mass;
                S.bin_count = next.count;
            }
            run = next;
        }
        __syncthreads();
        before = {S.before_mass, S.before_count};
        prefix |= static_cast<uint64_t>(digits - S.bin) << low;
    }
    return {prefix, {S.bin_mass, S.bin_count}};
}

template <bool CAP>
__global__ __launch_bounds__(kThreads)
void draw_row_kernel(DrawView D) {
    __shared__ Shared S;
    const int64_t m = blockIdx.x, V = D.a.V;
    const int t = threadIdx.x, wave = t / kWave, lane = t & (kWave - 1);
    const float* y = D.a.logits + m * D.a.ldl;
    fill_exp_table();
    // the first of the order
    uint64_t best = 0;
    for (int64_t i = t; i < V; i += kThreads) {
        const float v = y[i];
        const uint64_t key = weighs(v) ? key_of(v, i) : 0;
        best = key > best ? key : best;
    }
    for (int d = 1; d < kWave; d <<= 1) {
        const uint64_t o = shfl_up64(best, d);
        if (lane >= d) best = o > best ? o : best;
    }
    if (lane == kWave - 1) S.best[wave] = best;
    __syncthreads();
    best = 0;
    for (int i = 0; i < kWaves; ++i) best = S.best[i] > best ? S.best[i] : best;
    int32_t token = best ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1, n = best ? 1 : 0;
    const float T = D.a.temperature[m];
    if (best && T > 0.0f) {
        RowWeights<CAP> R;
        R.w.k = kLog2e / static_cast<double>(T);
        R.w.cap = static_cast<double>(D.a.softcap) * R.w.k;
        R.w.twice = D.twice;
        R.unit = static_cast<double>(uint64_t{1} << D.q);
        R.top = R.w.template level<CAP>(logit_of(static_cast<uint32_t>(best >> 32)));
        const float min_p = D.a.min_p ? D.a.min_p[m] : 0.0f;
        const double floor_e = min_p > 0.0f ? log2(static_cast<double>(min_p)) : 0.0;
        Sum all = {0, 0}, above = {0, 0};
        for (int64_t i = t; i < V; i += kThreads) {
            const float v = y[i];
            if (!weighs(v)) continue;
            const uint64_t w = R.mass(v);
            all.mass += w;
            all.count += 1;
            if (min_p > 0.0f && R.exponent(v) >= floor_e) {
                above.mass += w;
                above.count += 1;
            }
        }
        Sum total, kept;
        block_before(S, above, &kept);
        block_before(S, all, &total);
        const Sum first = {uint64_t{1} << D.q, 1};
        if (!(min_p > 0.0f)) kept = total;
        if (kept.count == 0) kept = first;
        Sum of_k = total;
        const int32_t k = D.a.top_k ? D.a.top_k[m] : 0;
        if (k > 0 && static_cast<uint32_t>(k) < total.count)
            of_k = find<CAP, false>(S, y, V, R, static_cast<uint64_t>(k)).upto;
        if (of_k.count < kept.count) kept = of_k;
        const float p = D.a.top_p ? D.a.top_p[m] : 1.0f;
        if (p < 1.0f) {
            const double border = ceil(fmax(static_cast<double>(p), 0.0) * static_cast<double>(of_k.mass));
            uint64_t need = static_cast<uint64_t>(border);
            need = need < 1 ? 1 : (need > of_k.mass ? of_k.mass : need);
            const Sum of_p = find<CAP, true>(S, y, V, R, need).upto;
            if (of_p.count < kept.count) kept = of_p;
        }
        n = static_cast<int32_t>(kept.count);
        const double u = fmin(fmax(static_cast<double>(D.a.u[m]), 0.0), 1.0);  // NaN: 0
        uint64_t need = static_cast<uint64_t>(u * static_cast<double>(kept.mass)) + 1;
        need = need > kept.mass ? kept.mass : need;
        token = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(find<CAP, true>(S, y, V, R, need).key));
    }
    if (t == 0) {
        D.a.token[m] = token;
        if (D.a.kept) D.a.kept[m] = n;
    }
}

}  // namespace

size_t draw_ws_bytes(int64_t, int64_t) { return 256; }

hipError_t launch_logits_draw(const DrawArgs& a, void*, hipStream_t stream) {
    DrawView D;
    D.a = a;
    D.twice = a.softcap > 0.0f ? 2.0 * kLog2e / static_cast<double>(a.softcap) : 0.0;
    int bits = 0;  // the smallest with V <= 2^bits
    while ((int64_t{1} << bits) < a.V) ++bits;
    D.q = 62 - bits < 51 ? 62 - bits : 51;
    const dim3 grid(static_cast<unsigned>(a.M)), block(kThreads);
    if (a.softcap > 0.0f)
        hipLaunchKernelGGL(draw_row_kernel<true>, grid, block, 0, stream, D);
    else
        hipLaunchKernelGGL(draw_row_kernel<false>, grid, block, 0, stream, D);
    return hipGetLastError();
}

}  // namespace qmv
