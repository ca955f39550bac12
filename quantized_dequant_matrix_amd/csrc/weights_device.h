// Weights of logits in 64 bits, shared by the kernels that draw tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_device.h"

namespace qmv {

constexpr double kLog2e = 1.4426950408889634074;
constexpr float kNegInf = -__builtin_inff();

// 2^(j / 256), j < 256, in LDS: filled by the first 256 threads of a
// workgroup before its first barrier.
static __shared__ double exp_table[256];

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

}  // namespace qmv
