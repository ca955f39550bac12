// Residual addition and root-mean-square norm, with a float32 output or Q8
// activation blocks.
//
//   z = x + r,  rstd = float32(1 / sqrt(mean(z^2) + eps)),  y = (z rstd) w
//
// The sum of squares is taken in 64 bits: a float32 sum would make the last
// bit of rstd, and with it the 8-bit code of an element next to a rounding
// border, depend on the order of the sum.  In 64 bits any order gives the
// same rstd, and everything after it is one float32 operation an element.
#include <stdint.h>

#include "qmv_device.h"
#include "qmv_internal.h"
#include "step_internal.h"

namespace qmv {
namespace {

// |v| of a block of 32 as an unsigned maximum of the bit patterns, which
// orders finite numbers, infinity and NaN: a block that is not finite ends
// with a maximum at or above infinity's pattern.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Code of one element.  Half away from zero, as the activation quantizer.
__device__ __forceinline__ uint32_t code_q8(float v, float d) {
    const float r = fminf(fmaxf(roundf(v / d), -127.0f), 127.0f);
    return static_cast<uint32_t>(static_cast<int>(r)) & 0xffu;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// One workgroup a row.  An element is read, added and written by the same
// thread in both passes, so z may be x or r.
template <int THREADS, bool Q8>
__global__ __launch_bounds__(THREADS)
void rmsnorm_kernel(const float* x, const float* r, const float* __restrict__ w, float* z, float* __restrict__ y,
                    int8_t* __restrict__ q, float* __restrict__ d, int64_t K, float eps) {
    __shared__ double part[THREADS / kWave];
    const int64_t row = blockIdx.x;
    x += row * K;
    if (r) r += row * K;
    if (z) z += row * K;
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < K; i += THREADS) {
        const float v = r ? x[i] + r[i] : x[i];
        sum = fma(static_cast<double>(v), static_cast<double>(v), sum);
    }
    sum = wave_sum_f64(sum);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) sum += part[i];
    const float rstd = static_cast<float>(1.0 / sqrt(sum / static_cast<double>(K) + static_cast<double>(eps)));
    // whole waves stay in the loop: the 32 lanes of a block exchange
    for (int64_t i0 = threadIdx.x & ~(kWave - 1); i0 < K; i0 += THREADS) {
        const int64_t i = i0 + (threadIdx.x & (kWave - 1));
        float v = 0.0f;
        if (i < K) {
            v = r ? x[i] + r[i] : x[i];
            if (z) z[i] = v;
            v = (v * rstd) * w[i];
            if constexpr (!Q8) y[row * K + i] = v;
        }
        if constexpr (Q8) {
            uint32_t a = mag_bits(v);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), o, 32)));
            const float db = a < 0x7f800000u ? __uint_as_float(a) / 127.0f : __uint_as_float(0x7fc00000u);
            if (i < K) {
                q[row * K + i] = a == 0u ? 0 : static_cast<int8_t>(code_q8(v, db));
                if ((i & 31) == 0) d[(row * K + i) / 32] = db;
            }
        }
    }
}

}  // namespace

hipError_t launch_rmsnorm(const float* x, const float* r, const float* w, float* z, float* y, int8_t* q, float* d,
                          int64_t K, int64_t M, float eps, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(M));
    if (q)
        hipLaunchKernelGGL((rmsnorm_kernel<1024, true>), grid, dim3(1024), 0, stream, x, r, w, z, y, q, d, K, eps);
    else
        hipLaunchKernelGGL((rmsnorm_kernel<1024, false>), grid, dim3(1024), 0, stream, x, r, w, z, y, q, d, K, eps);
    return hipGetLastError();
}

}  // namespace qmv
