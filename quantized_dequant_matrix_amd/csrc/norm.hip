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
#include "step_device.h"
#include "step_internal.h"

namespace qmv {
namespace {

// Sum over the workgroup, every thread with the same bits.
template <int WAVES_MAX>
__device__ __forceinline__ double block_sum(double v, double* part, int waves) {
    v = wave_add(v);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < WAVES_MAX; ++i)
        if (i < waves) v += part[i];
    return v;
}

__device__ __forceinline__ float rstd_of(double sum, int64_t K, float eps) {
    return static_cast<float>(1.0 / sqrt(sum / static_cast<double>(K) + static_cast<double>(eps)));
}

// One workgroup a row of K = 4 Q elements, the whole row in registers: thread
// t holds the float4 t, t + threads, ... .  Memory bounds it: 8 bytes in and 8
// (5.1 with codes) out an element, each once.  2048 rows of 5376 take 27-32
// us, 5.5-6.5 TB/s (52 us with a second read 4 bytes at a time and plain stores).
template <int VPT, bool Q8>
__global__ __launch_bounds__(1024)
void rmsnorm_row_kernel(const float* x, const float* r, const float* __restrict__ w, float* z, float* __restrict__ y,
                        int8_t* __restrict__ q, float* __restrict__ d, int Q, float eps, bool vec) {
    __shared__ double part[16];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * Q;  // in float4
    const int t = threadIdx.x, threads = blockDim.x;
    float4 v[VPT], f[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = t + j * threads;
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < Q) v[j] = load4(x + 4 * (row + i), vec);
    }
    if (r) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = t + j * threads;
            f[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < Q) f[j] = load4(r + 4 * (row + i), vec);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            v[j] = make_float4(v[j].x + f[j].x, v[j].y + f[j].y, v[j].z + f[j].z, v[j].w + f[j].w);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = t + j * threads;
        if (i < Q) f[j] = load4(w + 4 * static_cast<int64_t>(i), vec);
    }
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = t + j * threads;
        if (z && i < Q) stream4(z + 4 * (row + i), v[j], vec);
        const double e[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) sum = fma(e[c], e[c], sum);
    }
    sum = block_sum<16>(sum, part, threads / kWave);
    const float rstd = rstd_of(sum, 4 * static_cast<int64_t>(Q), eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = t + j * threads;
        const bool in = i < Q;
        const float4 o = make_float4((v[j].x * rstd) * f[j].x, (v[j].y * rstd) * f[j].y, (v[j].z * rstd) * f[j].z,
                                     (v[j].w * rstd) * f[j].w);
        if constexpr (Q8) {
            // 8 lanes hold a block: Q is a multiple of 8 and so is threads
            uint32_t a = in ? mag_bits4(o) : 0u;
#pragma unroll
            for (int s = 4; s > 0; s >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), s, 8)));
            if (in) {
                const float db = scale_q8(a);
                __builtin_nontemporal_store(codes_q8(o, a, db), reinterpret_cast<uint32_t*>(q) + row + i);
                if ((i & 7) == 0) d[(row + i) >> 3] = db;
            }
        } else {
            if (in) stream4(y + 4 * (row + i), o, vec);
        }
    }
}

// Rows that no workgroup's registers hold, or of a length that is not a
// multiple of four: the row is read again after the sum.  An element is read,
// added and written by the same thread in both passes, so z may be x or r.
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
    sum = block_sum<THREADS / kWave>(sum, part, THREADS / kWave);
    const float rstd = rstd_of(sum, K, eps);
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
            const float db = scale_q8(a);
            if (i < K) {
                q[row * K + i] = static_cast<int8_t>(codes_q8(make_float4(v, 0.0f, 0.0f, 0.0f), a, db));
                if ((i & 31) == 0) d[(row * K + i) / 32] = db;
            }
        }
    }
}

}  // namespace

hipError_t launch_rmsnorm(const float* x, const float* r, const float* w, float* z, float* y, int8_t* q, float* d,
                          int64_t K, int64_t M, float eps, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(M));
    // Four float4 a thread where a workgroup holds the row that way: two or
    // eight differ by less than 10% from it, for one row as for thousands.
    const int64_t Q = K / 4, vpt = Q <= 4 * 1024 ? 4 : 8;
    if (K % 4 != 0 || Q > 8 * 1024) {
        if (q)
            hipLaunchKernelGGL((rmsnorm_kernel<1024, true>), grid, dim3(1024), 0, stream, x, r, w, z, y, q, d, K, eps);
        else
            hipLaunchKernelGGL((rmsnorm_kernel<1024, false>), grid, dim3(1024), 0, stream, x, r, w, z, y, q, d, K, eps);
        return hipGetLastError();
    }
    const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(r) | reinterpret_cast<uintptr_t>(w) |
                          reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(y);
    const bool vec = (all & 15) == 0;
    const int64_t threads = ((Q + vpt - 1) / vpt + kWave - 1) / kWave * kWave;
    const dim3 block(static_cast<unsigned>(threads));
#define ROW(V)                                                                                                     \
    do {                                                                                                           \
        if (q)                                                                                                     \
            hipLaunchKernelGGL((rmsnorm_row_kernel<V, true>), grid, block, 0, stream, x, r, w, z, y, q, d,         \
                               static_cast<int>(Q), eps, vec);                                                     \
        else                                                                                                       \
            hipLaunchKernelGGL((rmsnorm_row_kernel<V, false>), grid, block, 0, stream, x, r, w, z, y, q, d,        \
                               static_cast<int>(Q), eps, vec);                                                     \
    } while (0)
    if (vpt == 4) ROW(4);
    else ROW(8);
#undef ROW
    return hipGetLastError();
}

}  // namespace qmv
