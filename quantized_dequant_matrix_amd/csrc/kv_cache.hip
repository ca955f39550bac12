// The paged key/value cache: quantizing new rows into it and reading rows
// back as float32.
//
// A row (one token's head) of D elements is stored as D int8 codes and one
// float32 scale d = max|x| / 127, or as D float16.  Both kernels move every
// byte once and compute a few operations an element, so memory bounds them:
// 4 bytes in and 1 (2) out an element for the write, the reverse for the
// read.
//
// Work split: blockIdx.x is a row of the batch, blockIdx.y keys or values.
// D / 4 lanes hold a head's row, four elements each, so that the row's
// maximum is a few lane exchanges and a wave writes whole rows of codes.
#include <stdint.h>

#include "kv_device.h"
#include "step_internal.h"

namespace qmv {
namespace {

__device__ __forceinline__ float4 load4(const float* p, bool vec) {
    if (vec) return *reinterpret_cast<const float4*>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
}

__device__ __forceinline__ void store4(float* p, float4 v, bool vec) {
    if (vec) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    }
}

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t code_q8(float v, float d) {
    const float r = fminf(fmaxf(roundf(v / d), -127.0f), 127.0f);
    return static_cast<uint32_t>(static_cast<int>(r)) & 0xffu;
}

struct KvPlanes {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
};

// F16: the row's maximum decides only whether every element is finite.
template <int D, bool F16>
__global__ __launch_bounds__(kBlockThreads)
void kv_write_kernel(KvView view, KvPlanes c, const float* __restrict__ k, int64_t ldk, const float* __restrict__ v,
                     int64_t ldv, bool vec) {
    constexpr int L = D / 4;                    // lanes of a head's row
    constexpr int kHeads = kBlockThreads / L;   // heads of one pass
    const int row = blockIdx.x;
    const bool values = blockIdx.y != 0;
    const float* src = values ? v + row * ldv : k + row * ldk;
    bool belongs;
    const int64_t slot = row_slot(view, row, &belongs);
    if (slot < 0) return;
    const int64_t page = slot >> view.page_shift, at = slot & ((1 << view.page_shift) - 1);
    const int sub = threadIdx.x % L;
    for (int h = threadIdx.x / L; h < view.heads; h += kHeads) {
        const float4 x = load4(src + static_cast<int64_t>(h) * D + 4 * sub, vec);
        const int64_t cell = ((page * view.heads + h) << view.page_shift) + at;
        if constexpr (F16) {
            _Float16 f[4] = {static_cast<_Float16>(x.x), static_cast<_Float16>(x.y), static_cast<_Float16>(x.z),
                             static_cast<_Float16>(x.w)};
            uint32_t a = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) a = max(a, mag_bits(static_cast<float>(f[e])));
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), o, L)));
            uint2 packed;
            packed.x = __builtin_bit_cast(uint16_t, f[0]) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, f[1])) << 16);
            packed.y = __builtin_bit_cast(uint16_t, f[2]) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, f[3])) << 16);
            if (a >= 0x7f800000u) packed = make_uint2(0x7e007e00u, 0x7e007e00u);
            reinterpret_cast<uint2*>(values ? c.v : c.k)[cell * L + sub] = packed;
        } else {
            uint32_t a = max(max(mag_bits(x.x), mag_bits(x.y)), max(mag_bits(x.z), mag_bits(x.w)));
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), o, L)));
            const float d = a < 0x7f800000u ? __uint_as_float(a) / 127.0f : __uint_as_float(0x7fc00000u);
            uint32_t packed = 0;
            if (a != 0u && a < 0x7f800000u)
                packed = code_q8(x.x, d) | (code_q8(x.y, d) << 8) | (code_q8(x.z, d) << 16) | (code_q8(x.w, d) << 24);
            reinterpret_cast<uint32_t*>(values ? c.v : c.k)[cell * L + sub] = packed;
            if (sub == 0) (values ? c.v_scale : c.k_scale)[cell] = d;
        }
    }
}

template <int D, bool F16>
__global__ __launch_bounds__(kBlockThreads)
void kv_read_kernel(KvView view, KvPlanes c, float* __restrict__ k, int64_t ldk, float* __restrict__ v, int64_t ldv,
                    bool vec) {
    constexpr int L = D / 4;
    constexpr int kHeads = kBlockThreads / L;
    const int row = blockIdx.x;
    const bool values = blockIdx.y != 0;
    float* dst = values ? v + row * ldv : k + row * ldk;
    bool belongs;
    const int64_t slot = row_slot(view, row, &belongs);
    if (!belongs) return;
    const int64_t page = slot >> view.page_shift, at = slot & ((1 << view.page_shift) - 1);
    const int sub = threadIdx.x % L;
    for (int h = threadIdx.x / L; h < view.heads; h += kHeads) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (slot >= 0) {
            const int64_t cell = ((page * view.heads + h) << view.page_shift) + at;
            if constexpr (F16) {
                const uint2 p = reinterpret_cast<const uint2*>(values ? c.v : c.k)[cell * L + sub];
                x = make_float4(half_bits_to_float(p.x & 0xffffu), half_bits_to_float(p.x >> 16),
                                half_bits_to_float(p.y & 0xffffu), half_bits_to_float(p.y >> 16));
            } else {
                const uint32_t p = reinterpret_cast<const uint32_t*>(values ? c.v : c.k)[cell * L + sub];
                const float d = (values ? c.v_scale : c.k_scale)[cell];
                x = make_float4(sbyte<0>(p) * d, sbyte<1>(p) * d, sbyte<2>(p) * d, sbyte<3>(p) * d);
            }
        }
        store4(dst + static_cast<int64_t>(h) * D + 4 * sub, x, vec);
    }
}

// float4 accesses need 16-byte aligned rows
bool vec_rows(const void* k, int64_t ldk, const void* v, int64_t ldv) {
    return ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 && ldk % 4 == 0 && ldv % 4 == 0;
}

}  // namespace

#define KV_LAUNCH(kernel, D, ...)                                                                                      \
    do {                                                                                                               \
        if (c.format == QMV_KV_F16)                                                                                    \
            hipLaunchKernelGGL((kernel<D, true>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__);                  \
        else                                                                                                           \
            hipLaunchKernelGGL((kernel<D, false>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__);                 \
    } while (0)

hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* k, int64_t ldk, const float* v,
                           int64_t ldv, hipStream_t stream) {
    const KvView view = view_of(c, b);
    const KvPlanes p{c.k, c.v, c.k_scale, c.v_scale};
    const bool vec = vec_rows(k, ldk, v, ldv);
    const dim3 grid(static_cast<unsigned>(b.T), 2);
    if (c.head_dim == 64) KV_LAUNCH(kv_write_kernel, 64, view, p, k, ldk, v, ldv, vec);
    else if (c.head_dim == 128) KV_LAUNCH(kv_write_kernel, 128, view, p, k, ldk, v, ldv, vec);
    else KV_LAUNCH(kv_write_kernel, 256, view, p, k, ldk, v, ldv, vec);
    return hipGetLastError();
}

hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_batch& b, float* k, int64_t ldk, float* v, int64_t ldv,
                          hipStream_t stream) {
    const KvView view = view_of(c, b);
    const KvPlanes p{c.k, c.v, c.k_scale, c.v_scale};
    const bool vec = vec_rows(k, ldk, v, ldv);
    const dim3 grid(static_cast<unsigned>(b.T), 2);
    if (c.head_dim == 64) KV_LAUNCH(kv_read_kernel, 64, view, p, k, ldk, v, ldv, vec);
    else if (c.head_dim == 128) KV_LAUNCH(kv_read_kernel, 128, view, p, k, ldk, v, ldv, vec);
    else KV_LAUNCH(kv_read_kernel, 256, view, p, k, ldk, v, ldv, vec);
    return hipGetLastError();
}

}  // namespace qmv
