// Rows of a quantized embedding table: y[m] = scale * W[tokens[m]].
//
// One thread forms four neighbouring elements: a few bytes of codes in, 16
// bytes out.  The output is 4 bytes an element against 0.56-1.06 of codes, so
// stores bound it: 8192 rows of 5376 from Q4_K (201 MB) take 34 us, 5.9 TB/s, from
// Q8_0, Q4_0 and Q6_K (223, 201, 212 MB) 34, 32 and 32; one row is a launch (2.3 us
// of kernel in a call of 5).  They go past the L2 and are whole cache lines a wave
// (a y that is not 16-byte aligned: 43-44 us); the codes' narrow loads (a Q8_0 or
// Q4_0 block is 2-byte aligned) stay in the L1.
//
// A weight's products are exact in float32: a float16 scale has 11 bits, codes
// and sub-scales add at most 13.  Only Q4_K's difference is rounded.
#include <stdint.h>

#include "qmv_device.h"
#include "serve_internal.h"
#include "step_device.h"

namespace qmv {
namespace {

__device__ __forceinline__ uint32_t u16_at(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// Four bytes at a 2-byte aligned address.
__device__ __forceinline__ uint32_t u32_at(const uint8_t* p) { return u16_at(p) | (u16_at(p + 2) << 16); }

// Elements 4 q .. 4 q + 3 of a row.
template <int F>
__device__ __forceinline__ float4 quad_of(const uint8_t* row, int64_t q) {
    if constexpr (F == kQ8_0) {
        const uint8_t* blk = row + (q >> 3) * 34;
        const float d = half_bits_to_float(u16_at(blk));
        const uint32_t c = u32_at(blk + 2 + 4 * (q & 7));
        return make_float4(sbyte<0>(c) * d, sbyte<1>(c) * d, sbyte<2>(c) * d, sbyte<3>(c) * d);
    } else if constexpr (F == kQ4_0) {
        const uint8_t* blk = row + (q >> 3) * 18;
        const float d = half_bits_to_float(u16_at(blk));
        // byte j has element j in its low nibble, element j + 16 in its high one
        const uint32_t c = (u32_at(blk + 2 + 4 * (q & 3)) >> (q & 4)) & 0x0f0f0f0fu;
        return make_float4((ubyte<0>(c) - 8.0f) * d, (ubyte<1>(c) - 8.0f) * d, (ubyte<2>(c) - 8.0f) * d,
                           (ubyte<3>(c) - 8.0f) * d);
    } else if constexpr (F == kQ4_K) {
        const uint8_t* blk = row + (q >> 6) * 144;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(blk);  // 16-byte aligned
        const int e = static_cast<int>(q & 63), sub = e >> 3, at = sub & 3;
        const uint32_t dd = w[0], low = (w[1] >> (8 * at)) & 255u, mid = (w[2] >> (8 * at)) & 255u,
                       high = (w[3] >> (8 * at)) & 255u;
        const uint32_t sc = sub < 4 ? low & 63u : (high & 15u) | ((low >> 6) << 4);
        const uint32_t mn = sub < 4 ? mid & 63u : (high >> 4) | ((mid >> 6) << 4);
        const float d = half_bits_to_float(dd & 0xffffu) * static_cast<float>(sc);
        const float m = half_bits_to_float(dd >> 16) * static_cast<float>(mn);
        const uint32_t c = (w[4 + 8 * (sub >> 1) + (e & 7)] >> (4 * (sub & 1))) & 0x0f0f0f0fu;
        return make_float4(ubyte<0>(c) * d - m, ubyte<1>(c) * d - m, ubyte<2>(c) * d - m, ubyte<3>(c) * d - m);
    } else {
        const uint8_t* blk = row + (q >> 6) * 210;
        const int e = static_cast<int>(q & 63), h = e >> 5, g = (e >> 3) & 3, at = 4 * (e & 7);
        const float d = half_bits_to_float(u16_at(blk + 208)) *
                        static_cast<float>(static_cast<int8_t>(blk[192 + (e >> 2)]));
        const uint32_t lo = (u32_at(blk + 64 * h + 32 * (g & 1) + at) >> (4 * (g >> 1))) & 0x0f0f0f0fu;
        const uint32_t hi = (u32_at(blk + 128 + 32 * h + at) >> (2 * g)) & 0x03030303u;
        const uint32_t c = lo | (hi << 4);
        return make_float4((ubyte<0>(c) - 32.0f) * d, (ubyte<1>(c) - 32.0f) * d, (ubyte<2>(c) - 32.0f) * d,
                           (ubyte<3>(c) - 32.0f) * d);
    }
}

template <int F>
__global__ __launch_bounds__(kBlockThreads)
void embed_kernel(const uint8_t* __restrict__ W, const int32_t* __restrict__ tokens, float* __restrict__ y, int64_t N,
                  int64_t K, int64_t row_bytes, float scale, bool vec) {
    const int64_t m = blockIdx.x, quads = K / 4;
    const int64_t token = tokens[m];
    const bool real = token >= 0 && token < N;
    const uint8_t* row = W + (real ? token : 0) * row_bytes;
    for (int64_t q = static_cast<int64_t>(blockIdx.y) * kBlockThreads + threadIdx.x; q < quads;
         q += static_cast<int64_t>(gridDim.y) * kBlockThreads) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (real) {
            v = quad_of<F>(row, q);
            v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
        }
        stream4(y + m * K + 4 * q, v, vec);
    }
}

}  // namespace

hipError_t launch_embed(int fmt, const void* W, const int32_t* tokens, float* y, int64_t N, int64_t K, int64_t M,
                        float scale, hipStream_t stream) {
    const uint8_t* w = static_cast<const uint8_t*>(W);
    const bool vec = (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    const int64_t parts = (K / 4 + kBlockThreads - 1) / kBlockThreads;
    const dim3 grid(static_cast<unsigned>(M), static_cast<unsigned>(parts < 64 ? parts : 64)), block(kBlockThreads);
    switch (fmt) {
    case kQ4_0:
        hipLaunchKernelGGL(embed_kernel<kQ4_0>, grid, block, 0, stream, w, tokens, y, N, K, K / 32 * 18, scale, vec);
        break;
    case kQ8_0:
        hipLaunchKernelGGL(embed_kernel<kQ8_0>, grid, block, 0, stream, w, tokens, y, N, K, K / 32 * 34, scale, vec);
        break;
    case kQ4_K:
        hipLaunchKernelGGL(embed_kernel<kQ4_K>, grid, block, 0, stream, w, tokens, y, N, K, K / 256 * 144, scale, vec);
        break;
    default:
        hipLaunchKernelGGL(embed_kernel<kQ6_K>, grid, block, 0, stream, w, tokens, y, N, K, K / 256 * 210, scale, vec);
        break;
    }
    return hipGetLastError();
}

}  // namespace qmv
