// Device-side helpers shared by the decode-step kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_device.h"

namespace qmv {

// |v| as an unsigned pattern: its maximum over a row orders finite numbers,
// infinity and NaN, so a row that is not finite ends at or above infinity's.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a row or block whose largest pattern is `a`: max|x| / 127, NaN
// if it is not finite.
__device__ __forceinline__ float scale_q8(uint32_t a) {
    return a < 0x7f800000u ? __uint_as_float(a) / 127.0f : __uint_as_float(0x7fc00000u);
}

// Four codes x / d, rounded half away from zero; 0 for a row whose scale is 0
// (zeros, or magnitudes below 2^-143 whose 127th part is) or that is not
// finite.  The quotient is taken as x times 1 / d, which is off by
// at most 127 2^-22 (2 roundings): that decides the code unless the quotient
// lies within 1e-4 of a border between two, where the wave divides.  (Dividing
// always: 25.7 against 21.5 us for 3222 rows of 16 heads of 128.)
__device__ __forceinline__ uint32_t codes_q8(const float4& x, uint32_t a, float d) {
    const bool none = d == 0.0f || a >= 0x7f800000u;
    const float v[4] = {x.x, x.y, x.z, x.w};
    const float inv = 1.0f / d;
    float r[4];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r[e] = fabsf(v[e] * inv);
        near |= !(fabsf(__builtin_amdgcn_fractf(r[e]) - 0.5f) > 1e-4f);  // also where 1 / d is no number
    }
    if (__ballot(near && !none) != 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = roundf(fabsf(v[e] / d));
    }
    uint32_t packed = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int q = static_cast<int>(fminf(r[e] + 0.5f, 127.0f));
        packed |= (static_cast<uint32_t>(v[e] < 0.0f ? -q : q) & 0xffu) << (8 * e);
    }
    return none ? 0u : packed;
}

__device__ __forceinline__ uint32_t mag_bits4(const float4& x) {
    return max(max(mag_bits(x.x), mag_bits(x.y)), max(mag_bits(x.z), mag_bits(x.w)));
}

// Four floats at p; vec: p is 16-byte aligned.
__device__ __forceinline__ float4 load4(const float* p, bool vec) {
    if (vec) return *reinterpret_cast<const float4*>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
}

// Stores of results that this kernel does not read again, past the L2: a
// result left dirty there has to be written back when the kernel ends anyway,
// since the next kernel's readers sit on other XCDs.  The norm of 2048 rows of
// 5376 takes 30 us with them and 49 us with plain stores.
typedef float f32x4_nt __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void stream4(float* p, float4 v, bool vec) {
    if (vec) {
        __builtin_nontemporal_store(f32x4_nt{v.x, v.y, v.z, v.w}, reinterpret_cast<f32x4_nt*>(p));
    } else {
        __builtin_nontemporal_store(v.x, p);
        __builtin_nontemporal_store(v.y, p + 1);
        __builtin_nontemporal_store(v.z, p + 2);
        __builtin_nontemporal_store(v.w, p + 3);
    }
}

// A double of another lane by a DPP pattern (0 where the pattern has none).
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

}  // namespace qmv
