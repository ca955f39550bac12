// Sorting 64-bit keys in registers, shared by the kernels that select logits
// (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_device.h"

namespace qmv {

__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t umin64(uint64_t a, uint64_t b) { return a < b ? a : b; }

// v of lane ^ d, for d = 1, 2, 4, 8, 16, 32 (a constant once the sorting
// loops are unrolled), without the LDS crossbar: DPP quad permutes for 1 and
// 2, two row shifts for 4, a row rotation for 8, and gfx950's row and
// half-wave swaps for 16 and 32.
__device__ __forceinline__ uint32_t xor_lanes(uint32_t v, int d) {
    const int lane = threadIdx.x & (kWave - 1);
    switch (d) {
    case 1: return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, false));
    case 2: return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, false));
    case 4: {
        const uint32_t up = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x104, 0xF, 0xF, false));
        const uint32_t dn = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x114, 0xF, 0xF, false));
        return (lane & 4) ? dn : up;
    }
    case 8: return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x128, 0xF, 0xF, false));
    case 16: {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return ((lane >> 4) & 1) ? r[0] : r[1];
    }
    default: {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (lane >= 32) ? r[0] : r[1];
    }
    }
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d) {
    const uint32_t lo = xor_lanes(static_cast<uint32_t>(v), d);
    const uint32_t hi = xor_lanes(static_cast<uint32_t>(v >> 32), d);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// One compare-exchange of a bitonic network, seen from one element: e is the
// element's index, d its partner's distance, s the size of the sequences
// being merged.  Sequences whose index has bit s clear are sorted largest
// first, so the final pass (s = n) leaves everything largest first.
__device__ __forceinline__ uint64_t bitonic_keep(uint64_t mine, uint64_t other, int e, int d, int s) {
    const bool lower = (e & d) == 0;
    const bool desc = (e & s) == 0;
    return (lower == desc) ? umax64(mine, other) : umin64(mine, other);
}

// Sorts the 64 NK keys of a wave, largest first: key[j] of lane l is element
// j * 64 + l.  Steps with distance >= 64 stay in the lane's registers, the
// others exchange with lane ^ d.
template <int NK>
__device__ __forceinline__ void wave_sort_desc(uint64_t (&key)[NK]) {
    const int lane = threadIdx.x & (kWave - 1);
    constexpr int n = kWave * NK;
#pragma unroll
    for (int s = 2; s <= n; s <<= 1) {
#pragma unroll
        for (int d = s >> 1; d > 0; d >>= 1) {
            if (d >= kWave) {
                const int dj = d / kWave;
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    if ((j ^ dj) > j) {
                        const uint64_t a = key[j], b = key[j ^ dj];
                        key[j] = bitonic_keep(a, b, j * kWave, d, s);
                        key[j ^ dj] = bitonic_keep(b, a, (j ^ dj) * kWave, d, s);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < NK; ++j) key[j] = bitonic_keep(key[j], shfl_xor64(key[j], d), j * kWave + lane, d, s);
            }
        }
    }
}

// Sorts NB * T keys held by a workgroup of T threads (a power of two), largest
// first: key[j] of thread t is element j * T + t.  Steps with distance < 64 are
// shuffles inside a wave, steps with distance >= T stay in registers, the
// rest exchange through LDS (two buffers alternate, so one barrier a step).
template <int T, int NB>
__device__ __forceinline__ void block_sort_desc(uint64_t (&key)[NB], uint64_t* lds /* 2 * NB * T */) {
    constexpr int n = T * NB;
    const int t = threadIdx.x;
    int buf = 0;
#pragma unroll
    for (int s = 2; s <= n; s <<= 1) {
#pragma unroll
        for (int d = s >> 1; d > 0; d >>= 1) {
            if (d >= T) {
                const int dj = d / T;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    if ((j ^ dj) > j) {
                        const uint64_t a = key[j], b = key[j ^ dj];
                        key[j] = bitonic_keep(a, b, j * T, d, s);
                        key[j ^ dj] = bitonic_keep(b, a, (j ^ dj) * T, d, s);
                    }
                }
            } else if (d >= kWave) {
                uint64_t* B = lds + buf * (NB * T);
#pragma unroll
                for (int j = 0; j < NB; ++j) B[j * T + t] = key[j];
                __syncthreads();
#pragma unroll
                for (int j = 0; j < NB; ++j) key[j] = bitonic_keep(key[j], B[j * T + (t ^ d)], j * T + t, d, s);
                buf ^= 1;
            } else {
#pragma unroll
                for (int j = 0; j < NB; ++j) key[j] = bitonic_keep(key[j], shfl_xor64(key[j], d), j * T + t, d, s);
            }
        }
    }
}

}  // namespace qmv
