// The paged key/value cache: quantizing new rows into it and reading rows
// back as float32.
//
// A row (one token's head) of D elements is stored as D int8 codes and one
// float32 scale d = max|x| / 127, or as D float16.  Both kernels move every
// byte once and compute a few operations an element, so memory bounds them:
// 4 bytes in and 1 (2) out an element for the write, the reverse for the
// read.
//
// Work split: blockIdx.x is one row of the batch or a few, blockIdx.y keys
// or values.  D / 4 lanes hold a head's row, four elements each, so that the
// row's maximum is a few lane exchanges and a wave writes whole rows of codes.
#include <stdint.h>

#include "kv_device.h"
#include "step_device.h"
#include "step_internal.h"

namespace qmv {
namespace {

struct KvPlanes {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
};

// Places of the ROWS rows from `first` on, in LDS: -1 without a place, -2 for
// a row of no sequence.  The wave that runs this finds the first row's
// sequence, holds the 64 row starts behind it, and counts for each row how
// many it has passed.
template <int ROWS>
__device__ __forceinline__ void find_slots(const KvView& view, int first, int64_t* slots) {
    const int lane = threadIdx.x & (kWave - 1);
    const int b0 = find_sequence(view.row_start, view.B, first);
    const int ahead = b0 + 1 + lane;
    const int start = ahead <= view.B ? view.row_start[ahead] : INT32_MAX;
    int row = -1, b = -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = first + i;
        int c = __popcll(__ballot(start <= r));
        if (c == kWave) c = find_sequence(view.row_start, view.B, r) - b0;  // 64 empty sequences in between
        if (lane == i) {
            row = r;
            b = b0 + c;
        }
    }
    if (lane < ROWS) {
        int64_t slot = -2;
        if (row < view.T && b < view.B) {
            const int lo = view.row_start[b], end = view.row_start[b + 1];
            if (row >= lo && row < end) {
                slot = -1;
                const int64_t pos = static_cast<int64_t>(view.kv_len[b]) - (end - static_cast<int64_t>(row));
                if (pos >= 0 && (pos >> view.page_shift) < view.max_pages) {
                    const int page = view.table[static_cast<int64_t>(b) * view.max_pages + (pos >> view.page_shift)];
                    if (page >= 0 && page < view.num_pages)
                        slot = (static_cast<int64_t>(page) << view.page_shift) + (pos & ((1 << view.page_shift) - 1));
                }
            }
        }
        slots[lane] = slot;
    }
}

// The (row, quad of elements) pairs of ROWS rows of `quads` quads, 256 a
// step: rows side by side where a row has fewer than 256.
template <int ROWS>
struct Steps {
    int quads, wide, sub, quad, per, count;
    __device__ __forceinline__ explicit Steps(int quads_) : quads(quads_) {
        wide = quads < kBlockThreads ? kBlockThreads / quads : 1;  // rows of a step
        sub = wide > 1 ? threadIdx.x / quads : 0;
        quad = threadIdx.x - sub * quads;
        if (sub >= wide) quad = quads;  // left over: never in
        per = (quads + kBlockThreads - 1) / kBlockThreads;  // steps of a row
        count = wide > 1 ? (ROWS + wide - 1) / wide : ROWS * per;
    }
    __device__ __forceinline__ bool at(int step, int* row, int* q) const {
        if (wide > 1) {
            *row = step * wide + sub;
            *q = quad;
        } else {
            *row = step / per;
            *q = quad + (step - *row * per) * kBlockThreads;
        }
        return step < count && *row < ROWS && *q < quads;
    }
};

constexpr int kUnroll = 4;  // steps whose loads are in flight together

// F16: the row's maximum decides only whether every element is finite.
template <int D, bool F16, int ROWS>
__global__ __launch_bounds__(kBlockThreads)
void kv_write_kernel(KvView view, KvPlanes c, const float* __restrict__ k, int64_t ldk, const float* __restrict__ v,
                     int64_t ldv, bool vec) {
    constexpr int L = D / 4;  // lanes of a head's row
    __shared__ int64_t slots[ROWS];
    const bool values = blockIdx.y != 0;
    const int first = blockIdx.x * ROWS;
    const float* src = values ? v : k;
    const int64_t ld = values ? ldv : ldk;
    void* codes = values ? c.v : c.k;
    float* scales = values ? c.v_scale : c.k_scale;
    if (threadIdx.x < kWave) find_slots<ROWS>(view, first, slots);
    const Steps<ROWS> steps(view.heads * L);
    const int in_page = (1 << view.page_shift) - 1;
    for (int s0 = 0; s0 < steps.count; s0 += kUnroll) {
        float4 x[kUnroll];
        int row[kUnroll], q[kUnroll];
        bool in[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            in[i] = steps.at(s0 + i, &row[i], &q[i]) && first + row[i] < view.T;
            x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (in[i]) x[i] = load4(src + (first + row[i]) * ld + 4 * q[i], vec);
        }
        if (s0 == 0) __syncthreads();  // the slots, found while the first rows come
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            // the D / 4 lanes of a head's row are in or out together
            const int64_t slot = in[i] ? slots[row[i]] : -1;
            const int h = q[i] / L, sub = q[i] % L;
            const int64_t cell = (((slot >> view.page_shift) * view.heads + h) << view.page_shift) + (slot & in_page);
            if constexpr (F16) {
                const _Float16 f[4] = {static_cast<_Float16>(x[i].x), static_cast<_Float16>(x[i].y),
                                       static_cast<_Float16>(x[i].z), static_cast<_Float16>(x[i].w)};
                uint32_t a = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) a = max(a, mag_bits(static_cast<float>(f[e])));
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), o, L)));
                uint2 packed;
                packed.x = __builtin_bit_cast(uint16_t, f[0]) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, f[1])) << 16);
                packed.y = __builtin_bit_cast(uint16_t, f[2]) | (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, f[3])) << 16);
                if (a >= 0x7f800000u) packed = make_uint2(0x7e007e00u, 0x7e007e00u);
                if (slot >= 0)
                    __builtin_nontemporal_store(packed.x | static_cast<uint64_t>(packed.y) << 32,
                                                reinterpret_cast<uint64_t*>(codes) + cell * L + sub);
            } else {
                uint32_t a = mag_bits4(x[i]);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), o, L)));
                const float d = scale_q8(a);
                const uint32_t packed = codes_q8(x[i], a, d);
                if (slot >= 0) {
                    __builtin_nontemporal_store(packed, reinterpret_cast<uint32_t*>(codes) + cell * L + sub);
                    if (sub == 0) __builtin_nontemporal_store(d, scales + cell);
                }
            }
        }
    }
}

template <int D, bool F16, int ROWS>
__global__ __launch_bounds__(kBlockThreads)
void kv_read_kernel(KvView view, KvPlanes c, float* __restrict__ k, int64_t ldk, float* __restrict__ v, int64_t ldv,
                    bool vec) {
    constexpr int L = D / 4;
    __shared__ int64_t slots[ROWS];
    const bool values = blockIdx.y != 0;
    const int first = blockIdx.x * ROWS;
    float* dst = values ? v : k;
    const int64_t ld = values ? ldv : ldk;
    const void* codes = values ? c.v : c.k;
    const float* scales = values ? c.v_scale : c.k_scale;
    if (threadIdx.x < kWave) find_slots<ROWS>(view, first, slots);
    const Steps<ROWS> steps(view.heads * L);
    const int in_page = (1 << view.page_shift) - 1;
    __syncthreads();
    for (int s0 = 0; s0 < steps.count; s0 += kUnroll) {
        uint2 p[kUnroll];
        float d[kUnroll];
        int row[kUnroll], q[kUnroll];
        int64_t slot[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            slot[i] = steps.at(s0 + i, &row[i], &q[i]) ? slots[row[i]] : -2;
            p[i] = make_uint2(0u, 0u);
            d[i] = 0.0f;
            if (slot[i] >= 0) {
                const int64_t cell =
                    (((slot[i] >> view.page_shift) * view.heads + q[i] / L) << view.page_shift) + (slot[i] & in_page);
                if constexpr (F16) {
                    p[i] = reinterpret_cast<const uint2*>(codes)[cell * L + q[i] % L];
                } else {
                    p[i].x = reinterpret_cast<const uint32_t*>(codes)[cell * L + q[i] % L];
                    d[i] = scales[cell];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (slot[i] == -2) continue;
            float4 x;
            if constexpr (F16) {
                x = make_float4(half_bits_to_float(p[i].x & 0xffffu), half_bits_to_float(p[i].x >> 16),
                                half_bits_to_float(p[i].y & 0xffffu), half_bits_to_float(p[i].y >> 16));
            } else {
                x = make_float4(sbyte<0>(p[i].x) * d[i], sbyte<1>(p[i].x) * d[i], sbyte<2>(p[i].x) * d[i],
                                sbyte<3>(p[i].x) * d[i]);
            }
            stream4(dst + (first + row[i]) * ld + 4 * q[i], x, vec);
        }
    }
}

// float4 accesses need 16-byte aligned rows
bool vec_rows(const void* k, int64_t ldk, const void* v, int64_t ldv) {
    return ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 && ldk % 4 == 0 && ldv % 4 == 0;
}

}  // namespace

// Rows of a workgroup: one of a few; of many, four wide ones or sixteen
// narrow ones (a row's places are found together, and the rows that a
// workgroup moves are about 2048 float4).  Whole sequences of 16 heads of 128,
// 20,527 rows: 69.5 us with four rows, 75.7 with eight, 88.1 with sixteen;
// 8693 rows of 3 heads of 64: 9.1, 7.4, 7.1 us.
inline int rows_of(int64_t T, int quads) { return T < 1024 ? 1 : quads >= 256 ? 4 : 16; }

#define KV_LAUNCH(kernel, D, ...)                                                                               \
    do {                                                                                                        \
        const int rows = rows_of(b.T, c.kv_heads * (D / 4));                                                    \
        const dim3 grid(static_cast<unsigned>((b.T + rows - 1) / rows), 2);                                     \
        if (c.format == QMV_KV_F16) {                                                                           \
            if (rows == 1) hipLaunchKernelGGL((kernel<D, true, 1>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__); \
            else if (rows == 4) hipLaunchKernelGGL((kernel<D, true, 4>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__); \
            else hipLaunchKernelGGL((kernel<D, true, 16>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__);  \
        } else {                                                                                                \
            if (rows == 1) hipLaunchKernelGGL((kernel<D, false, 1>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__); \
            else if (rows == 4) hipLaunchKernelGGL((kernel<D, false, 4>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__); \
            else hipLaunchKernelGGL((kernel<D, false, 16>), grid, dim3(kBlockThreads), 0, stream, __VA_ARGS__); \
        }                                                                                                       \
    } while (0)

hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* k, int64_t ldk, const float* v,
                           int64_t ldv, hipStream_t stream) {
    const KvView view = view_of(c, b);
    const KvPlanes p{c.k, c.v, c.k_scale, c.v_scale};
    const bool vec = vec_rows(k, ldk, v, ldv);
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
    if (c.head_dim == 64) KV_LAUNCH(kv_read_kernel, 64, view, p, k, ldk, v, ldv, vec);
    else if (c.head_dim == 128) KV_LAUNCH(kv_read_kernel, 128, view, p, k, ldk, v, ldv, vec);
    else KV_LAUNCH(kv_read_kernel, 256, view, p, k, ldk, v, ldv, vec);
    return hipGetLastError();
}

}  // namespace qmv
