// Low-rank adapters of the sequences of a batch, added to a shared
// projection's output:  y_r = base_r + scale_s Bm_s (A_s x_r).
//
// Two launches, over tiles of up to 16 rows of one sequence:
//   shrink  v = A_s x, split over K: a workgroup a (tile, K share), its four
//           waves a quarter each; shares are summed by the next launch in
//           their order, so that no atomics are needed
//   expand  y = base + scale_s Bm_s v, a workgroup a (tile, N share)
//
// Both products are float32 matrix instructions (16 x 16 x 4, 36 cycles) on
// weights that become float32 exactly: x and v are not rounded, and the 140
// TFLOP/s that they reach are more than the memory asks for up to ranks around
// 64 (a 16 x 16 tile of y moves 2 KB, which takes as long as 64 ranks'
// products).  A single row would waste 15 of 16 columns: it has the same loads
// and ordinary multiplications (32 rows of rank 64: 12.4 -> 8.5 us for shrink).
//
// Bounds, and what was measured: chunks are bound by HBM (1611 rows, 5376 ->
// 21504, rank 16: 308 MB in 67 us, 4.6 TB/s); single rows with many adapters by
// the lines of Bm (a row of Bm of max_rank 64 is a 128-byte line, read whole
// whatever the adapter's own rank: 28 rows over 18 adapters 24 us, of which
// expand takes 15 and reads 75 MB by the counters of HBM, 50 of lines of Bm and
// again what rows of one adapter on different dies do not share); one row by its
// two launches (7.9 us).  Two to eight rows of each of those sequences take 31-40
// us: lines of 75-100 MB at 2.7-3.6 TB/s, by tiles of 16 rows.  Rows of y that are
// not 16-byte aligned are stored by 4 bytes: chunks of 1600 rows take 126 us then,
// not 66.
//
// The operands' k index is a dummy: lane (i, g) = (l % 16, l / 16) holds
// eight neighbouring elements of its row (four of ranks up to 16), and
// instruction e takes element e of each, so that loads are 16 (8) bytes.
// Results: lane (i, g) has rows 4 g .. 4 g + 3 of column i.  In shrink these
// are four neighbouring ranks of x's row i; in expand rows of y, whose column i
// is output n0 + 4 i + u in the u-th of four products, so that the four are
// neighbours and a load or store of y is 256 bytes in a row of four rows.
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "qmv_device.h"
#include "serve_internal.h"
#include "sort_device.h"
#include "step_device.h"

namespace qmv {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;
constexpr int kWaves = kWavesPerBlock;

struct LoraView {
    qmv_lora l;
    LoraArgs a;
    float* part;       // [k_shares][T][max_rank]
    int k_shares;
    int64_t k_wave;    // K of a wave, a multiple of 32
    int64_t n_share;   // N of a workgroup of the expand kernel, a multiple of 256
    bool x_vec, y_vec; // rows of x, and of base and y, are 16-byte aligned
};

// A tile's rows and its adapter.
struct Tile {
    int row, rows;  // rows 0: nothing to do
    int slot;       // as the caller gave it
};

// Sequence b's tiles have the numbers from row_start[b] / 16 + b on: enough for
// its rows whatever their alignment, and in the order of the sequences, so
// that a tile's sequence is found by a search (64 entries a step, by the whole
// wave) without sums over the batch.  Numbers below row_start[0] / 16 are found
// in the first sequence and are of rows before it, which belong to none.
__device__ __forceinline__ Tile tile_of(const LoraView& D, int tile) {
    const int32_t* start = D.a.row_start;
    const int lane = threadIdx.x & (kWave - 1), B = static_cast<int>(D.a.B);
    Tile t = {0, 0, -1};
    int lo = 0;
    int64_t first, end;
    if (B <= kWave) {  // all entries at once
        const int b = min(lane, B - 1);
        const int32_t s0 = start[b], s1 = start[b + 1], slot = D.a.adapter[b];
        lo = __popcll(__ballot(lane < B && (s1 >> 4) + static_cast<int64_t>(lane + 1) <= tile));
        if (lo >= B) return t;
        first = __builtin_amdgcn_readlane(s0, lo);
        end = __builtin_amdgcn_readlane(s1, lo);
        t.slot = __builtin_amdgcn_readlane(slot, lo);
    } else {
        int span = B;
        while (span > 0) {
            const int step = (span + kWave - 1) / kWave;
            const int off = (lane + 1) * step;
            const bool below = off <= span && (start[lo + off] >> 4) + static_cast<int64_t>(lo + off) <= tile;
            const int c = __popcll(__ballot(below));
            const int left = span - c * step;
            lo += c * step;
            span = left < step - 1 ? left : step - 1;
        }
        if (lo >= B) return t;
        first = start[lo];
        end = start[lo + 1];
        t.slot = D.a.adapter[lo];
    }
    end = min(end, D.a.T);
    const int64_t row = first + kTile * (tile - (first >> 4) - lo);
    if (row < 0 || row < first || row >= end) return t;
    t.row = static_cast<int>(row);
    t.rows = static_cast<int>(min(end - row, static_cast<int64_t>(kTile)));
    return t;
}

// The tile's rank, 0 without an adapter.
__device__ __forceinline__ int rank_of(const LoraView& D, const Tile& t) {
    if (t.slot < 0 || t.slot >= D.l.slots) return 0;
    const int r = D.l.rank ? D.l.rank[t.slot] : D.l.max_rank;
    return r < 0 ? 0 : (r > D.l.max_rank ? D.l.max_rank : r);
}

// Elements I of a vector of 16-bit weights, as float32.
template <bool BF16, int I>
__device__ __forceinline__ float element(const uint32_t* w) {
    const uint32_t d = w[I / 2];
    if constexpr (BF16) return __uint_as_float(I % 2 ? d & 0xffff0000u : d << 16);
    return half_bits_to_float(I % 2 ? d >> 16 : d & 0xffffu);
}

// v of lane ^ d.
__device__ __forceinline__ float xor_lane(float v, int d) {
    return __uint_as_float(xor_lanes(__float_as_uint(v), d));
}

template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
    [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
    (std::make_integer_sequence<int, N>{});
}

// A wave's share of v = A x: lo .. hi of K, NT times 16 ranks.  Nothing here
// branches between a load and the next: addresses are held inside the buffers,
// and what does not count is taken out where it is used.  (Loads behind
// branches were waited for one by one.)
template <bool BF16, int NT, bool VEC, bool ONE>
__device__ __forceinline__ void shrink_wave(const LoraView& D, const float* x, const uint16_t* A, int rank, int64_t lo,
                                            int64_t hi, f32x4 (&acc)[NT]) {
    // steps of 32 k that are loaded at once: their latency is the time of this
    // kernel, and 128 k are a wave's share where there are many.  Of several rows
    // and many ranks fewer at once, for a wave more a SIMD (1620 rows, rank up to
    // 128: 20.8 -> 18.6 us).
    constexpr int kSteps = NT <= 2 ? 4 : (NT <= 4 ? (ONE ? 4 : 2) : (NT <= 8 ? (ONE ? 2 : 1) : 1));
    const int lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
    const uint16_t* row[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) row[r] = A + min(16 * r + i, rank - 1) * D.l.K;
    for (int64_t k0 = lo; k0 < hi; k0 += 32 * kSteps) {
        f32x4 xs[kSteps][2];
        uint4 a[kSteps][NT];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t k = min(k0 + 32 * s + 8 * g, hi - 8);
            if constexpr (VEC) {
                xs[s][0] = *reinterpret_cast<const f32x4*>(x + k);
                xs[s][1] = *reinterpret_cast<const f32x4*>(x + k + 4);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xs[s][0][e] = x[k + e];
                    xs[s][1][e] = x[k + 4 + e];
                }
            }
#pragma unroll
            for (int r = 0; r < NT; ++r) a[s][r] = *reinterpret_cast<const uint4*>(row[r] + k);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const bool in = k0 + 32 * s + 8 * g < hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xs[s][0][e] = in ? xs[s][0][e] : 0.0f;
                xs[s][1][e] = in ? xs[s][1][e] : 0.0f;
            }
            uint32_t w[NT][4];
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                // what lies behind the rank may be anything, and so may x beside it
                const bool real = in && 16 * r + i < rank;
                w[r][0] = real ? a[s][r].x : 0u;
                w[r][1] = real ? a[s][r].y : 0u;
                w[r][2] = real ? a[s][r].z : 0u;
                w[r][3] = real ? a[s][r].w : 0u;
            }
            static_for<8>([&](auto e) {
                constexpr int kE = decltype(e)::value;
#pragma unroll
                for (int r = 0; r < NT; ++r)
                    if constexpr (ONE)
                        acc[r][kE % 4] = fmaf(element<BF16, kE>(w[r]), xs[s][kE / 4][kE % 4], acc[r][kE % 4]);
                    else
                        acc[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(element<BF16, kE>(w[r]), xs[s][kE / 4][kE % 4], acc[r], 0, 0,
                                                                  0);
            });
        }
    }
}

// The workgroup's: the waves' sums through LDS, in their order.
template <bool BF16, int NT>
__device__ __forceinline__ void shrink_tile(const LoraView& D, const Tile& t, int rank, f32x4* lds) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), i = lane & 15;
    const float* x = D.a.x + (t.row + min(i, t.rows - 1)) * D.a.ldx;
    const uint16_t* A = static_cast<const uint16_t*>(D.l.A) + static_cast<int64_t>(t.slot) * D.l.max_rank * D.l.K;
    const int64_t lo = (static_cast<int64_t>(blockIdx.y) * kWaves + wave) * D.k_wave, hi = min(lo + D.k_wave, D.l.K);
    f32x4 acc[NT] = {};
    float* part = D.part + (static_cast<int64_t>(blockIdx.y) * D.a.T + t.row) * D.l.max_rank;
    if (t.rows == 1) {
        // lane (i, g) has the sum over its k for rank 16 r + i
        if (D.x_vec)
            shrink_wave<BF16, NT, true, true>(D, x, A, rank, lo, hi, acc);
        else
            shrink_wave<BF16, NT, false, true>(D, x, A, rank, lo, hi, acc);
        float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            float v = (acc[r][0] + acc[r][1]) + (acc[r][2] + acc[r][3]);
            v += xor_lane(v, 16);
            v += xor_lane(v, 32);
            if (lane < 16) sums[wave * (NT * 16) + 16 * r + lane] = v;
        }
        __syncthreads();
        const int j = threadIdx.x;
        if (j < NT * 16 && j < D.l.max_rank) {
            float v = sums[j];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += sums[w * (NT * 16) + j];
            part[j] = v;
        }
        return;
    }
    if (D.x_vec)
        shrink_wave<BF16, NT, true, false>(D, x, A, rank, lo, hi, acc);
    else
        shrink_wave<BF16, NT, false, false>(D, x, A, rank, lo, hi, acc);
#pragma unroll
    for (int r = 0; r < NT; ++r) lds[(wave * NT + r) * kWave + lane] = acc[r];
    __syncthreads();
#pragma unroll
    for (int r0 = 0; r0 < NT; r0 += kWaves) {
        const int r = r0 + wave, j = 16 * r + 4 * (lane >> 4);
        if (r >= NT || i >= t.rows || j >= D.l.max_rank) continue;
        f32x4 sum = lds[r * kWave + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += lds[(w * NT + r) * kWave + lane];
        *reinterpret_cast<f32x4*>(part + static_cast<int64_t>(i) * D.l.max_rank + j) = sum;
    }
}

// RT: 16 ranks each, at most; a tile takes the next power of two of its own.
template <bool BF16, int RT>
__global__ __launch_bounds__(kBlockThreads)
void lora_shrink_kernel(LoraView D) {
    __shared__ f32x4 lds[kWaves * RT * kWave];
    const Tile t = tile_of(D, blockIdx.x);
    if (t.rows == 0) return;
    const int rank = rank_of(D, t);
    if (rank == 0) return;
    if constexpr (RT > 8) {
        if (rank > 128) return shrink_tile<BF16, 16>(D, t, rank, lds);
    }
    if constexpr (RT > 4) {
        if (rank > 64) return shrink_tile<BF16, 8>(D, t, rank, lds);
    }
    if constexpr (RT > 2) {
        if (rank > 32) return shrink_tile<BF16, 4>(D, t, rank, lds);
    }
    if constexpr (RT > 1) {
        if (rank > 16) return shrink_tile<BF16, 2>(D, t, rank, lds);
    }
    shrink_tile<BF16, 1>(D, t, rank, lds);
}

// Four elements of a row from n on, whose last one is n_end - 1 (zeros behind it).
__device__ __forceinline__ f32x4 load4_of(const float* p, int64_t n, int64_t n_end, bool vec) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (vec && n + 4 <= n_end) {
        v = *reinterpret_cast<const f32x4*>(p + n);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < n_end) v[e] = p[n + e];
    }
    return v;
}

// Results are not read again here and go past the L2.
__device__ __forceinline__ void store4_of(float* p, int64_t n, int64_t n_end, bool vec, const f32x4& v) {
    if (vec && n + 4 <= n_end) {
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(p + n));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < n_end) p[n + e] = v[e];
    }
}

// v of the tile's rows, summed over the K shares in their order, into LDS (16
// rows, kStride apart).  Eight shares are asked for at once.
template <int RT, int kStride>
__device__ __forceinline__ void sum_shares(const LoraView& D, const Tile& t, int rank, float* lds) {
    constexpr int kQuads = RT * 4;  // of a row
    const int64_t share = D.a.T * D.l.max_rank;
    for (int o = threadIdx.x; o < t.rows * kQuads; o += kBlockThreads) {
        const int row = o / kQuads, j = 4 * (o & (kQuads - 1));
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        if (j < rank) {
            const float* p = D.part + static_cast<int64_t>(t.row + row) * D.l.max_rank + j;
            for (int s0 = 0; s0 < D.k_shares; s0 += 8) {
                f32x4 v[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) v[s] = *reinterpret_cast<const f32x4*>(p + min(s0 + s, D.k_shares - 1) * share);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s0 + s < D.k_shares) sum += v[s];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = j + e < rank ? sum[e] : 0.0f;
        }
        *reinterpret_cast<f32x4*>(lds + row * kStride + j) = sum;
    }
    __syncthreads();
}

// Several rows: 64 outputs a wave and turn.  No branch between loads (see
// shrink_wave) where the 64 are all there and aligned.
template <bool BF16, int NT, int kStride>
__device__ __forceinline__ void expand_rows(const LoraView& D, const Tile& t, int rank, float scale, const uint16_t* Bm,
                                            int64_t lo, int64_t hi, float* v_lds) {
    constexpr int kE = NT == 1 ? 4 : 8;       // neighbouring ranks of a lane
    constexpr int kR = NT * 16 / (4 * kE);    // steps of 4 kE ranks
    constexpr int kAtOnce = kR < 2 ? kR : 2;  // steps whose weights are in registers
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
    const int rows_here = t.rows - 4 * g;  // of this lane's four
    int64_t at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = t.row + min(4 * g + q, t.rows - 1);
    f32x4 b[4];
    uint32_t w[kAtOnce][4][kE / 2];
    auto load_base = [&](int64_t n0) {
        const int64_t n = n0 + 4 * i;
        if (!D.a.base) {
#pragma unroll
            for (int q = 0; q < 4; ++q) b[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        } else if (D.y_vec && n0 + 64 <= hi) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                b[q] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(D.a.base + at[q] * D.a.ldb + n));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) b[q] = load4_of(D.a.base + at[q] * D.a.ldb, n, hi, false);
        }
    };
    auto load_weights = [&](int64_t n0, int r0) {
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
            const int j = 4 * kE * (r0 + r) + kE * g;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint16_t* p = Bm + min(n0 + 4 * i + u, D.l.N - 1) * D.l.max_rank + (j < rank ? j : 0);
                if constexpr (kE == 8) {
                    const uint4 q = *reinterpret_cast<const uint4*>(p);
                    w[r][u][0] = q.x; w[r][u][1] = q.y; w[r][u][2] = q.z; w[r][u][3] = q.w;
                } else {
                    const uint2 q = *reinterpret_cast<const uint2*>(p);
                    w[r][u][0] = q.x; w[r][u][1] = q.y;
                }
            }
        }
    };
    // the first turn's loads while v is summed
    const int64_t first = lo + wave * 64;
    if (first < hi) {
        load_base(first);
        load_weights(first, 0);
    }
    sum_shares<NT, kStride>(D, t, rank, v_lds);
    float v[kR][kE];  // of row i
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int e = 0; e < kE; ++e) v[r][e] = v_lds[min(i, t.rows - 1) * kStride + 4 * kE * r + kE * g + e];
    for (int64_t n0 = first; n0 < hi; n0 += kWaves * 64) {
        const int64_t n = n0 + 4 * i;
        if (n0 > first) load_base(n0);
        f32x4 acc[4] = {};
#pragma unroll
        for (int r0 = 0; r0 < kR; r0 += kAtOnce) {
            if (n0 > first || r0 > 0) load_weights(n0, r0);
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
                const int left = rank - (4 * kE * (r0 + r) + kE * g);  // ranks of this lane that count
                static_for<kE>([&](auto e) {
                    constexpr int kI = decltype(e)::value;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float a = element<BF16, kI>(w[r][u]);
                        acc[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[r0 + r][kI], kI < left ? a : 0.0f, acc[u], 0, 0, 0);
                    }
                });
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 o;
#pragma unroll
            for (int u = 0; u < 4; ++u) o[u] = fmaf(scale, acc[u][q], b[q][u]);
            if (q < rows_here) store4_of(D.a.y + at[q] * D.a.ldy, n, hi, D.y_vec && n0 + 64 <= hi, o);
        }
    }
}

template <bool BF16, int RT>
__global__ __launch_bounds__(kBlockThreads)
void lora_expand_kernel(LoraView D) {
    constexpr int kStride = RT * 16 + 4;
    __shared__ __align__(16) float v_lds[kTile * kStride];
    const Tile t = tile_of(D, blockIdx.x);
    if (t.rows == 0) return;
    const int64_t lo = static_cast<int64_t>(blockIdx.y) * D.n_share, hi = min(lo + D.n_share, D.l.N);
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int rank = rank_of(D, t);
    if (rank == 0) {
        if (D.a.base == D.a.y) return;
        for (int64_t n = lo + 4 * threadIdx.x; n < hi; n += 4 * kBlockThreads) {
#pragma unroll 4
            for (int r = 0; r < t.rows; ++r) {
                const f32x4 b = D.a.base ? load4_of(D.a.base + (t.row + r) * D.a.ldb, n, hi, D.y_vec) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                store4_of(D.a.y + (t.row + r) * D.a.ldy, n, hi, D.y_vec, b);
            }
        }
        return;
    }
    const float scale = D.l.scale[t.slot];
    const uint16_t* Bm = static_cast<const uint16_t*>(D.l.Bm) + static_cast<int64_t>(t.slot) * D.l.N * D.l.max_rank;
    if (t.rows == 1) {
        sum_shares<RT, kStride>(D, t, rank, v_lds);
        // kL lanes hold a row of Bm, eight ranks each, so that a wave reads
        // whole rows one after the other; of kL loads every lane keeps one sum
        constexpr int kL = RT * 2, kRows = kWave / kL;
        const int piece = lane & (kL - 1), sub = lane / kL;
        const bool in = 8 * piece < rank;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v_lds[8 * piece + e];
        for (int64_t n0 = lo + wave * kWave; n0 < hi; n0 += kWaves * kWave) {
            uint4 w[kL];
#pragma unroll
            for (int u = 0; u < kL; ++u) {
                const int64_t n = min(n0 + u * kRows + sub, D.l.N - 1);
                w[u] = *reinterpret_cast<const uint4*>(Bm + n * D.l.max_rank + (in ? 8 * piece : 0));
            }
            const int64_t n = n0 + piece * kRows + sub;
            const float b = D.a.base && n < hi ? D.a.base[t.row * D.a.ldb + n] : 0.0f;
            float out = 0.0f;
#pragma unroll
            for (int u = 0; u < kL; ++u) {
                const uint32_t d[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                float sum = 0.0f;
                static_for<8>([&](auto e) {
                    constexpr int kE = decltype(e)::value;
                    const float a = element<BF16, kE>(d);
                    // what lies behind the rank may be anything
                    sum = fmaf(8 * piece + kE < rank ? a : 0.0f, v[kE], sum);
                });
#pragma unroll
                for (int d = 1; d < kL; d <<= 1) sum += xor_lane(sum, d);
                out = piece == u ? sum : out;
            }
            if (n < hi) D.a.y[t.row * D.a.ldy + n] = fmaf(scale, out, b);
        }
        return;
    }
    if constexpr (RT > 8) {
        if (rank > 128) return expand_rows<BF16, 16, kStride>(D, t, rank, scale, Bm, lo, hi, v_lds);
    }
    if constexpr (RT > 4) {
        if (rank > 64) return expand_rows<BF16, 8, kStride>(D, t, rank, scale, Bm, lo, hi, v_lds);
    }
    if constexpr (RT > 2) {
        if (rank > 32) return expand_rows<BF16, 4, kStride>(D, t, rank, scale, Bm, lo, hi, v_lds);
    }
    if constexpr (RT > 1) {
        if (rank > 16) return expand_rows<BF16, 2, kStride>(D, t, rank, scale, Bm, lo, hi, v_lds);
    }
    expand_rows<BF16, 1, kStride>(D, t, rank, scale, Bm, lo, hi, v_lds);
}

// Tiles of the numbering above.
int64_t tiles_of(int64_t B, int64_t T) { return T / kTile + B; }

int64_t tiles_with_rows(int64_t B, int64_t T) { return tiles_of(B, T) < T ? tiles_of(B, T) : T; }  // at most

// K shares: enough that some 4096 waves are at work, each with 128 k (what it
// loads at once) or a multiple.  More shares of fewer k gain nothing here and
// cost the expansion their sums (32 rows of rank up to 64: 128 k a wave 24 us,
// 64 k 25, 32 k 33 when the rest was 4 us slower).
int64_t most_shares(const qmv_lora& l) { return (l.K + kWaves * 128 - 1) / (kWaves * 128); }

void split_k(const qmv_lora& l, int64_t B, int64_t T, int* shares, int64_t* per_wave) {
    const int64_t most = most_shares(l);
    int64_t want = 1024 / tiles_with_rows(B, T);
    want = want < 1 ? 1 : (want > most ? most : want);
    *per_wave = ((l.K + want * kWaves - 1) / (want * kWaves) + 127) / 128 * 128;
    *shares = static_cast<int>((l.K + *per_wave * kWaves - 1) / (*per_wave * kWaves));
}

// Outputs of a workgroup of the expand kernel, a multiple of 256: some 4096
// workgroups for ranks up to 32, where HBM is the limit and an even end counts
// (1611 rows of 21504, rank 16: 67 us, with 1024 of them 76), some 1024 above,
// where the start of one, v and its own registers cost more (1620 rows of 5376,
// rank up to 128: 49 us, with 4096 of them 53).
int64_t share_n(const qmv_lora& l, int64_t B, int64_t T) {
    const int64_t workgroups = l.max_rank <= 32 ? 4096 : 1024;
    int64_t share = (l.N * tiles_with_rows(B, T) / workgroups + 255) / 256 * 256;
    share = share < 256 ? 256 : (share > 2048 ? 2048 : share);
    const int64_t least = (l.N / 65535 + 256) / 256 * 256;  // a grid has at most 65535 of them
    return share < least ? least : share;
}

template <bool BF16, int RT>
hipError_t launch(const LoraView& D, hipStream_t stream) {
    const unsigned tiles = static_cast<unsigned>(tiles_of(D.a.B, D.a.T));
    hipLaunchKernelGGL((lora_shrink_kernel<BF16, RT>), dim3(tiles, static_cast<unsigned>(D.k_shares)), dim3(kBlockThreads), 0,
                       stream, D);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((lora_expand_kernel<BF16, RT>),
                       dim3(tiles, static_cast<unsigned>((D.l.N + D.n_share - 1) / D.n_share)), dim3(kBlockThreads), 0, stream,
                       D);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_rank(const LoraView& D, hipStream_t stream) {
    if (D.l.max_rank <= 16) return launch<BF16, 1>(D, stream);
    if (D.l.max_rank <= 32) return launch<BF16, 2>(D, stream);
    if (D.l.max_rank <= 64) return launch<BF16, 4>(D, stream);
    if (D.l.max_rank <= 128) return launch<BF16, 8>(D, stream);
    return launch<BF16, 16>(D, stream);
}

bool rows_aligned(const float* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0; }

}  // namespace

// Enough for every batch of up to T rows, of any sequences.  Shares fall as the
// batch grows: the shares times the tiles are 1024 at most where there are
// several, and a tile has 16 rows at most; else there is one share.
size_t lora_ws_bytes(const qmv_lora& l, int64_t, int64_t T) {
    int64_t rows = most_shares(l) * T;
    if (rows > 1024 * kTile) rows = 1024 * kTile;
    return static_cast<size_t>(rows > T ? rows : T) * static_cast<size_t>(l.max_rank) * sizeof(float);
}

hipError_t launch_lora(const qmv_lora& l, const LoraArgs& a, void* ws, hipStream_t stream) {
    LoraView D;
    D.l = l;
    D.a = a;
    D.part = static_cast<float*>(ws);
    split_k(l, a.B, a.T, &D.k_shares, &D.k_wave);
    D.n_share = share_n(l, a.B, a.T);
    D.x_vec = rows_aligned(a.x, a.ldx);
    D.y_vec = rows_aligned(a.y, a.ldy) && (!a.base || rows_aligned(a.base, a.ldb));
    return l.format == QMV_LORA_BF16 ? launch_rank<true>(D, stream) : launch_rank<false>(D, stream);
}

}  // namespace qmv
