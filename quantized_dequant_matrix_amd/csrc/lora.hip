// Low-rank adapters of the sequences of a batch, added to a shared
// projection's output:  y_r = base_r + scale_s Bm_s (A_s x_r).
//
// Two launches, over tiles of up to 16 rows of one sequence:
//   shrink  v = A_s x, split over K: a workgroup a (tile, K share), its four
//           waves a quarter each; shares are summed by the next launch in
//           their order, so that no atomics are needed
//   expand  y = base + scale_s Bm_s v, a workgroup a (tile, N share)
//
// Both products are float32 matrix instructions (16 x 16 x 4) on weights that
// become float32 exactly: x and v are not rounded, and the 134 TFLOP/s that
// they reach are more than the memory asks for up to ranks around 64 (a 16 x
// 16 tile of y moves 2 KB, which takes as long as 64 ranks' products).  A
// single row would waste 15 of 16 columns: its expansion, which reads most of
// the weights, has a lane an output instead.
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
// wave) without sums over the batch.
__device__ __forceinline__ Tile tile_of(const LoraView& D, int tile) {
    const int32_t* start = D.a.row_start;
    const int lane = threadIdx.x & (kWave - 1);
    int lo = 0, span = static_cast<int>(D.a.B);
    while (span > 0) {
        const int step = (span + kWave - 1) / kWave;
        const int off = (lane + 1) * step;
        const bool below = off <= span && (start[lo + off] >> 4) + static_cast<int64_t>(lo + off) <= tile;
        const int c = __popcll(__ballot(below));
        const int left = span - c * step;
        lo += c * step;
        span = left < step - 1 ? left : step - 1;
    }
    Tile t = {0, 0, -1};
    if (lo >= D.a.B) return t;
    const int64_t first = start[lo], end = min(static_cast<int64_t>(start[lo + 1]), D.a.T);
    const int64_t row = first + kTile * (tile - (first >> 4) - lo);
    if (row < 0 || row >= end) return t;
    t.row = static_cast<int>(row);
    t.rows = static_cast<int>(min(end - row, static_cast<int64_t>(kTile)));
    t.slot = D.a.adapter[lo];
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

template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
    [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
    (std::make_integer_sequence<int, N>{});
}

// RT: 16 ranks each, at most.
template <bool BF16, int RT>
__global__ __launch_bounds__(kBlockThreads)
void lora_shrink_kernel(LoraView D) {
    __shared__ f32x4 lds[kWaves][RT][kWave];
    // steps of 32 k that are loaded at once: their latency is the time of this
    // kernel, and 128 k are a wave's share where there are many
    constexpr int kSteps = RT <= 4 ? 4 : (RT <= 8 ? 2 : 1);
    const Tile t = tile_of(D, blockIdx.x);
    if (t.rows == 0) return;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
    const float* x = D.a.x + (t.row + min(i, t.rows - 1)) * D.a.ldx;
    const int64_t lo = (static_cast<int64_t>(blockIdx.y) * kWaves + wave) * D.k_wave, hi = min(lo + D.k_wave, D.l.K);
    f32x4 xs[kSteps][2];
    auto load_x = [&](int64_t k0) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t k = k0 + 32 * s + 8 * g;
            const bool in = k < hi;
            const float* p = x + (in ? k : 0);
            if (D.x_vec) {
                xs[s][0] = *reinterpret_cast<const f32x4*>(p);
                xs[s][1] = *reinterpret_cast<const f32x4*>(p + 4);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xs[s][0][e] = p[e];
                    xs[s][1][e] = p[4 + e];
                }
            }
            if (!in) xs[s][0] = xs[s][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    };
    load_x(lo);  // while the adapter is looked up
    const int rank = rank_of(D, t);
    if (rank == 0) return;
    const int tiles = (rank + 15) / 16;
    const uint16_t* A = static_cast<const uint16_t*>(D.l.A) + static_cast<int64_t>(t.slot) * D.l.max_rank * D.l.K;
    f32x4 acc[RT] = {};
    for (int64_t k0 = lo; k0 < hi; k0 += 32 * kSteps) {
        if (k0 > lo) load_x(k0);
        uint32_t a[kSteps][RT][4];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t k = k0 + 32 * s + 8 * g;
            const bool in = k < hi;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r >= tiles) continue;
                const int j = 16 * r + i;
                const bool real = in && j < rank;  // what lies behind the rank or K may be anything
                const uint4 w = *reinterpret_cast<const uint4*>(A + (j < rank ? j : 0) * D.l.K + (in ? k : 0));
                a[s][r][0] = real ? w.x : 0u;
                a[s][r][1] = real ? w.y : 0u;
                a[s][r][2] = real ? w.z : 0u;
                a[s][r][3] = real ? w.w : 0u;
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (k0 + 32 * s >= hi) continue;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r >= tiles) continue;
                static_for<8>([&](auto e) {
                    constexpr int kE = decltype(e)::value;
                    acc[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(element<BF16, kE>(a[s][r]), xs[s][kE / 4][kE % 4], acc[r], 0,
                                                                  0, 0);
                });
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
        if (r < tiles) lds[wave][r][lane] = acc[r];
    __syncthreads();
    float* part = D.part + (static_cast<int64_t>(blockIdx.y) * D.a.T + t.row) * D.l.max_rank;
    for (int o = threadIdx.x; o < tiles * kWave; o += kBlockThreads) {
        const int r = o / kWave, l = o & (kWave - 1), row = l & 15, j = 16 * r + 4 * (l >> 4);
        f32x4 sum = lds[0][r][l];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += lds[w][r][l];
        if (row < t.rows && j < D.l.max_rank) *reinterpret_cast<f32x4*>(part + static_cast<int64_t>(row) * D.l.max_rank + j) = sum;
    }
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

template <bool BF16, int RT>
__global__ __launch_bounds__(kBlockThreads)
void lora_expand_kernel(LoraView D) {
    __shared__ float v_row[256];
    const Tile t = tile_of(D, blockIdx.x);
    if (t.rows == 0) return;
    const int64_t lo = static_cast<int64_t>(blockIdx.y) * D.n_share, hi = min(lo + D.n_share, D.l.N);
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
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
    const int64_t share = D.a.T * D.l.max_rank;  // of K, in part
    const float* part = D.part + static_cast<int64_t>(t.row) * D.l.max_rank;
    if (t.rows == 1) {
        const int64_t n = lo + threadIdx.x;  // the share is a thread's output each, or a few
        constexpr int kVec = RT * 2;         // 16-byte pieces of a row of Bm
        uint4 w[kVec];
        float b = 0.0f;
        auto load = [&](int64_t n) {
            b = D.a.base ? D.a.base[t.row * D.a.ldb + n] : 0.0f;
#pragma unroll
            for (int c = 0; c < kVec; ++c)
                if (8 * c < rank) w[c] = *reinterpret_cast<const uint4*>(Bm + n * D.l.max_rank + 8 * c);
        };
        if (n < hi) load(n);  // while v is summed
        if (threadIdx.x < RT * 16) {
            float sum = 0.0f;
            if (threadIdx.x < rank)
                for (int s = 0; s < D.k_shares; ++s) sum += part[s * share + threadIdx.x];
            v_row[threadIdx.x] = sum;
        }
        __syncthreads();
        for (int64_t m = n; m < hi; m += kBlockThreads) {
            if (m > n) load(m);
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                if (8 * c >= rank) continue;
                const uint32_t d[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                static_for<8>([&](auto e) {
                    constexpr int kE = decltype(e)::value;
                    const float a = element<BF16, kE>(d);
                    // what lies behind the rank may be anything
                    sum = fmaf(8 * c + kE < rank ? a : 0.0f, v_row[8 * c + kE], sum);
                });
            }
            D.a.y[t.row * D.a.ldy + m] = fmaf(scale, sum, b);
        }
        return;
    }
    constexpr int kE = RT == 1 ? 4 : 8;        // neighbouring ranks of a lane
    constexpr int kR = RT * 16 / (4 * kE);     // steps of 4 kE ranks
    constexpr int kAtOnce = kR < 4 ? kR : 4;   // steps whose weights are in registers
    const int steps = (rank + 4 * kE - 1) / (4 * kE);
    float v[kR][kE];  // of row i
    {
        f32x4 sum[kR][kE / 4] = {};
        const float* p = part + static_cast<int64_t>(min(i, t.rows - 1)) * D.l.max_rank + kE * g;
        for (int s = 0; s < D.k_shares; ++s, p += share) {
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int h = 0; h < kE / 4; ++h)
                    if (4 * kE * r + kE * g + 4 * h < rank) sum[r][h] += *reinterpret_cast<const f32x4*>(p + 4 * kE * r + 4 * h);
        }
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int e = 0; e < kE; ++e) v[r][e] = 4 * kE * r + kE * g + e < rank ? sum[r][e / 4][e % 4] : 0.0f;
    }
    for (int64_t n0 = lo + wave * 64; n0 < hi; n0 += kWaves * 64) {
        const int64_t n = n0 + 4 * i;
        f32x4 b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // row 4 g + q
            b[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (D.a.base && 4 * g + q < t.rows) b[q] = load4_of(D.a.base + (t.row + 4 * g + q) * D.a.ldb, n, hi, D.y_vec);
        }
        f32x4 acc[4] = {};
#pragma unroll
        for (int r0 = 0; r0 < kR; r0 += kAtOnce) {
            if (r0 >= steps) continue;
            uint32_t w[kAtOnce][4][kE / 2];
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = 4 * kE * (r0 + r) + kE * g;
                    const uint16_t* p = Bm + min(n + u, D.l.N - 1) * D.l.max_rank + j;
#pragma unroll
                    for (int d = 0; d < kE / 2; ++d) w[r][u][d] = 0u;
                    if (j >= rank) continue;
                    if constexpr (kE == 8) {
                        const uint4 q = *reinterpret_cast<const uint4*>(p);
                        w[r][u][0] = q.x; w[r][u][1] = q.y; w[r][u][2] = q.z; w[r][u][3] = q.w;
                    } else {
                        const uint2 q = *reinterpret_cast<const uint2*>(p);
                        w[r][u][0] = q.x; w[r][u][1] = q.y;
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
                if (r0 + r >= steps) continue;
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
            if (4 * g + q >= t.rows) continue;
            f32x4 o;
#pragma unroll
            for (int u = 0; u < 4; ++u) o[u] = fmaf(scale, acc[u][q], b[q][u]);
            store4_of(D.a.y + (t.row + 4 * g + q) * D.a.ldy, n, hi, D.y_vec, o);
        }
    }
}

// Tiles of the numbering above.
int64_t tiles_of(int64_t B, int64_t T) { return T / kTile + B; }

// K shares: enough that some 4096 waves are at work, of 128 k a wave at least.
void split_k(const qmv_lora& l, int64_t B, int64_t T, int* shares, int64_t* per_wave) {
    const int64_t real = tiles_of(B, T) < T ? tiles_of(B, T) : T;  // tiles that can have rows
    int64_t want = 1024 / real, most = (l.K + 4 * 128 - 1) / (4 * 128);
    want = want < 1 ? 1 : (want > most ? most : want);
    *per_wave = ((l.K + want * kWaves - 1) / (want * kWaves) + 31) / 32 * 32;
    *shares = static_cast<int>((l.K + *per_wave * kWaves - 1) / (*per_wave * kWaves));
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

size_t lora_ws_bytes(const qmv_lora& l, int64_t B, int64_t T) {
    int shares;
    int64_t per_wave;
    split_k(l, B, T, &shares, &per_wave);
    return static_cast<size_t>(shares) * static_cast<size_t>(T) * static_cast<size_t>(l.max_rank) * sizeof(float);
}

hipError_t launch_lora(const qmv_lora& l, const LoraArgs& a, void* ws, hipStream_t stream) {
    LoraView D;
    D.l = l;
    D.a = a;
    D.part = static_cast<float*>(ws);
    split_k(l, a.B, a.T, &D.k_shares, &D.k_wave);
    const int64_t real = tiles_of(a.B, a.T) < a.T ? tiles_of(a.B, a.T) : a.T;
    int64_t share = (l.N * real / 2048 + 255) / 256 * 256;
    share = share < 256 ? 256 : (share > 2048 ? 2048 : share);
    const int64_t least = (l.N / 65535 + 256) / 256 * 256;  // a grid has at most 65535 of them
    D.n_share = share < least ? least : share;
    D.x_vec = rows_aligned(a.x, a.ldx);
    D.y_vec = rows_aligned(a.y, a.ldy) && (!a.base || rows_aligned(a.base, a.ldb));
    return l.format == QMV_LORA_BF16 ? launch_rank<true>(D, stream) : launch_rank<false>(D, stream);
}

}  // namespace qmv
