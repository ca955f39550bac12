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
// eight (four in expand) neighbouring elements of its row, and instruction e
// takes element e of each, so that loads are 16 (8) bytes.  Results: lane (i,
// g) has rows 4 g .. 4 g + 3 of column i: four neighbouring ranks, or outputs,
// of row i.
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
    int row, rows;  // rows <= 0: nothing to do
    int slot;       // -1: no adapter
    int rank;
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
    Tile t = {0, 0, -1, 0};
    if (lo >= D.a.B) return t;
    const int64_t first = start[lo], end = min(static_cast<int64_t>(start[lo + 1]), D.a.T);
    const int64_t row = first + kTile * (tile - (first >> 4) - lo);
    if (row < 0 || row >= end) return t;
    t.row = static_cast<int>(row);
    t.rows = static_cast<int>(min(end - row, static_cast<int64_t>(kTile)));
    const int s = D.a.adapter[lo];
    if (s < 0 || s >= D.l.slots) return t;
    t.slot = s;
    const int r = D.l.rank ? D.l.rank[s] : D.l.max_rank;
    t.rank = r < 0 ? 0 : (r > D.l.max_rank ? D.l.max_rank : r);
    return t;
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
    const Tile t = tile_of(D, blockIdx.x);
    if (t.rows <= 0 || t.slot < 0 || t.rank == 0) return;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
    const int tiles = (t.rank + 15) / 16;
    const float* x = D.a.x + (t.row + min(i, t.rows - 1)) * D.a.ldx;
    const uint16_t* A = static_cast<const uint16_t*>(D.l.A) + static_cast<int64_t>(t.slot) * D.l.max_rank * D.l.K;
    const int64_t lo = (static_cast<int64_t>(blockIdx.y) * kWaves + wave) * D.k_wave, hi = min(lo + D.k_wave, D.l.K);
    f32x4 acc[RT] = {};
    struct Loads {
        f32x4 x[2];
        uint32_t a[RT][4];
    };
    auto load = [&](int64_t k0) {
        Loads L;
        const int64_t k = k0 + 8 * g;
        const bool in = k < hi;
        const int64_t kc = in ? k : 0;
        if (D.x_vec) {
            L.x[0] = *reinterpret_cast<const f32x4*>(x + kc);
            L.x[1] = *reinterpret_cast<const f32x4*>(x + kc + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                L.x[0][e] = x[kc + e];
                L.x[1][e] = x[kc + 4 + e];
            }
        }
        if (!in) L.x[0] = L.x[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if (r >= tiles) continue;
            const int j = 16 * r + i;
            const bool real = in && j < t.rank;  // what lies behind the rank or K may be anything
            const uint4 w = *reinterpret_cast<const uint4*>(A + (j < t.rank ? j : 0) * D.l.K + kc);
            L.a[r][0] = real ? w.x : 0u;
            L.a[r][1] = real ? w.y : 0u;
            L.a[r][2] = real ? w.z : 0u;
            L.a[r][3] = real ? w.w : 0u;
        }
        return L;
    };
    if (lo < hi) {
        Loads now = load(lo);
        for (int64_t k0 = lo; k0 < hi; k0 += 32) {
            Loads next;
            if (k0 + 32 < hi) next = load(k0 + 32);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r >= tiles) continue;
                static_for<8>([&](auto e) {
                    acc[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(element<BF16, e>(now.a[r]), now.x[decltype(e)::value / 4][decltype(e)::value % 4], acc[r], 0,
                                                                  0, 0);
                });
            }
            now = next;
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

// base + add to y, four outputs from n on (fewer at the end of the row).
__device__ __forceinline__ void update4(const LoraView& D, int64_t row, int64_t n, const f32x4& add) {
    const float* b = D.a.base ? D.a.base + row * D.a.ldb + n : nullptr;
    float* y = D.a.y + row * D.a.ldy + n;
    if (D.y_vec && n + 4 <= D.l.N) {
        f32x4 v = b ? *reinterpret_cast<const f32x4*>(b) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        *reinterpret_cast<f32x4*>(y) = v + add;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < D.l.N) y[e] = (b ? b[e] : 0.0f) + add[e];
    }
}

template <bool BF16, int RT>
__global__ __launch_bounds__(kBlockThreads)
void lora_expand_kernel(LoraView D) {
    __shared__ float v_row[256];
    const Tile t = tile_of(D, blockIdx.x);
    if (t.rows <= 0) return;
    const int64_t lo = static_cast<int64_t>(blockIdx.y) * D.n_share, hi = min(lo + D.n_share, D.l.N);
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
    if (t.slot < 0 || t.rank == 0) {
        if (D.a.base == D.a.y) return;
        for (int r = 0; r < t.rows; ++r)
            for (int64_t n = lo + 4 * threadIdx.x; n < hi; n += 4 * kBlockThreads)
                update4(D, t.row + r, n, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        return;
    }
    const float scale = D.l.scale[t.slot];
    const uint16_t* Bm = static_cast<const uint16_t*>(D.l.Bm) + static_cast<int64_t>(t.slot) * D.l.N * D.l.max_rank;
    const int64_t share = D.a.T * D.l.max_rank;  // of K, in part
    const float* part = D.part + static_cast<int64_t>(t.row) * D.l.max_rank;
    if (t.rows == 1) {
        if (threadIdx.x < t.rank) {
            float sum = 0.0f;
            for (int s = 0; s < D.k_shares; ++s) sum += part[s * share + threadIdx.x];
            v_row[threadIdx.x] = sum;
        }
        __syncthreads();
        for (int64_t n = lo + threadIdx.x; n < hi; n += kBlockThreads) {
            const uint16_t* w = Bm + n * D.l.max_rank;
            float sum = 0.0f;
            for (int j = 0; j + 8 <= t.rank; j += 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(w + j);
                const uint32_t d[4] = {q.x, q.y, q.z, q.w};
                static_for<8>([&](auto e) { sum = fmaf(element<BF16, e>(d), v_row[j + e], sum); });
            }
            if (t.rank & 7) {
                const int j = t.rank & ~7;
                const uint4 q = *reinterpret_cast<const uint4*>(w + j);
                const uint32_t d[4] = {q.x, q.y, q.z, q.w};
                static_for<8>([&](auto e) {
                    if (j + e < t.rank) sum = fmaf(element<BF16, e>(d), v_row[j + e], sum);
                });
            }
            const float b = D.a.base ? D.a.base[t.row * D.a.ldb + n] : 0.0f;
            D.a.y[t.row * D.a.ldy + n] = fmaf(scale, sum, b);
        }
        return;
    }
    // v of row i, ranks 16 r + 4 g ..
    const int tiles = (t.rank + 15) / 16;
    f32x4 v[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        v[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int j = 16 * r + 4 * g;
        if (r >= tiles || j >= D.l.max_rank) continue;
        for (int s = 0; s < D.k_shares; ++s)
            v[r] += *reinterpret_cast<const f32x4*>(part + s * share + static_cast<int64_t>(min(i, t.rows - 1)) * D.l.max_rank + j);
    }
    constexpr int kU = RT <= 2 ? 4 : 2;  // tiles of outputs at a time
    for (int64_t n0 = lo + wave * (kU * 16); n0 < hi; n0 += kWaves * kU * 16) {
        f32x4 acc[kU] = {};
        uint2 w[kU][RT];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t n = min(n0 + 16 * u + i, D.l.N - 1);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int j = 16 * r + 4 * g;
                w[u][r] = make_uint2(0u, 0u);
                if (r < tiles && j < t.rank) w[u][r] = *reinterpret_cast<const uint2*>(Bm + n * D.l.max_rank + j);
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if (r >= tiles) continue;
            const int left = t.rank - (16 * r + 4 * g);  // ranks of this lane that count
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                uint32_t d[2] = {w[u][r].x, w[u][r].y};
                if (left < 4) {  // what lies behind the rank may be anything
                    d[1] = left < 3 ? 0u : d[1] & 0xffffu;
                    d[0] = left < 1 ? 0u : (left < 2 ? d[0] & 0xffffu : d[0]);
                }
                static_for<4>([&](auto e) {
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(element<BF16, e>(d), v[r][decltype(e)::value], acc[u], 0, 0, 0);
                });
            }
        }
        if (i < t.rows) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int64_t n = n0 + 16 * u + 4 * g;
                if (n < D.l.N) update4(D, t.row + i, n, acc[u] * scale);
            }
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
