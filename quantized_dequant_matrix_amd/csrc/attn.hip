// Attention of new tokens over the paged cache.
//
//   s_j = scale q . k_j over the visible positions j,
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s)
//
// One pass over keys and values with the running maximum and sum of the
// softmax.  For few rows the cache's bytes bound it, for a chunk of many rows
// the matrix instructions and the conversions that feed them.
//
// Rows.  The query heads of one key/value head and the new tokens of one
// sequence are the rows of one matrix: row rho = i G + g is token i, head
// h G + g.  A workgroup takes 16 R of them (an "item": sequence, row tile,
// key/value head) and its four waves share the item's keys, 32 at a time.
//
// Matrix instructions, with nothing moved between lanes from load to result:
//   S^T = K Q^T   A = 16 keys, B = 16 rows.  Lane (n = lane % 16, g = lane /
//     16) of the result holds row n and keys 4 g .. 4 g + 3 of the 16.
//   O^T = V^T P^T  contraction over 32 keys.  The order of a contraction is
//     free as long as both operands agree, so it is taken as the keys lie in
//     the results of two S^T tiles: lane (n, g) already holds its operand,
//     P of row n at keys {4 g + e, 16 + 4 g + e}.  The other operand needs,
//     for each dimension, those eight keys in one lane: lane (m, g) loads
//     D / 16 consecutive elements of each of the eight keys, and
//     instruction t takes element t of all eight (byte permutes inside the
//     lane), which makes result row m the dimension m D / 16 + t.
//
// Accuracy.  The operands of the matrix instructions are narrower than
// float32, so a float32 value enters as several terms whose products are
// exact and summed in float32 (int32):
//   8-bit keys: q is held to 21 bits of the row's largest magnitude as three
//     signed 7-bit parts, against the int8 codes as they are
//     (v_mfma_i32_16x16x64_i8, no conversion of K at all); the key's scale
//     multiplies the finished score.
//   float16 keys: q as two float16 terms (22 bits).
//   p: two float16 terms.  The scale of a value row is multiplied into p
//     before the split, relative to a power of two near the largest scale
//     the row has seen (float16 has too few exponents for it otherwise).
//     8-bit codes become float16 exactly: a byte u = code + 128 read as a
//     float16 is u 2^-24, and one fused multiply-add makes it
//     (u - 128) 2^-9.
//
// Split.  The work is cut into units (128 keys of an item) and the units are
// dealt in equal runs to the workgroups of one round, whatever the lengths of
// the sequences: every workgroup finds its run from the batch's arrays by
// itself.  A run covers pieces of items; a piece that is a whole item is
// written as it is, the first and the last piece of a run may be parts, go to
// the workspace (two slots a workgroup) and are joined by a second kernel in
// a fixed order.  Where there are more items than two rounds of workgroups a
// unit is a whole item and there is no second kernel.
#include <stdint.h>

#include "kv_device.h"
#include "qmv_internal.h"
#include "step_internal.h"

namespace qmv {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_inff();
constexpr int kTile = 32;                        // keys of one wave's step
constexpr int kStep = kTile * kWavesPerBlock;    // keys of the workgroup's step
constexpr int kUnit = kStep;                     // keys of one unit of work
constexpr float kQParts = 127.0f * 16384.0f;     // largest |q| in parts: 127 2^14
constexpr float kSlack = 3.0f;                   // p may reach 2^3 before the maximum moves

struct AttnArgs {
    KvView view;
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    const float* q;
    float* out;
    float* part;       // partial results, slot(w, s) = part + (2 w + s) * slot size
    int64_t ldq, ldo;
    int group;         // query heads of a key/value head
    float scale_log2;  // |scale| log2(e)
    float sign;        // of scale
    int window;
    int unit;          // keys of one unit
    int workgroups;    // of one round (a run each)
    bool vec_q, vec_o;
};

// What the batch's arrays say about a sequence, made safe.
struct Seq {
    int first, n;   // rows first .. first + n - 1
    int base;       // position of its first row
    int lo, hi;     // positions that any row may see (lo a multiple of 32)
    int tiles;      // row tiles
    int units;      // of one row tile and head
};

template <int ROWS>
__device__ __forceinline__ Seq sequence(const AttnArgs& A, int b) {
    Seq s;
    s.first = A.view.row_start[b];
    const int end = A.view.row_start[b + 1];
    s.n = (s.first >= 0 && end <= A.view.T && end > s.first) ? end - s.first : 0;
    const int len = max(A.view.kv_len[b], 0);
    const int top = A.view.max_pages << A.view.page_shift;
    s.base = len - s.n;
    s.hi = min(len, top);
    const int64_t lo = A.window > 0 ? static_cast<int64_t>(s.base) - A.window + 1 : 0;
    s.lo = lo > 0 ? static_cast<int>(lo) & ~(kTile - 1) : 0;
    s.tiles = (s.n * A.group + ROWS - 1) / ROWS;
    // an item whose rows see nothing is one empty unit: its zeros are written
    s.units = s.hi > s.lo ? (s.hi - s.lo - 1) / A.unit + 1 : 1;
    return s;
}

struct Place {
    int b;
    int64_t units_before;  // units of all sequences before b
    int tiles_before;
    int64_t total;         // units of the batch
};

// Finds the sequence that holds unit `key` (of the batch's units in order of
// sequence, row tile, head, position), or, with BY_TILE, row tile `key`.
// All 256 threads; B sequences, 256 at a time.  b = B if there is none.
template <int ROWS, bool BY_TILE>
__device__ Place locate(const AttnArgs& A, int64_t key, bool by_share, int64_t* lds /* 12 */) {
    const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
    const int heads = A.view.heads;
    int64_t* sums = lds;       // [4]: units of the waves' sequences
    int64_t* tsum = lds + 4;   // [4]: row tiles
    int64_t* found = lds + 8;  // b, units before, tiles before
    const bool one = A.view.B <= kBlockThreads;
    int64_t u = 0, c = 0;
    Place P;
    P.total = 0;
    if (t == 0) found[0] = A.view.B;
    for (int b0 = 0; b0 < A.view.B; b0 += kBlockThreads) {
        u = c = 0;
        if (b0 + t < A.view.B) {
            const Seq s = sequence<ROWS>(A, b0 + t);
            c = s.tiles;
            u = static_cast<int64_t>(s.tiles) * heads * s.units;
        }
        if (one) break;
        int64_t w = u;
        for (int o = kWave / 2; o > 0; o >>= 1) w += __shfl_xor(w, o, kWave);
        __syncthreads();
        if (lane == 0) sums[wave] = w;
        __syncthreads();
        P.total += sums[0] + sums[1] + sums[2] + sums[3];
    }
    int64_t base_u = 0, base_c = 0;
    for (int b0 = 0; b0 < A.view.B; b0 += kBlockThreads) {
        if (!one) {
            u = c = 0;
            if (b0 + t < A.view.B) {
                const Seq s = sequence<ROWS>(A, b0 + t);
                c = s.tiles;
                u = static_cast<int64_t>(s.tiles) * heads * s.units;
            }
        }
        int64_t iu = u, ic = c;
        for (int o = 1; o < kWave; o <<= 1) {
            const int64_t xu = __shfl_up(iu, o, kWave), xc = __shfl_up(ic, o, kWave);
            if (lane >= o) {
                iu += xu;
                ic += xc;
            }
        }
        __syncthreads();
        if (lane == kWave - 1) {
            sums[wave] = iu;
            tsum[wave] = ic;
        }
        __syncthreads();
        int64_t strip = 0, strip_c = 0, before = base_u, before_c = base_c;
        for (int w = 0; w < kWavesPerBlock; ++w) {
            if (w < wave) {
                before += sums[w];
                before_c += tsum[w];
            }
            strip += sums[w];
            strip_c += tsum[w];
        }
        if (one) P.total = strip;
        if (by_share && b0 == 0) {
            // the first unit of workgroup `key`'s run, of min(workgroups, total) runs
            const int64_t W = P.total < A.workgroups ? P.total : A.workgroups;
            key = key < W ? key * P.total / W : P.total;
        }
        const int64_t end = BY_TILE ? before_c + ic : before + iu;
        const int64_t begin = end - (BY_TILE ? c : u);
        if (key >= begin && key < end) {
            found[0] = b0 + t;
            found[1] = before + iu - u;
            found[2] = before_c + ic - c;
        }
        base_u += strip;
        base_c += strip_c;
    }
    __syncthreads();
    P.b = static_cast<int>(found[0]);
    P.units_before = P.b < A.view.B ? found[1] : 0;
    P.tiles_before = P.b < A.view.B ? static_cast<int>(found[2]) : 0;
    return P;
}

__device__ __forceinline__ float xor16_max(float v) { return fmaxf(v, __shfl_xor(v, 16, kWave)); }
__device__ __forceinline__ float xor32_max(float v) { return fmaxf(v, __shfl_xor(v, 32, kWave)); }
// over the four lanes that hold one row
__device__ __forceinline__ float row_max(float v) { return xor32_max(xor16_max(v)); }
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

__device__ __forceinline__ uint32_t pk(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
}

template <int D, bool F16>
struct KvRegs {
    static constexpr int kE = F16 ? 2 : 1;        // bytes of an element
    static constexpr int kKLoads = D * kE / 64;   // 16-byte pieces of a key that a lane holds
    static constexpr int kVWords = D * kE / 64;   // dwords of a value row that a lane holds
    u32x4 k[2][kKLoads];
    uint32_t v[8][kVWords];
    f32x4 ks[2], vs[2];
};

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&r)[WORDS], const uint8_t* p) {
    if constexpr (WORDS == 1) {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (WORDS == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        r[0] = x.x;
        r[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const u32x4 x = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) r[4 * i + e] = x[e];
        }
    }
}

// The two 16-key halves of a tile: the pages they lie in.
struct Pages {
    int64_t cell[2];  // index of the half's first row in the planes
    bool ok[2];       // the half has a page
};

__device__ __forceinline__ Pages pages_of(const AttnArgs& A, int b, int h, int key) {
    Pages p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pos = key + 16 * i;
        const int j = pos >> A.view.page_shift;
        int page = -1;
        if (j < A.view.max_pages) page = A.view.table[static_cast<int64_t>(b) * A.view.max_pages + j];
        p.ok[i] = page >= 0 && page < A.view.num_pages;
        page = p.ok[i] ? page : 0;  // read but not seen
        p.cell[i] = ((static_cast<int64_t>(page) * A.view.heads + h) << A.view.page_shift) +
                    (pos & ((1 << A.view.page_shift) - 1));
    }
    return p;
}

template <int D, bool F16>
__device__ __forceinline__ void load_tile(const AttnArgs& A, const Pages& p, KvRegs<D, F16>& r) {
    using T = KvRegs<D, F16>;
    constexpr int kRow = D * T::kE;  // bytes of a key
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint8_t* kp = A.k + p.cell[u] * kRow + (n * kRow + g * 16);
#pragma unroll
        for (int s = 0; s < T::kKLoads; ++s) r.k[u][s] = *reinterpret_cast<const u32x4*>(kp + 64 * s);
        if constexpr (!F16) {
            r.ks[u] = *reinterpret_cast<const f32x4*>(A.ks + p.cell[u] + 4 * g);
            r.vs[u] = *reinterpret_cast<const f32x4*>(A.vs + p.cell[u] + 4 * g);
        }
        const uint8_t* vp = A.v + p.cell[u] * kRow + (4 * g * kRow + n * (kRow / 16));
#pragma unroll
        for (int e = 0; e < 4; ++e) load_words(r.v[4 * u + e], vp + e * kRow);
    }
}

// The rows of a workgroup as each wave holds them.
template <int D, bool F16, int R>
struct Rows {
    static constexpr int kQ = F16 ? D / 32 : D / 64;  // instructions of one term over D
    static constexpr int kTerms = F16 ? 2 : 3;
    u32x4 q[R][kTerms][kQ];
    float qs[R];   // score in log2 units = qs * (integer or float16 score) [* key scale]
    int pos[R];    // position of the lane's row, -1 for a row past the item's
    f32x4 o[R][D / 16];
    float m[R];    // running maximum, before qs
    float l[R];    // this lane's share of the sum
    float c[R];    // 8-bit values: factor of the value scales
    float lim[R];  // ... and the largest scale it is good for
};

// q of row rho: 16 (8 for float16) dimensions at a time as the lane's B
// operand takes them: dimension 64 s + 16 g + byte (32 s + 8 g + e).
template <int D, bool F16, int R>
__device__ __forceinline__ void load_rows(const AttnArgs& A, const Seq& S, int tile, int h, Rows<D, F16, R>& W) {
    using T = Rows<D, F16, R>;
    constexpr int kPer = F16 ? 8 : 16;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int rho = (tile * R + r) * 16 + n;
        const bool real = rho < S.n * A.group;
        const int i = real ? rho / A.group : 0;
        const int head = h * A.group + (real ? rho - i * A.group : 0);
        W.pos[r] = real ? S.base + i : -1;
        const float* src = A.q + static_cast<int64_t>(S.first + i) * A.ldq + static_cast<int64_t>(head) * D;
        float x[T::kQ][kPer];
        float amax = 0.0f;
        bool broken = false;
#pragma unroll
        for (int s = 0; s < T::kQ; ++s) {
            const float* p = src + s * (4 * kPer) + g * kPer;
            if (A.vec_q) {
#pragma unroll
                for (int e = 0; e < kPer; e += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(p + e);
                    x[s][e] = f.x; x[s][e + 1] = f.y; x[s][e + 2] = f.z; x[s][e + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e) x[s][e] = p[e];
            }
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (!real) x[s][e] = 0.0f;
                amax = fmaxf(amax, fabsf(x[s][e]));
                broken |= !(fabsf(x[s][e]) < kInf);
            }
        }
        amax = row_max(amax);
        // whole row scaled by a power of two first: amax in [1/2, 1)
        int k = 0;
        if (amax > 0.0f && amax < kInf) k = __builtin_amdgcn_frexp_expf(amax);
        const float an = __builtin_amdgcn_ldexpf(amax, -k);
        float inv, back;
        if constexpr (F16) {
            inv = 1024.0f;
            back = 1.0f / 1024.0f;
        } else {
            inv = an > 0.0f ? kQParts / an : 0.0f;
            back = an * (1.0f / kQParts);
        }
        W.qs[r] = __builtin_amdgcn_ldexpf(back * A.scale_log2, k);
        broken = row_max(broken ? 1.0f : 0.0f) != 0.0f;
        if (broken) W.qs[r] = __uint_as_float(0x7fc00000u);
        inv *= A.sign;
#pragma unroll
        for (int s = 0; s < T::kQ; ++s) {
            if constexpr (F16) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float a = __builtin_amdgcn_ldexpf(x[s][e], -k) * inv;
                    const float b = __builtin_amdgcn_ldexpf(x[s][e + 1], -k) * inv;
                    const f16x2 f = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
                    hi[e / 2] = __builtin_bit_cast(uint32_t, f);
                    const f16x2 d = {static_cast<_Float16>(a - static_cast<float>(f[0])),
                                     static_cast<_Float16>(b - static_cast<float>(f[1]))};
                    lo[e / 2] = __builtin_bit_cast(uint32_t, d);
                }
                W.q[r][0][s] = u32x4{hi[0], hi[1], hi[2], hi[3]};
                W.q[r][1][s] = u32x4{lo[0], lo[1], lo[2], lo[3]};
            } else {
                u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0}, c = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    // x = a 2^14 + b 2^7 + c, b and c in [-64, 63]
                    const int v = static_cast<int>(rintf(__builtin_amdgcn_ldexpf(x[s][e], -k) * inv));
                    const int vc = ((v + 64) & 127) - 64;
                    const int v1 = (v - vc) >> 7;
                    const int vb = ((v1 + 64) & 127) - 64;
                    const int va = (v1 - vb) >> 7;
                    a[e / 4] |= (static_cast<uint32_t>(va) & 0xffu) << (8 * (e % 4));
                    b[e / 4] |= (static_cast<uint32_t>(vb) & 0xffu) << (8 * (e % 4));
                    c[e / 4] |= (static_cast<uint32_t>(vc) & 0xffu) << (8 * (e % 4));
                }
                W.q[r][0][s] = a;
                W.q[r][1][s] = b;
                W.q[r][2][s] = c;
            }
        }
        W.m[r] = -kInf;
        W.l[r] = 0.0f;
        W.c[r] = 1.0f;
        W.lim[r] = 0.0f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) W.o[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

// One tile of 32 keys, at positions key ..; MASK: some row does not see some
// key of it (or a half has no page).
template <bool MASK, int D, bool F16, int R>
__device__ __forceinline__ void tile_step(const AttnArgs& A, KvRegs<D, F16>& kv, Rows<D, F16, R>& W, int key,
                                          bool ok0, bool ok1, int hi_any, int lo_any) {
    using T = Rows<D, F16, R>;
    using V = KvRegs<D, F16>;
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4;

    // float16 values at positions no row sees may be anything: zero times
    // them has to be zero.  At positions that only some rows see, a value
    // that is not finite is taken out and makes those rows NaN by their sum.
    uint32_t broken = 0;
    if constexpr (MASK && F16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = key + 16 * (e >> 2) + 4 * g + (e & 3);
            const bool any = (e < 4 ? ok0 : ok1) && j < hi_any && j >= lo_any;
            bool bad = false;
#pragma unroll
            for (int w = 0; w < V::kVWords; ++w) {
                const uint32_t x = kv.v[e][w];
                bad |= (x & 0x7c00u) == 0x7c00u || (x & 0x7c000000u) == 0x7c000000u;
            }
            const uint64_t where = __ballot(bad && any);
            const bool out = ((where >> (16 * g)) & 0xffffu) != 0;
            if (out) broken |= 1u << e;
#pragma unroll
            for (int w = 0; w < V::kVWords; ++w) kv.v[e][w] = (any && !out) ? kv.v[e][w] : 0u;
        }
    }

    uint32_t ph[R][4], pl[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float s[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (F16) {
                f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < T::kQ; ++i)
#pragma unroll
                    for (int term = 1; term >= 0; --term)
                        a = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, kv.k[u][i]),
                                                                   __builtin_bit_cast(f16x8, W.q[r][term][i]), a, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[4 * u + e] = a[e];
            } else {
                i32x4 a[3] = {};
#pragma unroll
                for (int i = 0; i < T::kQ; ++i)
#pragma unroll
                    for (int term = 0; term < 3; ++term)
                        a[term] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, kv.k[u][i]),
                                                                        __builtin_bit_cast(i32x4, W.q[r][term][i]), a[term],
                                                                        0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[4 * u + e] = fmaf(static_cast<float>(a[0][e]), 16384.0f,
                                        static_cast<float>((a[1][e] << 7) + a[2][e])) * kv.ks[u][e];
            }
        }
        bool seen[8];
        float top = -kInf, big = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (MASK) {
                const int j = key + 16 * (e >> 2) + 4 * g + (e & 3);
                seen[e] = (e < 4 ? ok0 : ok1) && j <= W.pos[r] && j < hi_any &&
                          (A.window == 0 || j - W.pos[r] > -A.window);
                s[e] = seen[e] ? s[e] : -kInf;
                if constexpr (!F16) big = fmaxf(big, seen[e] ? kv.vs[e >> 2][e & 3] : 0.0f);
            } else {
                seen[e] = true;
                if constexpr (!F16) big = fmaxf(big, kv.vs[e >> 2][e & 3]);
            }
            top = fmaxf(top, s[e]);
        }
        // The maximum and the factor of the value scales move only when a
        // row has outgrown them: p and its products stay within float16.
        const bool grow = (top - W.m[r]) * W.qs[r] > kSlack || (W.m[r] == -kInf && top > -kInf) || big > W.lim[r];
        if (__ballot(grow) != 0) {
            top = row_max(top);
            const float mn = fmaxf(W.m[r], top);
            const float alpha = W.m[r] == -kInf ? 0.0f : __builtin_amdgcn_exp2f((W.m[r] - mn) * W.qs[r]);
            float f = alpha;
            if constexpr (!F16) {
                big = row_max(big);
                if (big > W.lim[r]) {
                    // c = 2^10 / 2^floor(log2 big); good up to four times that power
                    const int e = static_cast<int>(__float_as_uint(big) >> 23);
                    const int ce = min(max(264 - e, 1), 254);
                    const float c = __uint_as_float(static_cast<uint32_t>(ce) << 23);
                    f *= W.lim[r] == 0.0f ? 1.0f : c / W.c[r];
                    W.c[r] = c;
                    W.lim[r] = __uint_as_float(static_cast<uint32_t>(min(max(e, 1) + 2, 254)) << 23);
                }
            }
            W.m[r] = mn;
            W.l[r] *= alpha;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) W.o[r][t] *= f;
        }
        const float mq = W.m[r] == -kInf ? 0.0f : W.m[r] * W.qs[r];
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], W.qs[r], -mq));
            if constexpr (MASK) p[e] = seen[e] ? p[e] : 0.0f;
            W.l[r] += p[e];
            if constexpr (MASK && F16)
                if (seen[e] && (broken >> e & 1)) W.l[r] = __uint_as_float(0x7fc00000u);
            if constexpr (F16) {
                p[e] *= 1024.0f;
            } else {
                p[e] *= kv.vs[e >> 2][e & 3] * W.c[r];
                if constexpr (MASK) p[e] = seen[e] ? p[e] : 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ph[r][e] = pk(p[2 * e], p[2 * e + 1]);
            const f16x2 h = __builtin_bit_cast(f16x2, ph[r][e]);
            pl[r][e] = pk(p[2 * e] - static_cast<float>(h[0]), p[2 * e + 1] - static_cast<float>(h[1]));
        }
    }

#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
        uint32_t a[4];
        if constexpr (F16) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                a[e] = __builtin_amdgcn_perm(kv.v[2 * e + 1][t / 2], kv.v[2 * e][t / 2], t % 2 ? 0x07060302u : 0x05040100u);
        } else {
            const uint32_t sel = 0x0c000c00u | static_cast<uint32_t>(t % 4) | (static_cast<uint32_t>(4 + t % 4) << 16);
            const f16x2 mul = {static_cast<_Float16>(32768.0f), static_cast<_Float16>(32768.0f)};
            const f16x2 add = {static_cast<_Float16>(-0.25f), static_cast<_Float16>(-0.25f)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = __builtin_amdgcn_perm(kv.v[2 * e + 1][t / 4] ^ 0x80808080u,
                                                         kv.v[2 * e][t / 4] ^ 0x80808080u, sel);
                a[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, x), mul, add));
            }
        }
        const f16x8 va = __builtin_bit_cast(f16x8, u32x4{a[0], a[1], a[2], a[3]});
#pragma unroll
        for (int r = 0; r < R; ++r) {
            W.o[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                va, __builtin_bit_cast(f16x8, u32x4{ph[r][0], ph[r][1], ph[r][2], ph[r][3]}), W.o[r][t], 0, 0, 0);
            W.o[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                va, __builtin_bit_cast(f16x8, u32x4{pl[r][0], pl[r][1], pl[r][2], pl[r][3]}), W.o[r][t], 0, 0, 0);
        }
    }
}

// Floats of one partial slot: 16 R rows of D sums, then their maxima, then sums.
template <int D, int R>
constexpr int kSlotFloats = 16 * R * (D + 2);

template <int D, bool F16, int R>
__global__ __launch_bounds__(kBlockThreads)
void attn_kernel(AttnArgs A) {
    constexpr int kRows = 16 * R;
    constexpr int kPad = D + 4;
    __shared__ __align__(16) float so[kWavesPerBlock * 16 * kPad];
    __shared__ float sm[kWavesPerBlock][kRows], sl[kWavesPerBlock][kRows];
    __shared__ int64_t place[12];
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int w = blockIdx.x;
    const Place P = locate<kRows, false>(A, w, true, place);
    if (P.b >= A.view.B) return;  // no run
    const int64_t W64 = P.total < A.workgroups ? P.total : A.workgroups;
    int64_t u = static_cast<int64_t>(w) * P.total / W64;
    const int64_t u_end = (static_cast<int64_t>(w) + 1) * P.total / W64;
    int b = __builtin_amdgcn_readfirstlane(P.b);
    int64_t before = P.units_before;
    Seq S = sequence<kRows>(A, b);
    bool first_piece = true;
    while (u < u_end) {
        // the piece: an item's units from u on, as far as the run goes
        while (u - before >= static_cast<int64_t>(S.tiles) * A.view.heads * S.units) {
            before += static_cast<int64_t>(S.tiles) * A.view.heads * S.units;
            S = sequence<kRows>(A, ++b);
        }
        const int64_t local = u - before;
        const int item = static_cast<int>(local / S.units);
        const int c0 = static_cast<int>(local - static_cast<int64_t>(item) * S.units);
        const int64_t left = u_end - u;
        const int c1 = static_cast<int>(left < S.units - c0 ? c0 + left : S.units);
        const int h = item % A.view.heads, tile = item / A.view.heads;
        u += c1 - c0;

        Rows<D, F16, R> rows;
        load_rows<D, F16, R>(A, S, tile, h, rows);

        // positions of the item's rows: tokens i0 .. i1
        const int i0 = tile * kRows / A.group;
        const int i1 = (min((tile + 1) * kRows, S.n * A.group) - 1) / A.group;
        const int p0 = S.base + i0, p1 = S.base + i1;
        const int hi_any = min(p1 + 1, S.hi);                           // keys that some row sees: below this
        const int hi_all = min(p0 + 1, S.hi);                           // that every row sees: below this
        int lo_any = 0, lo_all = 0;                                     // ... and from these on
        if (A.window > 0) {
            lo_any = static_cast<int>(max(static_cast<int64_t>(p0) - A.window + 1, int64_t{0}));
            lo_all = static_cast<int>(max(static_cast<int64_t>(p1) - A.window + 1, int64_t{0}));
        }
        int64_t k1 = S.lo + static_cast<int64_t>(c1) * A.unit;
        k1 = k1 < hi_any ? k1 : hi_any;
        int64_t k0 = S.lo + static_cast<int64_t>(c0) * A.unit;
        const int64_t low = lo_any & ~(kTile - 1);
        k0 = k0 > low ? k0 : low;
        const int end = static_cast<int>(k1 > 0 ? k1 : 0);
        int key = static_cast<int>(k0 < end ? k0 : end) + wave * kTile;
        if (key < end) {
            KvRegs<D, F16> cur, nxt;
            Pages pg = pages_of(A, b, h, key), pn;
            load_tile<D, F16>(A, pg, cur);
            pn = pages_of(A, b, h, min(key + kStep, end - 1) & ~(kTile - 1));
            for (;;) {
                const bool more = end - key > kStep;
                if (more) load_tile<D, F16>(A, pn, nxt);
                const Pages pt = pages_of(A, b, h, end - key > 2 * kStep ? key + 2 * kStep : key);
                if (pg.ok[0] && pg.ok[1] && key + kTile <= hi_all && key >= lo_all)
                    tile_step<false, D, F16, R>(A, cur, rows, key, true, true, hi_any, lo_any);
                else
                    tile_step<true, D, F16, R>(A, cur, rows, key, pg.ok[0], pg.ok[1], hi_any, lo_any);
                if (!more) break;
                key += kStep;
                cur = nxt;
                pg = pn;
                pn = pt;
            }
        }

        // join the four waves, 16 rows at a time
        float mq[R], ls[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mq[r] = rows.m[r] == -kInf ? -kInf : rows.m[r] * rows.qs[r];
            ls[r] = row_sum(rows.l[r]);
            if (g == 0) {
                sm[wave][16 * r + n] = mq[r];
                sl[wave][16 * r + n] = ls[r];
            }
        }
        const bool whole = c0 == 0 && c1 == S.units;
        float* slot = A.part + (2 * static_cast<int64_t>(w) + (first_piece ? 0 : 1)) * kSlotFloats<D, R>;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            __syncthreads();
            float M = -kInf;
#pragma unroll
            for (int i = 0; i < kWavesPerBlock; ++i) M = fmaxf(M, sm[i][16 * r + n]);
            const float f = __builtin_amdgcn_exp2f(mq[r] - (M == -kInf ? 0.0f : M)) *
                            (F16 ? 1.0f / 1024.0f : 512.0f / rows.c[r]);
            float* dst = so + (wave * 16 + n) * kPad + 4 * g * (D / 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int t = 0; t < D / 16; t += 4)
                    *reinterpret_cast<f32x4*>(dst + e * (D / 16) + t) =
                        f32x4{rows.o[r][t][e], rows.o[r][t + 1][e], rows.o[r][t + 2][e], rows.o[r][t + 3][e]} * f;
            __syncthreads();
            for (int x = threadIdx.x; x < 16 * (D / 4); x += kBlockThreads) {
                const int row = x / (D / 4), d = x % (D / 4) * 4;
                const int rho = (tile * R + r) * 16 + row;
                if (rho >= S.n * A.group) continue;
                f32x4 v = *reinterpret_cast<const f32x4*>(so + row * kPad + d);
#pragma unroll
                for (int i = 1; i < kWavesPerBlock; ++i)
                    v += *reinterpret_cast<const f32x4*>(so + (i * 16 + row) * kPad + d);
                float Mr = -kInf, L = 0.0f;
#pragma unroll
                for (int i = 0; i < kWavesPerBlock; ++i) Mr = fmaxf(Mr, sm[i][16 * r + row]);
#pragma unroll
                for (int i = 0; i < kWavesPerBlock; ++i)
                    L += sl[i][16 * r + row] * __builtin_amdgcn_exp2f(sm[i][16 * r + row] - (Mr == -kInf ? 0.0f : Mr));
                if (whole) {
                    v = L == 0.0f ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : v / L;
                    const int i = rho / A.group;
                    float* o = A.out + static_cast<int64_t>(S.first + i) * A.ldo +
                               static_cast<int64_t>(h * A.group + rho - i * A.group) * D + d;
                    if (A.vec_o) {
                        *reinterpret_cast<f32x4*>(o) = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = v[e];
                    }
                } else {
                    *reinterpret_cast<f32x4*>(slot + (16 * r + row) * D + d) = v;
                    if (d == 0) {
                        slot[kRows * D + 16 * r + row] = Mr;
                        slot[kRows * D + kRows + 16 * r + row] = L;
                    }
                }
            }
        }
        __syncthreads();
        first_piece = false;
    }
}

// Joins the parts of every item that more than one workgroup worked on: one
// workgroup a (row tile, head), slots in order of position.
template <int D, int R>
__global__ __launch_bounds__(kBlockThreads)
void attn_join_kernel(AttnArgs A) {
    constexpr int kRows = 16 * R;
    __shared__ int64_t place[12];
    const int h = blockIdx.x % A.view.heads, tile_all = blockIdx.x / A.view.heads;
    const Place P = locate<kRows, true>(A, tile_all, false, place);
    if (P.b >= A.view.B) return;
    const Seq S = sequence<kRows>(A, P.b);
    const int tile = tile_all - P.tiles_before;
    const int64_t W = P.total < A.workgroups ? P.total : A.workgroups;
    const int64_t ua = P.units_before + (static_cast<int64_t>(tile) * A.view.heads + h) * S.units;
    const int64_t ub = ua + S.units;
    // owner of unit u: the largest w with floor(w total / W) <= u
    const int64_t w0 = ((ua + 1) * W - 1) / P.total, w1 = (ub * W - 1) / P.total;
    if (w0 == w1) return;
    const int rows = min(kRows, S.n * A.group - tile * kRows);
    for (int x = threadIdx.x; x < rows * (D / 4); x += kBlockThreads) {
        const int row = x / (D / 4), d = x % (D / 4) * 4;
        float M = -kInf;
        for (int64_t w = w0; w <= w1; ++w) {
            const float* slot = A.part + (2 * w + (w * P.total / W >= ua ? 0 : 1)) * kSlotFloats<D, R>;
            M = fmaxf(M, slot[kRows * D + row]);
        }
        if (M == -kInf) M = 0.0f;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        float L = 0.0f;
        for (int64_t w = w0; w <= w1; ++w) {
            const float* slot = A.part + (2 * w + (w * P.total / W >= ua ? 0 : 1)) * kSlotFloats<D, R>;
            const float f = __builtin_amdgcn_exp2f(slot[kRows * D + row] - M);
            L += slot[kRows * D + kRows + row] * f;
            v += *reinterpret_cast<const f32x4*>(slot + row * D + d) * f;
        }
        v = L == 0.0f ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : v / L;
        const int rho = tile * kRows + row, i = rho / A.group;
        float* o = A.out + static_cast<int64_t>(S.first + i) * A.ldo +
                   static_cast<int64_t>(h * A.group + rho - i * A.group) * D + d;
        if (A.vec_o) {
            *reinterpret_cast<f32x4*>(o) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = v[e];
        }
    }
}

// Everything about a call that depends on the descriptors' numbers.
struct AttnPlan {
    int r = 1;             // 16-row tiles of a workgroup
    int64_t tiles = 0;     // at most this many row tiles in the batch
    int workgroups = 0;
    bool split = true;     // units of 128 keys and a second kernel; else whole items
};

constexpr int kRound = 512;  // workgroups of one round: two on each of 256 CUs

AttnPlan plan_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, int q_heads) {
    AttnPlan p;
    const int64_t group = q_heads / c.kv_heads;
    p.r = 1;
    const int64_t rows = 16 * p.r;
    // sum over sequences of ceil(n group / rows), for any split of T rows
    const int64_t seqs = b.B < b.T ? b.B : b.T;
    const int64_t x = b.T * ((group + rows - 1) / rows), y = (b.T * group + seqs * (rows - 1)) / rows;
    p.tiles = x < y ? x : y;
    const int64_t items = p.tiles * c.kv_heads;
    p.split = items < 2 * kRound;
    p.workgroups = p.split ? kRound : static_cast<int>(items < (1 << 24) - 1 ? items : (1 << 24) - 1);
    return p;
}

}  // namespace

size_t attn_ws_bytes(const qmv_kv_cache& c, const qmv_kv_batch& b, int q_heads) {
    const AttnPlan p = plan_attn(c, b, q_heads);
    if (!p.split) return 256;
    return static_cast<size_t>(2 * p.workgroups) * static_cast<size_t>(16 * p.r * (c.head_dim + 2)) * sizeof(float);
}

hipError_t launch_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* q, int64_t ldq, float* out,
                       int64_t ldo, int q_heads, float scale, int window, void* ws, hipStream_t stream) {
    const AttnPlan p = plan_attn(c, b, q_heads);
    AttnArgs A;
    A.view = view_of(c, b);
    A.k = static_cast<const uint8_t*>(c.k);
    A.v = static_cast<const uint8_t*>(c.v);
    A.ks = c.k_scale;
    A.vs = c.v_scale;
    A.q = q;
    A.out = out;
    A.part = static_cast<float*>(ws);
    A.ldq = ldq;
    A.ldo = ldo;
    A.group = q_heads / c.kv_heads;
    A.scale_log2 = (scale < 0.0f ? -scale : scale) * kLog2e;
    A.sign = scale < 0.0f ? -1.0f : 1.0f;
    A.window = window;
    A.unit = p.split ? kUnit : INT32_MAX;
    A.workgroups = p.workgroups;
    A.vec_q = (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ldq % 4 == 0;
    A.vec_o = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ldo % 4 == 0;
    const dim3 grid(static_cast<unsigned>(p.workgroups)), join(static_cast<unsigned>(p.tiles * c.kv_heads));
#define ATTN(D, F16, R)                                                                                     \
    do {                                                                                                    \
        hipLaunchKernelGGL((attn_kernel<D, F16, R>), grid, dim3(kBlockThreads), 0, stream, A);              \
        if (p.split) hipLaunchKernelGGL((attn_join_kernel<D, R>), join, dim3(kBlockThreads), 0, stream, A); \
    } while (0)
    if (c.format == QMV_KV_F16) {
        if (c.head_dim == 64) ATTN(64, true, 1);
        else if (c.head_dim == 128) ATTN(128, true, 1);
        else ATTN(256, true, 1);
    } else {
        if (c.head_dim == 64) ATTN(64, false, 1);
        else if (c.head_dim == 128) ATTN(128, false, 1);
        else ATTN(256, false, 1);
    }
    return hipGetLastError();
}

}  // namespace qmv
