// Attention of new tokens over the paged cache.
//
//   s_j = scale q . k_j over the visible positions j,
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s)
//
// One pass over keys and values with a running reference and sum of the
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
//   p: two float16 terms, the scale of a value row multiplied in before the
//     split.  float16 has few exponents, so what is split is p dv 2^-c with a
//     reference c of the row's own, a whole number: where c moves, the
//     largest p dv comes to lie in [2^9, 2^11), and it may grow to 2^15
//     before c moves again.  The second term is rounded to half a step of
//     2^-24, 2^-34 of the largest product of a weight and a value's scale: a
//     large value that weighs nothing takes nothing from the others.
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
// a fixed order.  Short tables, many items and chunks of many rows are computed
// an item a workgroup instead, without a second kernel (plan_attn says where).
#include <cmath>
#include <stdint.h>

#include "attn_plan.h"
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
static_assert(kAttnWaves == kWavesPerBlock && kWaveThreads == kWave && kOwnerBytes == sizeof(int4));
constexpr float kQParts = 127.0f * 16384.0f;     // largest |q| in parts: 127 2^14 (its digits: 127, 0, 0)
// Weights are exp2(score - c), c the row's reference (tile_step):
constexpr float kTop = 9.0f;                     // log2 of the largest p dv where c is set, rounded down
constexpr float kTopMax = 15.0f;                 // ... and without a move: float16 holds it
constexpr float kPTop = 80.0f, kPMax = 90.0f;    // the same of p itself (values of zero would ask for any)
// Value scales are taken times 2^16, which brings ordinary ones (2^-7) near
// kTop.  So the exponent that makes a weight which counts is near 0: at 16 its
// rounding to float32 alone takes 2^-20 of the weight.  (8 multiplications a
// tile, for all its rows; no difference in time.)
constexpr int kScaleShift = 16;
constexpr float kScaleUp = 65536.0f;
constexpr float kNoRef = -3.4028234663852886e38f;  // c before any key: the first weight is infinite and sets it

struct AttnArgs {
    KvView view;
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    const float* q;
    float* out;
    float* part;       // partial results: slot i of workgroup w at part + (2 w + i) * slot size
    int4* owners;      // of item (tile slot, head): first and last workgroup, slot of the first
    int64_t ldq, ldo;
    int group;         // query heads of a key/value head
    float scale_log2;  // |scale| log2(e) without scale's exponent: in [0.72, 1.45), or 0
    int scale_exp;     // ... and that, added to the query's: neither leaves float32 alone
    float sign;        // of scale
    int window;
    int unit_shift;    // log2 of a unit's keys (split only)
    int workgroups;    // of one round, a run of units each (split only)
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

template <int ROWS, bool SPLIT>
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
    s.units = SPLIT && s.hi > s.lo ? ((s.hi - s.lo - 1) >> A.unit_shift) + 1 : 1;
    return s;
}

// Row tiles are numbered without a sum over the sequences before: sequence b
// has the numbers from floor(row_start[b] group / ROWS) + b on, as many as
// it can need (its last ones may be unused).
template <int ROWS>
__device__ __forceinline__ int first_tile(const AttnArgs& A, int b) {
    return min(max(A.view.row_start[b], 0), A.view.T) * A.group / ROWS + b;
}

// The sequence whose numbers hold tile x: the wave tests 64 entries a step.
template <int ROWS>
__device__ __forceinline__ int sequence_of_tile(const AttnArgs& A, int x) {
    const int lane = threadIdx.x & (kWave - 1);
    int lo = 0, span = A.view.B - 1;
    while (span > 0) {
        const int step = (span + kWave - 1) / kWave;
        const int off = (lane + 1) * step;
        const bool below = off <= span && first_tile<ROWS>(A, lo + off) <= x;
        const int c = __popcll(__ballot(below));
        const int left = span - c * step;
        lo += c * step;
        span = left < step - 1 ? left : step - 1;
    }
    return lo;
}

// Inclusive sum over the lanes of a wave: within rows of 16 (row_shr 1, 2, 4,
// 8), then across them (row_bcast 15 and 31).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// Runs: `total` units in as many runs as there are workgroups, or units if
// these are fewer, run w from floor(w total / runs) on.  Where the runs are a
// multiple of equally long items no run crosses from one item to the next.
struct Runs {
    int total, runs, per, rest;
    __device__ __forceinline__ Runs(int total_, int workgroups)
        : total(total_), runs(max(min(workgroups, total_), 1)),
          per(static_cast<int>(static_cast<uint32_t>(total_) / static_cast<uint32_t>(runs))), rest(total_ - per * runs) {}
    __device__ __forceinline__ int start(int w) const {
        return w * per + static_cast<int>(static_cast<uint32_t>(w * rest) / static_cast<uint32_t>(runs));
    }
    // the run that holds unit u: the largest w with floor(w total / runs) <= u
    __device__ __forceinline__ int owner(int u) const {
        return static_cast<int>(((static_cast<int64_t>(u) + 1) * runs - 1) / total);
    }
};

struct Place {
    int b;       // the sequence that holds the first unit of the run; B: no run
    int before;  // units of the sequences before it
    int total;   // units of the batch
    Seq s;       // the sequence
};

// Units are numbered by sequence, row tile, head, position.  All 256 threads
// sum the sequences' units, 256 sequences at a time.  Row starts that are out
// of order could make more units than there are numbers: then there is no run.
template <int ROWS>
__device__ Place locate(const AttnArgs& A, int w, int* lds /* 5 */, Place* found) {
    const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
    const bool one = A.view.B <= kBlockThreads;
    int total = 0;
    bool ordered = true;  // the same in every thread
    if (t == 0) found->b = A.view.B;
    for (int pass = one ? 1 : 0; pass < 2; ++pass) {  // the sum, then the place
        int base = 0;
        for (int b0 = 0; b0 < A.view.B; b0 += kBlockThreads) {
            Seq s = {};
            int mine = 0;
            bool disorder = false;
            if (b0 + t < A.view.B) {
                s = sequence<ROWS, true>(A, b0 + t);
                mine = s.tiles * A.view.heads * s.units;
                disorder = A.view.row_start[b0 + t] > A.view.row_start[b0 + t + 1];
            }
            const int scan = __ballot(disorder) == 0 ? wave_scan(mine) : -1;
            __syncthreads();
            if (lane == kWave - 1) lds[wave] = scan;
            __syncthreads();
            int before = base;
            for (int i = 0; i < kWavesPerBlock; ++i) {
                if (i < wave) before += lds[i];
                base += lds[i];
                ordered &= lds[i] >= 0;
            }
            if (pass == 0) continue;
            if (one) total = base;
            if (!ordered) continue;
            const Runs R(total, A.workgroups);
            const int key = w < R.runs ? R.start(w) : -1;
            const int begin = before + scan - mine;
            if (key >= begin && key < begin + mine) *found = Place{b0 + t, begin, total, s};
        }
        if (pass == 0) total = base;
    }
    __syncthreads();
    Place P;
    int* to = reinterpret_cast<int*>(&P);
    const int* from = reinterpret_cast<const int*>(found);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(Place) / sizeof(int)); ++i)
        to[i] = __builtin_amdgcn_readfirstlane(from[i]);
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

// The largest of eight, NaN if one is: gfx950's three-operand maximum, which
// needs no quieting of its operands first (fmaxf of values that the compiler
// cannot trace to an arithmetic result does).  No inline assembly: its operands
// come from matrix instructions, whose results the compiler waits for only
// where it knows the reader.
__device__ __forceinline__ float largest(const float (&x)[8]) {
    auto max3 = [](float a, float b, float c) { return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c); };
    return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), __builtin_elementwise_maximum(x[6], x[7]));
}

// Two float16, rounded to nearest, once: of a conversion that the compiler may
// repeat, one is fused with the product before it and another is not, and the
// two differ by a step of float16.  HOLD: nor fused at all (two instructions
// that each write half a register are slower than the packed conversion); not
// for results of exponentials, whose readers the compiler has to know.
template <bool HOLD>
__device__ __forceinline__ uint32_t pk(float a, float b) {
    if constexpr (HOLD) asm("" : "+v"(a), "+v"(b));
    uint32_t r = __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
    asm("" : "+v"(r));
    return r;
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
    bool has[2];      // the half has a page; without one page 0 is read and not seen
    __device__ __forceinline__ bool ok(int i) const { return has[i]; }
};

__device__ __forceinline__ Pages pages_of(const AttnArgs& A, int b, int h, int key) {
    Pages p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pos = key + 16 * i;
        const int j = pos >> A.view.page_shift;
        int page = -1;
        if (j < A.view.max_pages) page = A.view.table[static_cast<int64_t>(b) * A.view.max_pages + j];
        p.has[i] = page >= 0 && page < A.view.num_pages;
        p.cell[i] = ((static_cast<int64_t>(p.has[i] ? page : 0) * A.view.heads + h) << A.view.page_shift) +
                    (pos & ((1 << A.view.page_shift) - 1));
    }
    return p;
}

// Keys and their scales, values and theirs: loaded apart, each into the
// registers that the step before has just used, so that a tile's keys arrive
// while the tile before is in its softmax and products, and its values while
// its own scores are computed.
template <int D, bool F16>
__device__ __forceinline__ void load_keys(const AttnArgs& A, const Pages& p, KvRegs<D, F16>& r) {
    using T = KvRegs<D, F16>;
    constexpr int kRow = D * T::kE;  // bytes of a key
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t cell = p.cell[u];
        const uint8_t* kp = A.k + cell * kRow + (n * kRow + g * 16);
#pragma unroll
        for (int s = 0; s < T::kKLoads; ++s) r.k[u][s] = *reinterpret_cast<const u32x4*>(kp + 64 * s);
        if constexpr (!F16) r.ks[u] = *reinterpret_cast<const f32x4*>(A.ks + cell + 4 * g);
    }
}

template <int D, bool F16>
__device__ __forceinline__ void load_values(const AttnArgs& A, const Pages& p, KvRegs<D, F16>& r) {
    using T = KvRegs<D, F16>;
    constexpr int kRow = D * T::kE;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t cell = p.cell[u];
        if constexpr (!F16) r.vs[u] = *reinterpret_cast<const f32x4*>(A.vs + cell + 4 * g);
        const uint8_t* vp = A.v + cell * kRow + (4 * g * kRow + n * (kRow / 16));
#pragma unroll
        for (int e = 0; e < 4; ++e) load_words(r.v[4 * u + e], vp + e * kRow);
    }
}

// What sums under reference `from` are multiplied by, as a power of two, to
// stand under `to`.  A factor of 2^-150 is met (tiny values before huge ones)
// and its sums still count: float32 holds the results but not the factor.
__device__ __forceinline__ int rebase(float from, float to) { return static_cast<int>(fmaxf(from - to, -1000.0f)); }

// The rows of a workgroup as each wave holds them.
template <int D, bool F16, int R>
struct Rows {
    static constexpr int kQ = F16 ? D / 32 : D / 64;  // instructions of one term over D
    static constexpr int kTerms = F16 ? 2 : 3;
    u32x4 q[R][kTerms][kQ];
    float qs[R];   // score in log2 units = qs * (integer or float16 score) [* key scale], > 0
    bool broken[R];  // the query is not finite
    int pos[R];    // position of the lane's row, -1 for a row past the item's
    f32x4 o[R][D / 16];
    float c[R];    // reference of the weights, log2: a whole number, so that changing it rounds nothing
    float l[R];    // this lane's share of their sum
};

// q of the lane's rows, 16 (8 for float16) dimensions at a time as the
// lane's B operand takes them: dimension 64 s + 16 g + byte (32 s + 8 g + e).
template <int D, bool F16, int R>
struct Queries {
    static constexpr int kPer = F16 ? 8 : 16;
    static constexpr int kQ = Rows<D, F16, R>::kQ;
    float x[R][kQ][kPer];
    int pos[R];
};

template <int D, bool F16, int R>
__device__ __forceinline__ void fetch_queries(const AttnArgs& A, const Seq& S, int tile, int h, Queries<D, F16, R>& Q) {
    constexpr int kPer = Queries<D, F16, R>::kPer;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int rho = (tile * R + r) * 16 + n;
        const bool real = rho < S.n * A.group;
        const int i = real ? rho / A.group : 0;
        const int head = h * A.group + (real ? rho - i * A.group : 0);
        Q.pos[r] = real ? S.base + i : INT32_MIN;
        const float* src = A.q + static_cast<int64_t>(S.first + i) * A.ldq + static_cast<int64_t>(head) * D;
#pragma unroll
        for (int s = 0; s < Queries<D, F16, R>::kQ; ++s) {
            const float* p = src + s * (4 * kPer) + g * kPer;
            if (A.vec_q) {
#pragma unroll
                for (int e = 0; e < kPer; e += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(p + e);
                    Q.x[r][s][e] = f.x; Q.x[r][s][e + 1] = f.y; Q.x[r][s][e + 2] = f.z; Q.x[r][s][e + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e) Q.x[r][s][e] = p[e];
            }
        }
    }
}

template <int D, bool F16, int R>
__device__ __forceinline__ void prepare_rows(const AttnArgs& A, Queries<D, F16, R>& Q, Rows<D, F16, R>& W) {
    using T = Rows<D, F16, R>;
    constexpr int kPer = Queries<D, F16, R>::kPer;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool real = Q.pos[r] != INT32_MIN;
        W.pos[r] = real ? Q.pos[r] : -1;
        float(&x)[T::kQ][kPer] = Q.x[r];
        // the largest magnitude by its bits: infinity and NaN come out on top
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < T::kQ; ++s)
#pragma unroll
            for (int e = 0; e < kPer; ++e) top = max(top, __float_as_uint(x[s][e]) & 0x7fffffffu);
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16, kWave)));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, kWave)));
        W.broken[r] = real && top >= 0x7f800000u;
        const float amax = top < 0x7f800000u ? __uint_as_float(top) : 0.0f;
        // the row scaled by a power of two first: amax in [1/2, 1)
        const int k = amax > 0.0f ? __builtin_amdgcn_frexp_expf(amax) : 0;
        const float an = __builtin_amdgcn_ldexpf(amax, -k);
        float inv, back;
        if constexpr (F16) {
            inv = 1024.0f;
            back = 1.0f / 1024.0f;
        } else {
            inv = an > 0.0f ? kQParts / an : 0.0f;
            back = an * (1.0f / kQParts);
        }
        W.qs[r] = __builtin_amdgcn_ldexpf(back * A.scale_log2, k + A.scale_exp);
        // all scores equal (a zero query or scale), a row that will be NaN or
        // one past the item's: zero parts, with a factor that keeps masked
        // scores at -infinity
        const bool flat = !real || !(W.qs[r] > 0.0f);
        if (flat) W.qs[r] = 1.0f;
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
                W.q[r][0][s] = flat ? u32x4{0, 0, 0, 0} : u32x4{hi[0], hi[1], hi[2], hi[3]};
                W.q[r][1][s] = flat ? u32x4{0, 0, 0, 0} : u32x4{lo[0], lo[1], lo[2], lo[3]};
            } else {
                // round(x) = a 2^14 + b 2^7 + c with a in [-128, 127], b and c
                // in [-64, 63]: adding 2^23 + 128 2^14 + 64 2^7 + 64 rounds x
                // and makes the digits the unsigned bit fields of the
                // mantissa, each its value plus 128 or 64.
                constexpr float kDigits = 8388608.0f + 128.0f * 16384.0f + 64.0f * 128.0f + 64.0f;
                u32x4 a, b, c;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    uint32_t v[4], w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = __float_as_uint(fmaf(__builtin_amdgcn_ldexpf(x[s][e + i], -k), inv, kDigits));
                        w[i] = v[i] << 2;  // a in byte 2, b in bits 1 .. 7 of byte 1
                    }
                    // the same byte of four words
                    auto bytes = [](const uint32_t(&x)[4], uint32_t sel) {
                        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(x[3], x[2], sel),
                                                     __builtin_amdgcn_perm(x[1], x[0], sel), 0x05040100u);
                    };
                    // a 7-bit field u as the byte u - 64
                    auto minus64 = [](uint32_t u) {
                        u ^= 0x40404040u;
                        return u | ((u & 0x40404040u) << 1);
                    };
                    a[e / 4] = bytes(w, 0x0c0c0602u) ^ 0x80808080u;
                    b[e / 4] = minus64((bytes(w, 0x0c0c0501u) >> 1) & 0x7f7f7f7fu);
                    c[e / 4] = minus64(bytes(v, 0x0c0c0400u) & 0x7f7f7f7fu);
                }
                W.q[r][0][s] = flat ? u32x4{0, 0, 0, 0} : a;
                W.q[r][1][s] = flat ? u32x4{0, 0, 0, 0} : b;
                W.q[r][2][s] = flat ? u32x4{0, 0, 0, 0} : c;
            }
        }
        W.c[r] = kNoRef;
        W.l[r] = 0.0f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) W.o[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

// One tile of 32 keys at positions key ..  edge: some row does not see some
// key of it, or a half has no page (wave-uniform).  `reload_keys` and
// `reload_values` fetch the next tile as soon as the registers are free.
template <int D, bool F16, int R, class LoadK, class LoadV>
__device__ __forceinline__ void tile_step(const AttnArgs& A, KvRegs<D, F16>& kv, Rows<D, F16, R>& W, int key, bool edge,
                                          bool ok0, bool ok1, int hi_any, int lo_any, LoadK reload_keys,
                                          LoadV reload_values) {
    using T = Rows<D, F16, R>;
    using V = KvRegs<D, F16>;
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4;

    float s[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
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
                for (int e = 0; e < 4; ++e) s[r][4 * u + e] = a[e];
            } else {
                // sums begin at the bits of 1.5 2^23: as float32 that is 1.5
                // 2^23 + sum, exactly (|sum| <= 128 128 256 = 2^22), and
                //   (a - 1.5 2^23 (1 + 1 / 2^14)) 2^14 + ((b - 1.5 2^23) 2^7 + c)
                // is a 2^14 + b 2^7 + c.  Both differences are exact, and so is
                // the inner sum while it lies below 2^24: rows of small codes
                // round once, at the end.  (With b's bias left in it, and taken
                // from a, a subtraction is saved and every score rounded to a
                // multiple of 2^6: 1 part in 2^15 of one key code of 1.  It was worth 1%
                // of a prefill chunk.)
                constexpr float kBias = 12582912.0f, kOff = kBias + kBias / 16384.0f;
                const int c = __float_as_int(kBias);
                i32x4 a[3] = {i32x4{c, c, c, c}, i32x4{c, c, c, c}, i32x4{c, c, c, c}};
#pragma unroll
                for (int i = 0; i < T::kQ; ++i)
#pragma unroll
                    for (int term = 0; term < 3; ++term)
                        a[term] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, kv.k[u][i]),
                                                                        __builtin_bit_cast(i32x4, W.q[r][term][i]), a[term],
                                                                        0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[r][4 * u + e] = fmaf(__int_as_float(a[0][e]) - kOff, 16384.0f,
                                           fmaf(__int_as_float(a[1][e]) - kBias, 128.0f, __int_as_float(a[2][e]))) *
                                      kv.ks[u][e];
            }
        }
    }
    reload_keys();

    // float16 values at positions no row sees may be anything: zero times
    // them has to be zero.  At positions that only some rows see, a value
    // that is not finite is taken out and makes those rows NaN by their sum.
    uint32_t taken = 0;
    if constexpr (F16) {
        if (edge) {
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
                if (out) taken |= 1u << e;
#pragma unroll
                for (int w = 0; w < V::kVWords; ++w) kv.v[e][w] = (any && !out) ? kv.v[e][w] : 0u;
            }
        }
    }

    // How far above the reference a score may lie: p dv within float16, and p
    // so that 2^30 of them have a sum.  From scales that the row sees only:
    // what lies in other places may be anything, and a NaN would lift the limit
    // for the values beside it.
    auto limit_of = [](const float(&x)[8]) { return fminf(kTopMax - __builtin_amdgcn_logf(largest(x)), kPMax); };
    float all = kTopMax;  // where every row sees every key
    float vs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) vs[e] = F16 ? 1.0f : kv.vs[e >> 2][e & 3] * kScaleUp;
    if constexpr (!F16) all = limit_of(vs);

    uint32_t ph[R][4], pl[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float dv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dv[e] = vs[e];
        if (edge) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = key + 16 * (e >> 2) + 4 * g + (e & 3);
                const bool seen = (e < 4 ? ok0 : ok1) && j <= W.pos[r] && j < hi_any &&
                                  (A.window == 0 || j - W.pos[r] > -A.window);
                s[r][e] = seen ? s[r][e] : -kInf;
                if constexpr (F16) {
                    if (seen && (taken >> e & 1)) W.l[r] = __uint_as_float(0x7fc00000u);
                } else {
                    dv[e] = seen ? dv[e] : 0.0f;
                }
            }
        }
        float limit = all;
        if constexpr (!F16) {
            if (edge) limit = limit_of(dv);
        }
        // The reference moves only when a row has outgrown it, or could have by
        // the lane's largest score and value scale.  (NaN is never above: it
        // stays in the sum or the products.)
        if (__ballot(fmaf(largest(s[r]), W.qs[r], -W.c[r]) > limit) != 0) {
            // the largest p dv becomes 2^9 .. 2^11 (log2 dv rounded down to the
            // exponent), unless p itself would pass 2^81
            float cn = W.c[r];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = s[r][e] * W.qs[r];
                if constexpr (F16) {
                    cn = fmaxf(cn, x - kTop);
                } else {
                    const int exponent = static_cast<int>(__float_as_uint(dv[e]) >> 23) - 127;
                    cn = fmaxf(cn, fmaxf(x + (static_cast<float>(exponent) - kTop), x - kPTop));
                }
            }
            cn = floorf(row_max(cn));
            const int by = rebase(W.c[r], cn);
            W.c[r] = cn;
            W.l[r] = __builtin_amdgcn_ldexpf(W.l[r], by);
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) W.o[r][t][i] = __builtin_amdgcn_ldexpf(W.o[r][t][i], by);
        }
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[r][e], W.qs[r], -W.c[r]));
            W.l[r] += p[e];
            if constexpr (!F16) p[e] *= dv[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ph[r][e] = pk<!F16>(p[2 * e], p[2 * e + 1]);
            const f16x2 h = __builtin_bit_cast(f16x2, ph[r][e]);
            pl[r][e] = pk<true>(p[2 * e] - static_cast<float>(h[0]), p[2 * e + 1] - static_cast<float>(h[1]));
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
    reload_values();
}

// Floats of one partial slot: 16 R rows of D sums, then their references, then
// the sums of their weights.
template <int D, int R>
constexpr int kSlotFloats = 16 * R * (D + 2);

// Four dimensions of a row's result.  A row that saw nothing has sum 0.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs& A, const Seq& S, int h, int rho, int d, f32x4 v, float sum) {
    v = sum == 0.0f ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : v / sum;
    const int i = rho / A.group;
    float* o = A.out + static_cast<int64_t>(S.first + i) * A.ldo + static_cast<int64_t>(h * A.group + rho - i * A.group) * D + d;
    if (A.vec_o) {
        *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = v[e];
    }
}

// Waves a SIMD that the registers have to allow: two (256 registers each),
// one for 256-wide heads, whose keys, values, queries and results take 32 to 64
// each (held to 256 registers, a decode step of 8-bit ones takes 32.7 us
// instead of 30.3).
template <int D>
constexpr int kWavesPerSimd = D == 256 ? 1 : 2;

template <int D, bool F16, int R, bool SPLIT, int WAVES = kWavesPerBlock>
__global__ __launch_bounds__(WAVES * kWave, WAVES == 8 ? 2 : kWavesPerSimd<D>)
void attn_kernel(AttnArgs A) {
    constexpr int kRows = 16 * R;
    constexpr int kPad = D + 4;
    constexpr int kThreads = WAVES * kWave;
    constexpr int kStep = kTile * WAVES;  // keys of the workgroup's step
    __shared__ __align__(16) float so[WAVES * 16 * kPad];
    __shared__ float sm[WAVES][kRows], sl[WAVES][kRows];
    __shared__ int sums[kWavesPerBlock];
    __shared__ Place place;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int w = blockIdx.x;
    int b, before = 0, total = 0, u = 0, u_end = 1;  // the run of units, and the units before sequence b
    int tile = 0, h = 0, c0 = 0, c1 = 1;  // the piece: units c0 .. c1 - 1 of an item
    Seq S;
    if constexpr (SPLIT) {
        const Place P = locate<kRows>(A, w, sums, &place);
        b = P.b;
        if (b >= A.view.B) return;  // no run
        before = P.before;
        total = P.total;
        S = P.s;
        const Runs runs(total, A.workgroups);
        u = runs.start(w);
        u_end = runs.start(w + 1);
    } else {
        // items in order of tile, heads fastest: workgroups w and w + 8 (one
        // XCD) work on the same few heads' keys
        const int x = w / A.view.heads;
        h = w - x * A.view.heads;
        b = __builtin_amdgcn_readfirstlane(sequence_of_tile<kRows>(A, x));
        S = sequence<kRows, false>(A, b);
        tile = x - first_tile<kRows>(A, b);
        if (tile < 0 || tile >= S.tiles) return;
        tile = S.tiles - 1 - tile;  // the longest first
    }
    bool first_piece = true;
    while (u < u_end) {
        if constexpr (SPLIT) {
            while (u - before >= S.tiles * A.view.heads * S.units) {
                before += S.tiles * A.view.heads * S.units;
                S = sequence<kRows, true>(A, ++b);
            }
            const int item = static_cast<int>(static_cast<uint32_t>(u - before) / static_cast<uint32_t>(S.units));
            c0 = u - before - item * S.units;
            c1 = min(c0 + (u_end - u), S.units);
            tile = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(A.view.heads));
            h = item - tile * A.view.heads;
            if (c0 == 0 && threadIdx.x == 0) {
                const Runs runs(total, A.workgroups);
                const int last = c1 == S.units ? w : runs.owner(u + S.units - 1);
                A.owners[static_cast<int64_t>(first_tile<kRows>(A, b) + tile) * A.view.heads + h] =
                    make_int4(w, last, first_piece ? 0 : 1, 0);
            }
            u += c1 - c0;
        } else {
            u = u_end;
        }

        // the queries first: their parts are formed while the first keys come
        Queries<D, F16, R> queries;
        fetch_queries<D, F16, R>(A, S, tile, h, queries);
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
        int end = hi_any, key = max(S.lo, lo_any & ~(kTile - 1));
        if constexpr (SPLIT) {
            const int64_t k1 = S.lo + (static_cast<int64_t>(c1) << A.unit_shift);
            if (k1 < end) end = static_cast<int>(k1);
            const int64_t k0 = S.lo + (static_cast<int64_t>(c0) << A.unit_shift);
            if (k0 > key) key = static_cast<int>(k0 < end ? k0 : end);
        }
        // a length near 2^31 with a window starts behind every table: there
        // the first key is `end`, so that nothing below can pass 31 bits
        key = min(key, max(end, 0)) + wave * kTile;

        // The next tile's pages are looked up, and their addresses formed, a
        // whole step ahead: formed where the loads start they cost 7% (32
        // sequences of up to 16384: 247 against 231 us).
        KvRegs<D, F16> kv;
        Pages pg = {};
        const bool any = key < end;
        if (any) {
            pg = pages_of(A, b, h, key);
            load_keys<D, F16>(A, pg, kv);
            load_values<D, F16>(A, pg, kv);
        }
        Rows<D, F16, R> rows;
        prepare_rows<D, F16, R>(A, queries, rows);
        if (any) {
            Pages pn = pages_of(A, b, h, end - key > kStep ? key + kStep : key);
            for (;;) {
                const bool more = end - key > kStep;
                const Pages pt = pages_of(A, b, h, end - key > 2 * kStep ? key + 2 * kStep : key);
                const bool edge = !(pg.ok(0) && pg.ok(1) && key + kTile <= hi_all && key >= lo_all);
                tile_step<D, F16, R>(
                    A, kv, rows, key, edge, pg.ok(0), pg.ok(1), hi_any, lo_any,
                    [&] { if (more) load_keys<D, F16>(A, pn, kv); },
                    [&] { if (more) load_values<D, F16>(A, pn, kv); });
                if (!more) break;
                key += kStep;
                pg = pn;
                pn = pt;
            }
        }

        // join the waves, 16 rows at a time
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float l = row_sum(rows.l[r]);
            if (rows.broken[r] && l != 0.0f) l = __uint_as_float(0x7fc00000u);
            if (g == 0) {
                sm[wave][16 * r + n] = rows.c[r];
                sl[wave][16 * r + n] = l;
            }
        }
        const bool whole = c0 == 0 && c1 == S.units;
        float* slot = A.part + (2 * static_cast<int64_t>(w) + (first_piece ? 0 : 1)) * kSlotFloats<D, R>;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            __syncthreads();
            float M = kNoRef;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) M = fmaxf(M, sm[i][16 * r + n]);
            const int f = rebase(rows.c[r], M) + (F16 ? 0 : 9 - kScaleShift);  // values enter times 2^-9
            float* dst = so + (wave * 16 + n) * kPad + 4 * g * (D / 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int t = 0; t < D / 16; t += 4)
                    *reinterpret_cast<f32x4*>(dst + e * (D / 16) + t) =
                        f32x4{__builtin_amdgcn_ldexpf(rows.o[r][t][e], f), __builtin_amdgcn_ldexpf(rows.o[r][t + 1][e], f),
                              __builtin_amdgcn_ldexpf(rows.o[r][t + 2][e], f), __builtin_amdgcn_ldexpf(rows.o[r][t + 3][e], f)};
            __syncthreads();
            for (int x = threadIdx.x; x < 16 * (D / 4); x += kThreads) {
                const int row = x / (D / 4), d = x % (D / 4) * 4;
                const int rho = (tile * R + r) * 16 + row;
                if (rho >= S.n * A.group) continue;
                f32x4 v = *reinterpret_cast<const f32x4*>(so + row * kPad + d);
#pragma unroll
                for (int i = 1; i < WAVES; ++i)
                    v += *reinterpret_cast<const f32x4*>(so + (i * 16 + row) * kPad + d);
                float Mr = kNoRef, L = 0.0f;
#pragma unroll
                for (int i = 0; i < WAVES; ++i) Mr = fmaxf(Mr, sm[i][16 * r + row]);
#pragma unroll
                for (int i = 0; i < WAVES; ++i)
                    L += __builtin_amdgcn_ldexpf(sl[i][16 * r + row], rebase(sm[i][16 * r + row], Mr));
                if (!SPLIT || whole) {
                    store_row<D>(A, S, h, rho, d, v, L);
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

// Joins the parts of every item that more than one workgroup worked on:
// blockIdx.x is an item (row tile, head), every kJoinRows-th of its rows from
// blockIdx.y on is this workgroup's.  D / 4 threads hold a row's dimensions,
// 1024 / D groups of them share the parts.
constexpr int kJoinRows = 8;

template <int D>
__global__ __launch_bounds__(kBlockThreads)
void attn_join_kernel(AttnArgs A) {
    constexpr int kRows = 16, R = 1;
    constexpr int kQuads = D / 4;
    constexpr int kShares = kBlockThreads / kQuads;
    __shared__ __align__(16) f32x4 sv[kShares][kQuads];
    __shared__ float sl[kShares], sm[kShares];
    const int x = blockIdx.x / A.view.heads, h = blockIdx.x - x * A.view.heads;
    const int4 own = A.owners[blockIdx.x];  // used only if x is an item's number
    const int b = __builtin_amdgcn_readfirstlane(sequence_of_tile<kRows>(A, x));
    const Seq S = sequence<kRows, false>(A, b);
    const int tile = x - first_tile<kRows>(A, b);
    if (tile < 0 || tile >= S.tiles) return;
    // the item's first workgroup wrote them in this call; a workspace that two
    // calls share by mistake must not send this one out of it
    if (own.x < 0 || own.y >= A.workgroups || own.x >= own.y) return;  // (equal: one workgroup, written already)
    const int w0 = own.x, parts = own.y - own.x + 1;
    const int rows = min(kRows, S.n * A.group - tile * kRows);
    const int share = threadIdx.x / kQuads, quad = threadIdx.x % kQuads;
    const int i0 = parts * share / kShares, i1 = parts * (share + 1) / kShares;
    for (int row = blockIdx.y; row < rows; row += kJoinRows) {
        float M = kNoRef, L = 0.0f;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        auto add = [&](float m, float l, f32x4 o) {
            const float mn = fmaxf(M, m);
            const int fa = rebase(M, mn), fb = rebase(m, mn);
            L = __builtin_amdgcn_ldexpf(L, fa) + __builtin_amdgcn_ldexpf(l, fb);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_ldexpf(v[e], fa) + __builtin_amdgcn_ldexpf(o[e], fb);
            M = mn;
        };
#pragma unroll 2
        for (int i = i0; i < i1; ++i) {
            const float* slot = A.part + (2 * static_cast<int64_t>(w0 + i) + (i == 0 ? own.z & 1 : 0)) * kSlotFloats<D, R>;
            add(slot[kRows * D + row], slot[kRows * D + kRows + row],
                *reinterpret_cast<const f32x4*>(slot + row * D + 4 * quad));
        }
        sv[share][quad] = v;
        if (quad == 0) {
            sl[share] = L;
            sm[share] = M;
        }
        __syncthreads();
        if (share == 0) {
#pragma unroll
            for (int i = 1; i < kShares; ++i) add(sm[i], sl[i], sv[i][quad]);
            store_row<D>(A, S, h, tile * kRows + row, 4 * quad, v, L);
        }
        __syncthreads();
    }
}

}  // namespace

// The size is the same for every window: a window only shortens the items.
size_t attn_ws_bytes(const qmv_kv_cache& c, const qmv_kv_batch& b, int q_heads) {
    const AttnPlan p = plan_attn(c, b, q_heads, 0);
    return p.split ? p.part_bytes + p.owner_bytes : 256;
}

hipError_t launch_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* q, int64_t ldq, float* out,
                       int64_t ldo, int q_heads, float scale, int window, void* ws, hipStream_t stream) {
    const AttnPlan p = plan_attn(c, b, q_heads, window);
    AttnArgs A;
    A.view = view_of(c, b);
    A.k = static_cast<const uint8_t*>(c.k);
    A.v = static_cast<const uint8_t*>(c.v);
    A.ks = c.k_scale;
    A.vs = c.v_scale;
    A.q = q;
    A.out = out;
    A.part = static_cast<float*>(ws);
    A.owners = reinterpret_cast<int4*>(static_cast<char*>(ws) + p.part_bytes);
    A.ldq = ldq;
    A.ldo = ldo;
    A.group = q_heads / c.kv_heads;
    A.scale_log2 = std::frexp(scale < 0.0f ? -scale : scale, &A.scale_exp) * kLog2e;
    A.sign = scale < 0.0f ? -1.0f : 1.0f;
    A.window = window;
    A.unit_shift = p.unit_shift;
    A.workgroups = p.workgroups;
    A.vec_q = (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ldq % 4 == 0;
    A.vec_o = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ldo % 4 == 0;
    const dim3 grid(static_cast<unsigned>(p.blocks(c))), threads(static_cast<unsigned>(p.threads()));
    const dim3 join(static_cast<unsigned>(p.join_blocks(c)), kJoinRows);
#define ATTN(D, F16)                                                                                                 \
    do {                                                                                                             \
        if (p.split) {                                                                                               \
            hipLaunchKernelGGL((attn_kernel<D, F16, 1, true>), grid, threads, 0, stream, A);                         \
            hipLaunchKernelGGL((attn_join_kernel<D>), join, dim3(kBlockThreads), 0, stream, A);                      \
        } else if (p.waves == 8) {                                                                                   \
            hipLaunchKernelGGL((attn_kernel<D, F16 && D != 256, 1, false, 8>), grid, threads, 0, stream, A);         \
        } else if (D == 128 && p.r == 2) {                                                                           \
            hipLaunchKernelGGL((attn_kernel<128, F16, 2, false>), grid, threads, 0, stream, A);                      \
        } else {                                                                                                     \
            hipLaunchKernelGGL((attn_kernel<D, F16, 1, false>), grid, threads, 0, stream, A);                        \
        }                                                                                                            \
    } while (0)
    if (c.format == QMV_KV_F16) {
        if (c.head_dim == 64) ATTN(64, true);
        else if (c.head_dim == 128) ATTN(128, true);
        else ATTN(256, true);
    } else {
        if (c.head_dim == 64) ATTN(64, false);
        else if (c.head_dim == 128) ATTN(128, false);
        else ATTN(256, false);
    }
    return hipGetLastError();
}

}  // namespace qmv
