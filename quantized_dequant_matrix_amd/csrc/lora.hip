// Low-rank adapters of the sequences of a batch, added to a shared
// projection's output:  y_r = base_r + scale_s Bm_s (A_s x_r).
//
// Two launches: the ranks v_r = A_s x_r into the workspace, then their
// products with Bm_s added to the rows.
#include <stdint.h>

#include "kv_device.h"
#include "serve_internal.h"
#include "step_device.h"

namespace qmv {
namespace {

struct LoraView {
    qmv_lora l;
    LoraArgs a;
    float* v;  // [T][max_rank]
};

template <bool BF16>
__device__ __forceinline__ float weight_at(const void* p, int64_t i) {
    const uint32_t b = static_cast<const uint16_t*>(p)[i];
    if constexpr (BF16) return __uint_as_float(b << 16);
    return half_bits_to_float(b);
}

// The adapter of a row and its rank: -1 without an adapter, -2 for a row of
// no sequence.  The whole wave asks for the same row.
__device__ __forceinline__ int adapter_of(const LoraView& D, int row, int* rank) {
    const int B = static_cast<int>(D.a.B);
    const int b = find_sequence(D.a.row_start, B, row);
    if (b >= B || row < D.a.row_start[b] || row >= D.a.row_start[b + 1]) return -2;
    const int s = D.a.adapter[b];
    if (s < 0 || s >= D.l.slots) return -1;
    const int r = D.l.rank ? D.l.rank[s] : D.l.max_rank;
    *rank = r < 0 ? 0 : (r > D.l.max_rank ? D.l.max_rank : r);
    return s;
}

// A wave a row and rank.
template <bool BF16>
__global__ __launch_bounds__(kBlockThreads)
void lora_shrink_kernel(LoraView D) {
    const int row = blockIdx.x, lane = threadIdx.x & (kWave - 1);
    const int j = blockIdx.y * kWavesPerBlock + threadIdx.x / kWave;
    int rank = 0;
    const int s = adapter_of(D, row, &rank);
    if (s < 0 || j >= rank) return;
    const float* x = D.a.x + row * D.a.ldx;
    const int64_t at = (static_cast<int64_t>(s) * D.l.max_rank + j) * D.l.K;
    float sum = 0.0f;
    for (int64_t k = lane; k < D.l.K; k += kWave) sum = fmaf(weight_at<BF16>(D.l.A, at + k), x[k], sum);
    sum = wave_sum(sum);
    if (lane == 0) D.v[static_cast<int64_t>(row) * D.l.max_rank + j] = sum;
}

// A thread an output.
template <bool BF16>
__global__ __launch_bounds__(kBlockThreads)
void lora_expand_kernel(LoraView D) {
    const int row = blockIdx.x;
    int rank = 0;
    const int s = adapter_of(D, row, &rank);
    const int64_t n = static_cast<int64_t>(blockIdx.y) * kBlockThreads + threadIdx.x;
    if (s == -2 || n >= D.l.N || (s == -1 && D.a.base == D.a.y)) return;
    float sum = 0.0f;
    if (s >= 0) {
        const float* v = D.v + static_cast<int64_t>(row) * D.l.max_rank;
        const int64_t at = (static_cast<int64_t>(s) * D.l.N + n) * D.l.max_rank;
        for (int j = 0; j < rank; ++j) sum = fmaf(weight_at<BF16>(D.l.Bm, at + j), v[j], sum);
        sum *= D.l.scale[s];
    }
    const float b = D.a.base ? D.a.base[row * D.a.ldb + n] : 0.0f;
    D.a.y[row * D.a.ldy + n] = b + sum;
}

template <bool BF16>
hipError_t launch(const LoraView& D, hipStream_t stream) {
    const unsigned T = static_cast<unsigned>(D.a.T);
    hipLaunchKernelGGL(lora_shrink_kernel<BF16>, dim3(T, static_cast<unsigned>(D.l.max_rank) / kWavesPerBlock),
                       dim3(kBlockThreads), 0, stream, D);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lora_expand_kernel<BF16>,
                       dim3(T, static_cast<unsigned>((D.l.N + kBlockThreads - 1) / kBlockThreads)),
                       dim3(kBlockThreads), 0, stream, D);
    return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(const qmv_lora& l, int64_t, int64_t T) {
    return static_cast<size_t>(T) * static_cast<size_t>(l.max_rank) * sizeof(float);
}

hipError_t launch_lora(const qmv_lora& l, const LoraArgs& a, void* ws, hipStream_t stream) {
    LoraView D;
    D.l = l;
    D.a = a;
    D.v = static_cast<float*>(ws);
    return l.format == QMV_LORA_BF16 ? launch<true>(D, stream) : launch<false>(D, stream);
}

}  // namespace qmv
