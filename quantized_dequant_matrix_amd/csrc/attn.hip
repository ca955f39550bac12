// Attention of new tokens over the paged cache.
//
//   s_j = scale q . k_j over the visible positions j, out = sum p_j v_j / sum p_j,
//   p_j = exp(s_j - max s)
//
// One wave a (row, query head), one pass over the keys in runs of 64 with the
// running maximum and sum of the softmax in float32: lane j takes the dot
// product of key j, then lane d the dimensions d, d + 64, ... of the values.
#include <stdint.h>

#include "kv_device.h"
#include "step_internal.h"

namespace qmv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool F16>
__global__ __launch_bounds__(kWave)
void attn_simple_kernel(KvView view, const void* kc, const void* vc, const float* ks, const float* vs,
                        const float* __restrict__ q, int64_t ldq, float* __restrict__ out, int64_t ldo, int group,
                        float scale, int window) {
    __shared__ float qs[D];
    __shared__ float ps[kWave];
    __shared__ int64_t cells[kWave];
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int b = find_sequence(view.row_start, view.B, row);
    if (b >= view.B) return;
    const int first = view.row_start[b], end = view.row_start[b + 1];
    if (row < first || row >= end) return;
    const int64_t len = view.kv_len[b];
    const int64_t pos = len - (end - static_cast<int64_t>(row));
    const int64_t top = static_cast<int64_t>(view.max_pages) << view.page_shift;
    const int64_t hi = pos + 1 < top ? pos + 1 : top;
    int64_t lo = window > 0 ? pos - window + 1 : 0;
    lo = lo > 0 ? lo : 0;
    for (int d = lane; d < D; d += kWave) qs[d] = q[row * ldq + h * D + d] * (scale * kLog2e);
    __syncthreads();
    constexpr int R = D / kWave;
    float acc[R] = {};
    float m = -__builtin_inff(), l = 0.0f;
    const int hk = h / group;
    for (int64_t j0 = lo; j0 < hi; j0 += kWave) {
        const int64_t j = j0 + lane;
        int64_t cell = -1;
        float s = -__builtin_inff();
        if (j < hi) {
            const int page = view.table[static_cast<int64_t>(b) * view.max_pages + (j >> view.page_shift)];
            if (page >= 0 && page < view.num_pages) {
                cell = ((static_cast<int64_t>(page) * view.heads + hk) << view.page_shift) + (j & ((1 << view.page_shift) - 1));
                float t = 0.0f;
                for (int d = 0; d < D; ++d) {
                    if constexpr (F16)
                        t = fmaf(qs[d], static_cast<float>(static_cast<const _Float16*>(kc)[cell * D + d]), t);
                    else
                        t = fmaf(qs[d], static_cast<float>(static_cast<const int8_t*>(kc)[cell * D + d]), t);
                }
                s = F16 ? t : t * ks[cell];
            }
        }
        float mt = s;
        for (int o = kWave / 2; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor(mt, o, kWave));
        const float mn = fmaxf(m, mt);
        const float use = mn == -__builtin_inff() ? 0.0f : mn;
        const float p = cell >= 0 ? exp2f(s - use) : 0.0f;
        const float alpha = exp2f(m - use);
        l = l * alpha + wave_sum(p);
        m = mn;
        __syncthreads();
        ps[lane] = p;
        cells[lane] = cell;
        __syncthreads();
        for (int i = 0; i < R; ++i) acc[i] *= alpha;
        for (int jj = 0; jj < kWave; ++jj) {
            const int64_t cj = cells[jj];
            if (cj < 0) continue;
            const float pj = F16 ? ps[jj] : ps[jj] * vs[cj];
            for (int i = 0; i < R; ++i) {
                if constexpr (F16)
                    acc[i] = fmaf(pj, static_cast<float>(static_cast<const _Float16*>(vc)[cj * D + lane + i * kWave]), acc[i]);
                else
                    acc[i] = fmaf(pj, static_cast<float>(static_cast<const int8_t*>(vc)[cj * D + lane + i * kWave]), acc[i]);
            }
        }
        __syncthreads();
    }
    for (int i = 0; i < R; ++i) out[row * ldo + h * D + lane + i * kWave] = l == 0.0f ? 0.0f : acc[i] / l;
}

}  // namespace

size_t attn_ws_bytes(const qmv_kv_cache&, const qmv_kv_batch&, int) { return 256; }

hipError_t launch_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, const float* q, int64_t ldq, float* out,
                       int64_t ldo, int q_heads, float scale, int window, void*, hipStream_t stream) {
    const KvView view = view_of(c, b);
    const dim3 grid(static_cast<unsigned>(b.T), static_cast<unsigned>(q_heads));
    const int group = q_heads / c.kv_heads;
#define ATTN(D, F16)                                                                                              \
    hipLaunchKernelGGL((attn_simple_kernel<D, F16>), grid, dim3(kWave), 0, stream, view, c.k, c.v, c.k_scale,     \
                       c.v_scale, q, ldq, out, ldo, group, scale, window)
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
