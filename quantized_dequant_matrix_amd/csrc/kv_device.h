// Device-side helpers shared by the kernels of the paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_device.h"
#include "../../include/qmv_step.h"

namespace qmv {

// What the kernels see of a cache and a batch (qmv_step.h).  page_size is a
// power of two: page_shift its logarithm.
struct KvView {
    const int32_t* table;
    const int32_t* row_start;
    const int32_t* kv_len;
    int64_t num_pages;
    int T, B, max_pages;
    int heads;
    int page_shift;
};

inline KvView view_of(const qmv_kv_cache& c, const qmv_kv_batch& b) {
    KvView v;
    v.table = b.page_table;
    v.row_start = b.row_start;
    v.kv_len = b.kv_len;
    v.num_pages = c.num_pages;
    v.T = static_cast<int>(b.T);
    v.B = b.B;
    v.max_pages = b.max_pages;
    v.heads = c.kv_heads;
    v.page_shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
    return v;
}

// The sequence that owns a row: the number of entries row_start[1 .. B] that
// are <= row, found by the whole wave 64 entries at a time (two steps up to
// B = 4096).  Returns B for a row behind the last sequence.  With an array
// that is not in order the result is some number in [0, B]; the caller checks
// the row against the two entries around it.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ row_start, int B, int row) {
    const int lane = threadIdx.x & (kWave - 1);
    int lo = 0, span = B;
    while (span > 0) {
        const int step = (span + kWave - 1) / kWave;
        const int off = (lane + 1) * step;
        const bool below = off <= span && row_start[lo + off] <= row;
        const int c = __popcll(__ballot(below));
        const int left = span - c * step;
        lo += c * step;
        span = left < step - 1 ? left : step - 1;
    }
    return lo;
}

}  // namespace qmv
