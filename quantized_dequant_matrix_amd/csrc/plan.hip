// The plan of a serving step: cache pages given back and taken, row starts,
// positions and slots, from the lengths of the sequences.
//
// With P(x) = ceil(x / page_size), a sequence gives back f = max(0, P(old) -
// P(new)) pages and takes t = max(0, P(new) - P(old)).  Exclusive sums of f,
// t and of the new rows over the sequences are all that the rest needs: the
// stack position of a page, the row of a sequence.  They are taken in 64-bit
// floating point, which is exact here (every sum is below 2^47) and has lane
// sums by DPP.
//
// A page that is taken need not be on the stack in memory: stack index s
// below the old count is read there, one above it is the (s - count)-th page
// given back, found by its sequence's sum.  So nothing that one thread writes
// is read by another, and everything after the sums can run at once: table
// entries are only read where nothing is written (behind the new length of
// sequences that give back, before the old one of those that take), stack
// entries below the old count, and written above it.
//
// Steps of few rows are one launch of one workgroup, which has the sums in LDS;
// others are two, the sums by one workgroup, then rows and pages by many.
// Latency bounds both: 6.5 us a call for 32 sequences, 10.4 for 256 with 173,000
// rows (kernels of 3.7 and 6.9).
#include <stdint.h>

#include "kv_device.h"
#include "serve_internal.h"
#include "step_device.h"

namespace qmv {
namespace {

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / kWave;
constexpr int kMostSmall = 64;  // sequences of a step in one launch
constexpr int kFillThreads = 256, kFillWaves = kFillThreads / kWave;

struct PlanHead {
    int32_t ok, count, full, pad;  // full: stack entries after everything was pushed
};

struct PlanView {
    qmv_kv_pool pool;
    PlanArgs a;
    PlanHead* head;
    int32_t* had;     // [B] P(kv_len)
    int32_t* pushed;  // [B] pages given back by the sequences before
    int32_t* popped;  // [B] pages taken by the sequences before
    int page_shift;
};

__device__ __forceinline__ int32_t pages_of(int32_t x, int shift) {
    return (x >> shift) + ((x & ((1 << shift) - 1)) != 0 ? 1 : 0);
}

// Exclusive sums over the workgroup in thread order and the totals, for three
// values at once.
__device__ __forceinline__ void block_sums(double (&v)[3], double (&total)[3], double (*part)[kPlanWaves]) {
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    double upto[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        upto[c] = wave_prefix(v[c]);
        if (lane == kWave - 1) part[c][wave] = upto[c];
    }
    __syncthreads();
    const int first = __builtin_amdgcn_readfirstlane(wave);
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const double waves = wave_prefix(lane < kPlanWaves ? part[c][lane] : 0.0);
        const double before = first > 0 ? lane_f64(waves, first - 1) : 0.0;
        v[c] = before + upto[c] - v[c];
        total[c] = lane_f64(waves, kPlanWaves - 1);
    }
    __syncthreads();
}

// Whether the step can be done, from the sums of new rows, pages given back and
// pages taken.
__device__ __forceinline__ void verdict(const PlanView& D, bool bad_length, int32_t count, const double (&sum)[3],
                                        int32_t* status, int32_t* lacking) {
    int32_t s = bad_length ? QMV_PLAN_LENGTH : 0;
    *lacking = 0;
    if (count < 0 || count > D.pool.num_pages || count + sum[1] > static_cast<double>(D.pool.num_pages)) s |= QMV_PLAN_STACK;
    if (sum[0] > static_cast<double>(D.a.T)) s |= QMV_PLAN_ROWS;
    if (!(s & QMV_PLAN_STACK) && sum[2] > count + sum[1]) {
        s |= QMV_PLAN_PAGES;
        *lacking = static_cast<int32_t>(fmin(sum[2] - count - sum[1], 2147483647.0));
    }
    *status = s;
}

// The last index i in [0, n) with sums[i] <= x (sums do not decrease and
// sums[0] <= x).
__device__ __forceinline__ int last_at_or_below(const int32_t* sums, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kPlanThreads)
void plan_sums_kernel(PlanView D) {
    __shared__ double part[3][kPlanWaves];
    __shared__ int bad_length;
    const int t = threadIdx.x, B = D.pool.B, shift = D.page_shift;
    const int32_t most = D.pool.max_pages << shift;  // at most 2^30
    if (t == 0) bad_length = 0;
    __syncthreads();
    double carry[3] = {0.0, 0.0, 0.0};
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        const int b = b0 + t;
        int32_t len = 0, keep = 0, n = 0;
        if (b < B) {
            len = D.a.kv_len[b];
            keep = D.a.keep ? D.a.keep[b] : len;
            n = D.a.n_new[b];
        }
        // keep is at most 2^30 and so is n before they are added
        if (len < 0 || len > most || keep < 0 || keep > len || n < 0 || n > most - keep) {
            bad_length = 1;
            len = keep = n = 0;
        }
        const int32_t had = pages_of(len, shift), has = pages_of(keep + n, shift);
        double v[3] = {static_cast<double>(n), had > has ? static_cast<double>(had - has) : 0.0,
                       has > had ? static_cast<double>(has - had) : 0.0};
        double total[3];
        block_sums(v, total, part);
        if (b < B) {
            D.had[b] = had;
            // sums beyond 31 bits only where the step is refused
            D.a.row_start[b + 1] = static_cast<int32_t>(fmin(carry[0] + v[0] + n, 2147483647.0));
            D.pushed[b] = static_cast<int32_t>(fmin(carry[1] + v[1], 2147483647.0));
            D.popped[b] = static_cast<int32_t>(fmin(carry[2] + v[2], 2147483647.0));
        }
#pragma unroll
        for (int c = 0; c < 3; ++c) carry[c] += total[c];
    }
    __syncthreads();
    // every thread with the same numbers
    const int32_t count = *D.a.free_count;
    int32_t status, lacking;
    verdict(D, bad_length != 0, count, carry, &status, &lacking);
    const bool ok = status == 0;
    __syncthreads();  // the count is read before it is written
    for (int b = t; b < B; b += kPlanThreads) {
        const int32_t len = D.a.kv_len[b];
        if (ok) {
            const int32_t keep = D.a.keep ? D.a.keep[b] : len;
            D.a.new_len[b] = keep + D.a.n_new[b];
        } else {
            D.a.new_len[b] = len;
            D.a.row_start[b + 1] = 0;
        }
    }
    if (t == 0) {
        D.a.row_start[0] = 0;
        *D.a.new_count = ok ? static_cast<int32_t>(count + carry[1] - carry[2]) : count;
        D.a.status[0] = status;
        D.a.status[1] = lacking;
        PlanHead h = {ok ? 1 : 0, count, ok ? static_cast<int32_t>(count + carry[1]) : count, 0};
        *D.head = h;
    }
}

// Page numbers of rows at `slot`s: the place, or -1 outside the cache.
__device__ __forceinline__ int64_t place(const PlanView& D, int32_t page, int32_t position) {
    const bool real = page >= 0 && page < D.pool.num_pages;
    return real ? (static_cast<int64_t>(page) << D.page_shift) + (position & ((1 << D.page_shift) - 1)) : -1;
}

// Sums of the sequences in LDS.
struct PlanLds {
    int32_t had[kMostSmall], has[kMostSmall], pushed[kMostSmall], popped[kMostSmall];
    int32_t start[kMostSmall], keep[kMostSmall];
    double part[3][kPlanWaves];
    int bad_length;
};

// Page j of sequence b after the step, with the sums in LDS.
__device__ __forceinline__ int32_t page_after(const PlanView& D, const PlanLds& S, int32_t count, int32_t full, int b, int32_t j) {
    if (j < S.had[b]) return D.pool.page_table[static_cast<int64_t>(b) * D.pool.max_pages + j];
    const int32_t s = full - 1 - (S.popped[b] + (j - S.had[b]));
    if (s < count) return D.pool.free_pages[s];
    const int32_t f = s - count;
    const int from = last_at_or_below(S.pushed, D.pool.B, f);
    return D.pool.page_table[static_cast<int64_t>(from) * D.pool.max_pages + S.has[from] + (f - S.pushed[from])];
}

// The whole step, B <= kMostSmall: a thread a sequence, then a row or a page.
__global__ __launch_bounds__(kPlanThreads)
void plan_small_kernel(PlanView D) {
    __shared__ PlanLds S;
    const int t = threadIdx.x, B = D.pool.B, shift = D.page_shift;
    const int32_t most = D.pool.max_pages << shift;
    const int32_t count = *D.a.free_count;
    int32_t len = 0, keep = 0, n = 0;
    if (t < B) {
        len = D.a.kv_len[t];
        keep = D.a.keep ? D.a.keep[t] : len;
        n = D.a.n_new[t];
    }
    const int32_t old_len = len;
    if (t == 0) S.bad_length = 0;
    __syncthreads();
    if (len < 0 || len > most || keep < 0 || keep > len || n < 0 || n > most - keep) {
        S.bad_length = 1;
        len = keep = n = 0;
    }
    const int32_t had = pages_of(len, shift), has = pages_of(keep + n, shift);
    double v[3] = {static_cast<double>(n), had > has ? static_cast<double>(had - has) : 0.0,
                   has > had ? static_cast<double>(has - had) : 0.0};
    double total[3];
    block_sums(v, total, S.part);  // its barriers are also behind bad_length, and the reads of what is written below
    int32_t status, lacking;
    verdict(D, S.bad_length != 0, count, total, &status, &lacking);
    const bool ok = status == 0;
    if (t < B) {
        D.a.new_len[t] = ok ? keep + n : old_len;
        D.a.row_start[t + 1] = ok ? static_cast<int32_t>(v[0]) + n : 0;
        S.had[t] = had;
        S.has[t] = has;
        S.keep[t] = keep;
        S.start[t] = static_cast<int32_t>(fmin(v[0], 2147483647.0));
        S.pushed[t] = static_cast<int32_t>(fmin(v[1], 2147483647.0));
        S.popped[t] = static_cast<int32_t>(fmin(v[2], 2147483647.0));
    }
    if (t == 0) {
        D.a.row_start[0] = 0;
        *D.a.new_count = ok ? static_cast<int32_t>(count + total[1] - total[2]) : count;
        D.a.status[0] = status;
        D.a.status[1] = lacking;
    }
    if (!ok) return;
    __syncthreads();
    const int32_t rows = static_cast<int32_t>(total[0]), back = static_cast<int32_t>(total[1]), taken = static_cast<int32_t>(total[2]);
    const int32_t full = count + back;
    if (D.a.position || D.a.slot) {
        for (int32_t r = t; r < rows; r += kPlanThreads) {
            const int b = last_at_or_below(S.start, B, r);  // sequences without rows share the next one's start
            const int32_t p = S.keep[b] + (r - S.start[b]);
            if (D.a.position) D.a.position[r] = p;
            if (D.a.slot) D.a.slot[r] = place(D, page_after(D, S, count, full, b, p >> shift), p);
        }
    }
    for (int32_t f = t; f < back; f += kPlanThreads) {
        const int b = last_at_or_below(S.pushed, B, f);
        D.pool.free_pages[count + f] = D.pool.page_table[static_cast<int64_t>(b) * D.pool.max_pages + S.has[b] + (f - S.pushed[b])];
    }
    for (int32_t f = t; f < taken; f += kPlanThreads) {
        const int b = last_at_or_below(S.popped, B, f);
        const int32_t j = S.had[b] + (f - S.popped[b]);
        D.pool.page_table[static_cast<int64_t>(b) * D.pool.max_pages + j] = page_after(D, S, count, full, b, j);
    }
}

// Page j of sequence b after the step.
__device__ __forceinline__ int32_t page_after(const PlanView& D, const PlanHead& h, int b, int32_t j) {
    const int32_t had = D.had[b];
    if (j < had) return D.pool.page_table[static_cast<int64_t>(b) * D.pool.max_pages + j];
    const int32_t s = h.full - 1 - (D.popped[b] + (j - had));
    if (s < h.count) return D.pool.free_pages[s];
    const int f = s - h.count;
    const int from = last_at_or_below(D.pushed, D.pool.B, f);  // the one that gives back page f
    const int32_t has = pages_of(D.a.new_len[from], D.page_shift);
    return D.pool.page_table[static_cast<int64_t>(from) * D.pool.max_pages + has + (f - D.pushed[from])];
}

// The first `row_blocks` workgroups take a row a thread, the others a
// sequence a wave.
__global__ __launch_bounds__(kFillThreads)
void plan_fill_kernel(PlanView D, unsigned row_blocks) {
    const PlanHead h = *D.head;
    if (!h.ok) return;
    const int lane = threadIdx.x & (kWave - 1), B = D.pool.B;
    if (blockIdx.x < row_blocks) {
        const int32_t r = static_cast<int32_t>(blockIdx.x * kFillThreads + threadIdx.x);
        if (r >= D.a.row_start[B]) return;
        const int b = last_at_or_below(D.a.row_start, B, r);
        // sequences without rows share their start with the next one: the
        // last one at or below r has rows
        const int32_t n = D.a.row_start[b + 1] - D.a.row_start[b];
        const int32_t p = D.a.new_len[b] - n + (r - D.a.row_start[b]);
        if (D.a.position) D.a.position[r] = p;
        if (D.a.slot) {
            const int32_t page = page_after(D, h, b, p >> D.page_shift);
            D.a.slot[r] = place(D, page, p);
        }
        return;
    }
    const int b = static_cast<int>((blockIdx.x - row_blocks) * kFillWaves + threadIdx.x / kWave);
    if (b >= B) return;
    const int32_t had = D.had[b], has = pages_of(D.a.new_len[b], D.page_shift);
    int32_t* table = D.pool.page_table + static_cast<int64_t>(b) * D.pool.max_pages;
    for (int32_t j = has + lane; j < had; j += kWave) D.pool.free_pages[h.count + D.pushed[b] + (j - has)] = table[j];
    for (int32_t j = had + lane; j < has; j += kWave) table[j] = page_after(D, h, b, j);
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t plan_ws_bytes(int B) { return 256 + 3 * align256(static_cast<size_t>(B) * sizeof(int32_t)); }

hipError_t launch_kv_plan(const qmv_kv_pool& pool, const PlanArgs& a, void* ws, hipStream_t stream) {
    PlanView D;
    D.pool = pool;
    D.a = a;
    char* p = static_cast<char*>(ws);
    const size_t each = align256(static_cast<size_t>(pool.B) * sizeof(int32_t));
    D.head = reinterpret_cast<PlanHead*>(p);
    D.had = reinterpret_cast<int32_t*>(p + 256);
    D.pushed = reinterpret_cast<int32_t*>(p + 256 + each);
    D.popped = reinterpret_cast<int32_t*>(p + 256 + 2 * each);
    D.page_shift = __builtin_ctz(static_cast<unsigned>(pool.page_size));
    // One workgroup goes through 1024 rows or pages at a time, a few
    // microseconds each, which a second launch costs once: 32 sequences with 100
    // rows take 7.1 us here and 9.4 there, with 5000 rows 11.7 and 9.7, 256
    // sequences of which some end and give back 12,000 pages 12.8 and 10.6.  How
    // many pages move is known on the device only, and a step that moves most of
    // its cache is here all the same: 8192 pages 7.0 and 9.1, 16,384 12.2 and 9.0,
    // 64 sequences of 1024 pages that end at once 43 and 9.2.
    if (pool.B <= kMostSmall && a.T <= 2048) {
        hipLaunchKernelGGL(plan_small_kernel, dim3(1), dim3(kPlanThreads), 0, stream, D);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(plan_sums_kernel, dim3(1), dim3(kPlanThreads), 0, stream, D);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned rows =
        a.position || a.slot ? static_cast<unsigned>((a.T + kFillThreads - 1) / kFillThreads) : 0u;
    const unsigned seqs = static_cast<unsigned>((pool.B + kFillWaves - 1) / kFillWaves);
    hipLaunchKernelGGL(plan_fill_kernel, dim3(rows + seqs), dim3(kFillThreads), 0, stream, D, rows);
    return hipGetLastError();
}

}  // namespace qmv
