// Sweeps attn_paged's documented limits through the argument checks
// (step_api.cpp) into the launch plan (attn_plan.h), and checks every planned
// launch against what a launch can hold: threads of a dimension below 2^32,
// item and unit numbers below 2^31, and a workspace of the size that
// attn_paged_ws_bytes names whatever the window.  Built and run by
// tests/test_attn_plan.py (host code only, no GPU).
#include <cstdint>
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

#include "attn_plan.h"
#include "step_internal.h"

static int failures = 0;
static int64_t planned = 0, eights = 0, splits = 0, doubles = 0;
#define CHECK(cond) do { if (!(cond)) { if (++failures < 20) \
    std::printf("line %d: %s (T %lld B %d heads %d over %d of %d, format %d, %d pages of %d, window %d)\n", __LINE__, #cond, \
                static_cast<long long>(b.T), b.B, q_heads, c.kv_heads, c.head_dim, c.format, b.max_pages, c.page_size, window); } } while (0)

size_t qmm_q4_0_q8act_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

namespace qmv {
hipError_t launch_kv_write(const qmv_kv_cache&, const qmv_kv_batch&, const float*, int64_t, const float*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_read(const qmv_kv_cache&, const qmv_kv_batch&, float*, int64_t, float*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_rmsnorm(const float*, const float*, const float*, float*, float*, int8_t*, float*, int64_t, int64_t, float, hipStream_t) { return hipSuccess; }
hipError_t launch_qmm_q8(const void*, const int8_t*, const float*, float*, int64_t, int64_t, int64_t, void*, hipStream_t) { return hipSuccess; }
size_t draft_ws_bytes(int64_t, int, int64_t) { return 0; }
hipError_t launch_draft_verify(const DraftArgs&, void*, hipStream_t) { return hipSuccess; }

size_t attn_ws_bytes(const qmv_kv_cache& c, const qmv_kv_batch& b, int q_heads) {
    const AttnPlan p = plan_attn(c, b, q_heads, 0);
    return p.split ? p.part_bytes + p.owner_bytes : 256;
}
hipError_t launch_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, const float*, int64_t, float*, int64_t, int q_heads,
                       float, int window, void*, hipStream_t) {
    const AttnPlan p = plan_attn(c, b, q_heads, window);
    const int64_t group = q_heads / c.kv_heads, limit = int64_t{1} << 32;
    ++planned;
    eights += !p.split && p.waves == 8;
    splits += p.split;
    doubles += p.r == 2;
    CHECK(p.blocks(c) >= 1 && p.blocks(c) < (int64_t{1} << 31));
    CHECK(p.threads() == 256 || p.threads() == 512);
    CHECK(p.blocks(c) * p.threads() < limit);
    CHECK(p.join_blocks(c) * 256 < limit);
    CHECK(!p.split || p.threads() == 256);
    CHECK(p.r == 1 || (p.threads() == 256 && c.head_dim == 128));
    CHECK(p.tiles >= b.T * group / (16 * p.r) + b.B);
    if (p.split) {
        const int64_t keys = static_cast<int64_t>(b.max_pages) * c.page_size;
        // items of a batch at most: of n tokens ceil(n group / 16) tiles a head, at most n ceil(group / 16)
        const int64_t seqs = b.B < b.T ? b.B : b.T, whole = (b.T * group + 15 * seqs) / 16, apart = b.T * ((group + 15) / 16);
        const int64_t items = (whole < apart ? whole : apart) * c.kv_heads, units = ((keys - 1) >> p.unit_shift) + 1;
        CHECK(static_cast<__int128>(items) * units < (__int128{1} << 31));
        CHECK(p.owner_bytes == static_cast<size_t>(p.join_blocks(c)) * 16);
        CHECK(p.part_bytes + p.owner_bytes <= attn_ws_bytes(c, b, q_heads));
    }
    return hipSuccess;
}
}  // namespace qmv

int main() {
    std::mt19937_64 rng(5);
    auto one_of = [&](std::initializer_list<int64_t> v) { return v.begin()[rng() % v.size()]; };
    auto spread = [&](double hi) {  // a whole number of [1, hi], spread over its logarithm
        return static_cast<int64_t>(std::exp(std::uniform_real_distribution<double>(0.0, std::log(hi))(rng)));
    };
    float* const p = reinterpret_cast<float*>(uintptr_t{1} << 20);
    int32_t* const i = reinterpret_cast<int32_t*>(p);
    int64_t refused = 0;
    auto call = [&](int64_t T, int B, int heads, int group, int dim, int format, int page, int pages, int window) {
        const qmv_kv_cache c = {p, p, p, p, 1000, heads, dim, page, format};
        const qmv_kv_batch b = {i, i, i, T, B, pages};
        const int64_t ld = int64_t{1} << 30;
        const int rc = attn_paged(&c, &b, p, ld, p, ld, heads * group, 0.1f, window, p, SIZE_MAX, nullptr);
        refused += rc != QMV_OK;
        if (rc != QMV_OK && rc != QMV_ERR_SHAPE) ++failures;
    };
    // few rows, very many sequences and heads: the item count is small and the grid is not
    call(1, 65535, 255, 1, 128, QMV_KV_Q8, 16, 128, 0);
    call(1, 65535, 200, 1, 128, QMV_KV_Q8, 16, 64, 0);
    call(2, 65535, 130, 1, 64, QMV_KV_F16, 16, 64, 0);
    if (eights || planned != 3) ++failures;
    for (int n = 0; n < 2000000; ++n) {
        const bool edge = n % 2;
        const int64_t T = edge ? one_of({1, 2, 15, 16, 17, 512, 65535, (1 << 24) - 1}) : spread((1 << 24) - 1);
        const int B = static_cast<int>(edge ? one_of({1, 2, 63, 64, 65, 256, 257, 32768, 65535}) : spread(65535));
        const int heads = static_cast<int>(edge ? one_of({1, 2, 8, 127, 128, 129, 255, 256, 65535}) : spread(65535));
        const int page = static_cast<int>(one_of({16, 32, 64, 128, 256, 512, 1024}));
        const int pages = static_cast<int>(edge ? one_of({1, 2, 4, 5, 9, 64, (1 << 30) / page}) : spread((1 << 30) / page));
        call(T, B, heads, static_cast<int>(edge ? one_of({1, 2, 3, 16, 64}) : spread(64)),
             static_cast<int>(one_of({64, 128, 256})), static_cast<int>(rng() % 2), page, pages,
             static_cast<int>(edge ? one_of({0, 1, 1024, (int64_t{1} << 31) - 1}) : rng() % 3 ? 0 : spread(1 << 20)));
    }
    if (planned < 100000 || refused < 100000 || eights < 1000 || splits < 1000 || doubles < 1000) ++failures;
    if (failures) {
        std::printf("attention plan driver: %d failures\n", failures);
        return 1;
    }
    std::printf("attention plan driver: ok (%lld planned, %lld of eight waves, %lld split)\n", static_cast<long long>(planned),
                static_cast<long long>(eights), static_cast<long long>(splits));
    return 0;
}
