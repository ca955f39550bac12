// Drives the argument checking of qmv_step.h's entry points (step_api.cpp)
// under AddressSanitizer and UndefinedBehaviorSanitizer, with the kernel
// launchers replaced by stubs that check the numbers they are given against
// the limits the kernels rely on.  Built and run by
// tests/test_native_sanitizers.py (host code only, no GPU).
// Every number takes the edges of its type and of its documented range, alone
// and in seeded random combinations: a call either reaches its launcher
// within the limits or returns an error and does not.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "qmv_step.h"
#include "step_internal.h"

static int failures = 0;
#define CHECK(cond) do { if (!(cond)) { \
    if (++failures < 20) std::printf("line %d: %s\n", __LINE__, #cond); } } while (0)

namespace {
int64_t g_calls = 0;

void check_kv(const qmv_kv_cache& c, const qmv_kv_batch& b, int64_t ld0, int64_t ld1, int64_t width) {
    ++g_calls;
    CHECK(c.format == QMV_KV_Q8 || c.format == QMV_KV_F16);
    CHECK(c.head_dim == 64 || c.head_dim == 128 || c.head_dim == 256);
    CHECK(c.page_size >= 16 && c.page_size <= 1024 && (c.page_size & (c.page_size - 1)) == 0);
    CHECK(c.kv_heads >= 1 && c.num_pages >= 1 && b.T >= 1 && b.T < (1 << 24) && b.B >= 1 && b.B <= 65535);
    CHECK(b.max_pages >= 1 && static_cast<__int128>(b.max_pages) * c.page_size <= (1 << 30));
    CHECK(static_cast<__int128>(c.num_pages) * c.kv_heads * c.page_size * c.head_dim * 2 <= INT64_MAX);
    CHECK(ld0 >= width && ld1 >= width);
    CHECK(static_cast<__int128>(ld0) * b.T * 4 <= INT64_MAX && static_cast<__int128>(ld1) * b.T * 4 <= INT64_MAX);
}
}  // namespace

size_t qmm_q4_0_q8act_ws_bytes(int64_t N, int64_t K, int64_t M) {
    return N < 1 || K < 1 || K % 32 != 0 || M < 1 || M > 65535 ? 0 : 4096;
}

namespace qmv {
hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_batch& b, const float*, int64_t ldk, const float*,
                           int64_t ldv, hipStream_t) {
    check_kv(c, b, ldk, ldv, static_cast<int64_t>(c.kv_heads) * c.head_dim);
    return hipSuccess;
}
hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_batch& b, float*, int64_t ldk, float*, int64_t ldv,
                          hipStream_t) {
    check_kv(c, b, ldk, ldv, static_cast<int64_t>(c.kv_heads) * c.head_dim);
    return hipSuccess;
}
size_t attn_ws_bytes(const qmv_kv_cache&, const qmv_kv_batch&, int) { return 4096; }
hipError_t launch_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, const float*, int64_t ldq, float*, int64_t ldo,
                       int q_heads, float scale, int window, void*, hipStream_t) {
    check_kv(c, b, ldq, ldo, static_cast<int64_t>(q_heads) * c.head_dim);
    CHECK(q_heads >= 1 && q_heads % c.kv_heads == 0 && q_heads / c.kv_heads <= 64 && window >= 0 && scale - scale == 0);
    CHECK((b.T * (q_heads / c.kv_heads) / 16 + b.B) * c.kv_heads < (1 << 24));
    return hipSuccess;
}
hipError_t launch_rmsnorm(const float*, const float*, const float*, float*, float* y, int8_t* q, float*, int64_t K,
                          int64_t M, float eps, hipStream_t) {
    ++g_calls;
    CHECK((y != nullptr) != (q != nullptr) && K >= 1 && K <= INT_MAX && M >= 1 && M <= 65535 && eps >= 0 && eps - eps == 0);
    CHECK(!q || K % 32 == 0);
    return hipSuccess;
}
hipError_t launch_qmm_q8(const void*, const int8_t*, const float*, float*, int64_t N, int64_t K, int64_t M, void*,
                         hipStream_t) {
    ++g_calls;
    CHECK(qmm_q4_0_q8act_ws_bytes(N, K, M) > 0);
    return hipSuccess;
}
size_t draft_ws_bytes(int64_t, int, int64_t) { return 4096; }
hipError_t launch_draft_verify(const DraftArgs& a, void*, hipStream_t) {
    ++g_calls;
    CHECK(a.B >= 1 && a.B <= 65535 && a.G >= 1 && a.G <= 64 && a.V >= 1 && a.V <= INT_MAX);
    CHECK(a.ldt >= a.V && a.ldd >= a.V && a.temperature > 0 && a.temperature - a.temperature == 0);
    CHECK(a.softcap >= 0 && a.softcap <= 65536.0f);
    CHECK(static_cast<__int128>(a.ldt) * a.B * (a.G + 1) * 4 <= INT64_MAX);
    CHECK(static_cast<__int128>(a.ldd) * a.B * a.G * 4 <= INT64_MAX);
    return hipSuccess;
}
}  // namespace qmv

int main() {
    std::mt19937_64 rng(1);
    const std::vector<int64_t> edges = {0, 1, -1, 2, 15, 16, 17, 31, 32, 64, 65, 100, 127, 128, 255, 256, 1023, 1024, 1025,
                                        2048, 65535, 65536, (1 << 24) - 1, 1 << 24, 1 << 30, INT_MAX, INT_MIN,
                                        int64_t{1} << 31, int64_t{1} << 40, int64_t{1} << 61, int64_t{1} << 62, INT64_MAX,
                                        INT64_MIN};
    const std::vector<float> floats = {0.0f, -0.0f, 1.0f, -1.0f, 30.0f, 65536.0f, 65537.0f, 1e-45f, 3.4e38f, -3.4e38f,
                                       __builtin_inff(), -__builtin_inff(), __builtin_nanf("")};
    auto edge = [&] { return edges[rng() % edges.size()]; };
    auto edge32 = [&] { return static_cast<int32_t>(edge()); };
    auto number = [&] { return floats[rng() % floats.size()]; };
    const uintptr_t base = 1 << 20;
    int64_t good = 0, refused = 0;
    for (int round = 0; round < 400000; ++round) {
        // one address in 40 is off or NULL, one number in 4 an edge
        auto at = [&](uintptr_t) { const auto r = rng() % 80; return r == 0 ? 0 : r == 1 ? base + 2 : base; };
        auto rare = [&](int64_t usual) { return rng() % 4 == 0 ? edge() : usual; };
        auto rare32 = [&](int32_t usual) { return rng() % 4 == 0 ? edge32() : usual; };
        auto P = [&] { return reinterpret_cast<float*>(at(0)); };
        auto I = [&] { return reinterpret_cast<int32_t*>(at(0)); };
        const bool q8 = rng() % 2;
        qmv_kv_cache c = {P(), P(), q8 ? P() : nullptr, q8 ? P() : nullptr, rare(100), rare32(4), rare32(128), rare32(64),
                          rare32(q8 ? QMV_KV_Q8 : QMV_KV_F16)};
        qmv_kv_batch b = {I(), I(), I(), rare(7), rare32(3), rare32(40)};
        const qmv_kv_cache* cp = rng() % 50 ? &c : nullptr;
        const qmv_kv_batch* bp = rng() % 50 ? &b : nullptr;
        const float eps = rng() % 2 ? 1e-6f : number();
        const int64_t before = g_calls;
        int rc = 0;
        switch (round % 8) {
            case 0: rc = kv_write(cp, bp, P(), rare(512), P(), rare(600), nullptr); break;
            case 1: rc = kv_read(cp, bp, P(), rare(512), P(), rare(600), nullptr); break;
            case 2: {
                const int32_t heads = rare32(8);
                const size_t need = attn_paged_ws_bytes(cp, bp, heads);
                rc = attn_paged(cp, bp, P(), rare(1024), P(), rare(2000), heads, rng() % 2 ? 0.1f : number(), rare32(0),
                                P(), rng() % 20 ? 4096 : 4095, nullptr);
                CHECK(rc != QMV_OK || need == 4096);
                break;
            }
            case 3: rc = rmsnorm_add(P(), P(), P(), P(), P(), rare(5376), rare(9), eps, nullptr); break;
            case 4: rc = rmsnorm_add_q8(P(), P(), P(), P(), reinterpret_cast<int8_t*>(at(0)), P(), rare(5376), rare(9), eps,
                                        nullptr); break;
            case 5: rc = qmm_q4_0_q8(P(), reinterpret_cast<int8_t*>(at(0)), P(), P(), rare(300), rare(256), rare(4), P(),
                                     rng() % 20 ? 4096 : 4095, nullptr); break;
            default: {
                const int64_t V = rare(1000), B = rare(3);
                const int32_t G = rare32(4);
                const size_t need = draft_verify_ws_bytes(B, G, V);
                rc = draft_verify(P(), rare(1000), P(), rare(1200), I(), I(), P(), I(), I(), B, G, V,
                                  rng() % 2 ? 0.8f : number(), rng() % 2 ? 30.0f : number(), P(), rng() % 20 ? 4096 : 4095,
                                  nullptr);
                CHECK(rc != QMV_OK || need == 4096);
            }
        }
        CHECK(g_calls - before == (rc == QMV_OK ? 1 : 0));
        ++(rc == QMV_OK ? good : refused);
    }
    CHECK(good > 20000 && refused > 20000);
    if (failures) {
        std::printf("step host driver: %d failures\n", failures);
        return 1;
    }
    std::printf("step host driver: ok (%lld accepted, %lld refused)\n", static_cast<long long>(good),
                static_cast<long long>(refused));
    return 0;
}
