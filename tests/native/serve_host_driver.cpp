// Drives the argument checking of qmv_serve.h's entry points (serve_api.cpp)
// under AddressSanitizer and UndefinedBehaviorSanitizer, with the kernel
// launchers replaced by stubs that check the numbers they are given against
// the limits the kernels rely on.  Built and run by
// tests/test_serve_sanitizers.py (host code only, no GPU).
// Every number takes the edges of its type and of its documented range, alone
// and in seeded random combinations: a call either reaches its launcher
// within the limits or returns an error and does not.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "qmv_serve.h"
#include "serve_internal.h"

static int failures = 0;
#define CHECK(cond) do { if (!(cond)) { \
    if (++failures < 20) std::printf("line %d: %s\n", __LINE__, #cond); } } while (0)

namespace {
int64_t g_calls = 0;
constexpr int64_t kRows = (1 << 24) - 1;
}  // namespace

namespace qmv {
size_t plan_ws_bytes(int) { return 4096; }
hipError_t launch_kv_plan(const qmv_kv_pool& p, const PlanArgs& a, void* ws, hipStream_t) {
    ++g_calls;
    CHECK(p.num_pages >= 1 && p.num_pages <= INT_MAX && p.B >= 1 && p.B <= 65535 && p.max_pages >= 1);
    CHECK(p.page_size >= 16 && p.page_size <= 1024 && (p.page_size & (p.page_size - 1)) == 0);
    CHECK(static_cast<__int128>(p.max_pages) * p.page_size <= (1 << 30));
    CHECK(a.T >= 1 && a.T <= kRows && ws && a.kv_len && a.n_new && a.free_count && a.new_len && a.new_count && a.row_start &&
          a.status && p.page_table && p.free_pages);
    CHECK(reinterpret_cast<uintptr_t>(a.slot) % 8 == 0);
    return hipSuccess;
}
hipError_t launch_embed(int fmt, const void*, const int32_t*, float*, int64_t N, int64_t K, int64_t M, float scale,
                        hipStream_t) {
    ++g_calls;
    CHECK(fmt >= 0 && fmt <= 3 && N >= 1 && N <= INT_MAX && M >= 1 && M <= kRows && K >= 1 && K <= INT_MAX);
    CHECK(K % (fmt >= 2 ? 256 : 32) == 0 && scale - scale == 0);
    CHECK(static_cast<__int128>(N) * (K / 32) * 34 <= INT64_MAX && static_cast<__int128>(M) * K * 4 <= INT64_MAX);
    return hipSuccess;
}
size_t lora_ws_bytes(const qmv_lora& l, int64_t B, int64_t T) {
    CHECK(l.max_rank >= 8 && l.max_rank <= 256 && B >= 1 && B <= 65535 && T >= 1 && T <= kRows);
    return 4096;
}
hipError_t launch_lora(const qmv_lora& l, const LoraArgs& a, void* ws, hipStream_t) {
    ++g_calls;
    CHECK(l.format == QMV_LORA_F16 || l.format == QMV_LORA_BF16);
    CHECK(l.K >= 8 && l.K <= kRows && l.K % 8 == 0 && l.N >= 1 && l.N <= kRows && l.slots >= 1 && l.slots < (1 << 20));
    CHECK(l.max_rank >= 8 && l.max_rank <= 256 && l.max_rank % 8 == 0);
    CHECK(static_cast<__int128>(l.slots) * l.max_rank * l.K * 2 <= INT64_MAX);
    CHECK(static_cast<__int128>(l.slots) * l.max_rank * l.N * 2 <= INT64_MAX);
    CHECK(a.B >= 1 && a.B <= 65535 && a.T >= 1 && a.T <= kRows && a.ldx >= l.K && a.ldy >= l.N && ws);
    CHECK(!a.base || a.ldb >= l.N);
    CHECK(a.base != a.y || a.ldb == a.ldy);
    CHECK(static_cast<__int128>(a.ldx) * a.T * 4 <= INT64_MAX && static_cast<__int128>(a.ldy) * a.T * 4 <= INT64_MAX);
    return hipSuccess;
}
size_t draw_ws_bytes(int64_t, int64_t) { return 4096; }
hipError_t launch_logits_draw(const DrawArgs& a, void* ws, hipStream_t) {
    ++g_calls;
    CHECK(a.V >= 1 && a.V <= INT_MAX && a.M >= 1 && a.M <= 65535 && a.ldl >= a.V && ws);
    CHECK(a.softcap >= 0 && a.softcap <= 65536.0f && a.temperature && a.u && a.token);
    CHECK(static_cast<__int128>(a.ldl) * a.M * 4 <= INT64_MAX);
    return hipSuccess;
}
}  // namespace qmv

int main() {
    std::mt19937_64 rng(1);
    const std::vector<int64_t> edges = {0, 1, -1, 7, 8, 12, 15, 16, 17, 24, 31, 32, 100, 255, 256, 257, 264, 1024, 2048, 65535,
                                        65536, (1 << 20) - 1, 1 << 20, (1 << 24) - 1, 1 << 24, 1 << 26, 1 << 30, INT_MAX,
                                        INT_MIN, int64_t{1} << 31, int64_t{1} << 40, int64_t{1} << 61, int64_t{1} << 62,
                                        INT64_MAX, INT64_MIN};
    const std::vector<float> floats = {0.0f, -0.0f, 1.0f, -1.0f, 30.0f, 65536.0f, 65537.0f, 1e-45f, 3.4e38f, -3.4e38f,
                                       __builtin_inff(), -__builtin_inff(), __builtin_nanf("")};
    auto edge = [&] { return edges[rng() % edges.size()]; };
    auto number = [&] { return floats[rng() % floats.size()]; };
    const uintptr_t base = 1 << 20;
    int64_t good = 0, refused = 0;
    for (int round = 0; round < 400000; ++round) {
        // one address in 40 is off or NULL, one number in 4 an edge
        auto at = [&] { const auto r = rng() % 80; return r == 0 ? 0 : r == 1 ? base + 2 : base + 16 * (rng() % 4); };
        auto rare = [&](int64_t usual) { return rng() % 4 == 0 ? edge() : usual; };
        auto rare32 = [&](int32_t usual) { return static_cast<int32_t>(rare(usual)); };
        auto P = [&] { return reinterpret_cast<float*>(at()); };
        auto I = [&] { return reinterpret_cast<int32_t*>(at()); };
        const size_t ws_bytes = rng() % 20 ? 4096 : 4095;
        const int64_t before = g_calls;
        int rc = 0;
        switch (round % 4) {
            case 0: {
                qmv_kv_pool p = {I(), I(), rare(100), rare32(3), rare32(40), rare32(64)};
                const qmv_kv_pool* pp = rng() % 50 ? &p : nullptr;
                const size_t need = kv_plan_ws_bytes(pp);
                rc = kv_plan(pp, I(), I(), I(), I(), I(), I(), I(), I(), reinterpret_cast<int64_t*>(at()), I(), rare(50), P(),
                             ws_bytes, nullptr);
                CHECK(rc != QMV_OK || need == 4096);
                break;
            }
            case 1: {
                auto* f = (round & 4) ? ((round & 8) ? embed_q8_0 : embed_q4_0) : ((round & 8) ? embed_q4_k : embed_q6_k);
                rc = f(P(), I(), P(), rare(1000), rare(512), rare(5), rng() % 2 ? 2.0f : number(), nullptr);
                break;
            }
            case 2: {
                qmv_lora l = {P(), P(), I(), P(), rare(64), rare(100), rare32(4), rare32(16), rare32(static_cast<int>(rng() % 2))};
                const qmv_lora* lp = rng() % 50 ? &l : nullptr;
                const int64_t B = rare(3), T = rare(9);
                const size_t need = lora_add_ws_bytes(lp, B, T);
                rc = lora_add(lp, I(), I(), P(), rare(64), P(), rare(100), P(), rare(100), B, T, P(), ws_bytes, nullptr);
                CHECK(rc != QMV_OK || need == 4096);
                break;
            }
            default: {
                const int64_t V = rare(1000), M = rare(3);
                const size_t need = logits_draw_ws_bytes(V, M);
                rc = logits_draw(P(), rare(1200), P(), I(), P(), P(), P(), I(), I(), V, M, rng() % 2 ? 30.0f : number(), P(),
                                 ws_bytes, nullptr);
                CHECK(rc != QMV_OK || need == 4096);
            }
        }
        CHECK(g_calls - before == (rc == QMV_OK ? 1 : 0));
        ++(rc == QMV_OK ? good : refused);
    }
    CHECK(good > 20000 && refused > 20000);
    if (failures) {
        std::printf("serve host driver: %d failures\n", failures);
        return 1;
    }
    std::printf("serve host driver: ok (%lld accepted, %lld refused)\n", static_cast<long long>(good),
                static_cast<long long>(refused));
    return 0;
}
