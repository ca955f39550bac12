// What an attention call launches, decided on the host from the descriptors'
// numbers alone (attn.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/qmv_step.h"

namespace qmv {

constexpr int kAttnWaves = 4;                       // waves of a workgroup, where not eight
constexpr int kTile = 32;                           // keys of one wave's step
constexpr int kAttnStep = kTile * kAttnWaves;       // keys of the workgroup's step
constexpr int kUnitShift = 7;                       // a unit of work is one step (more for huge tables)
constexpr int kWaveThreads = 64;
constexpr size_t kOwnerBytes = 16;                  // of an item's record (split)
// A launch's threads in one dimension fit 32 bits.
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;

// Everything about a call that depends on the descriptors' numbers.
struct AttnPlan {
    int r = 1;             // 16-row tiles of a workgroup
    bool split = true;     // units of keys and a second kernel; else whole items
    int waves = kAttnWaves;  // of a workgroup (whole items)
    int unit_shift = kUnitShift;
    int workgroups = 0;    // of the split
    int64_t tiles = 0;     // numbers of row tiles (first_tile)
    size_t part_bytes = 0, owner_bytes = 0;
    // the launches: the main kernel's and, of the split, the second kernel's
    int64_t blocks(const qmv_kv_cache& c) const { return split ? workgroups : tiles * c.kv_heads; }
    int threads() const { return (split ? kAttnWaves : waves) * kWaveThreads; }
    int64_t join_blocks(const qmv_kv_cache& c) const { return split ? tiles * c.kv_heads : 0; }
};

// Workgroups of one round: two on each of 256 CUs, one where the registers
// allow no more.
constexpr int kRound = 512, kRoundWide = 256;

inline AttnPlan plan_attn(const qmv_kv_cache& c, const qmv_kv_batch& b, int q_heads, int window) {
    AttnPlan p;
    const int64_t group = q_heads / c.kv_heads;
    const int64_t seqs = b.B < b.T ? b.B : b.T;
    // the items that there can be with `rows` rows a tile: sum of
    // ceil(n group / rows) over the sequences, for any split of T rows
    auto items_of = [&](int64_t rows) {
        const int64_t x = b.T * ((group + rows - 1) / rows), y = (b.T * group + seqs * (rows - 1)) / rows;
        return (x < y ? x : y) * c.kv_heads;
    };
    const int round = c.head_dim == 256 ? kRoundWide : kRound;
    const int64_t items = items_of(16);
    // keys of the longest item there can be, and the workgroup's steps over them
    const int64_t keys = static_cast<int64_t>(b.max_pages) * c.page_size;
    const int64_t span = window > 0 && window < keys - 64 ? window + 64 : keys;
    const int64_t steps = (span + kAttnStep - 1) / kAttnStep;
    // Runs of units cost the second kernel and, where items are many, the
    // change from one to the next; whole items cost the wait for the longest.
    // One item a CU, or fewer, take eight waves (two on 64-wide heads, whose
    // registers allow it): 256 items of 9 steps 14.1 us against 18.8 with
    // four, of 17 21.3 against 30.0, but 320 of 9 22.0 against 18.6; 256-wide
    // heads, 256 of 17, 38.5 against 54.0, as float16 (whose registers spill
    // with two waves a SIMD) 129 against 71.
    // Runs / whole with eight waves, us: 16 items of 5 steps 10.9 / 9.6, of 9
    // 11.9 / 12.5, of 17 12.9 / 18.7; 32 of 9 12.2 / 13.1; 128 of 9 19.2 /
    // 13.5, of 17 20.8 / 19.7, of 33 26.9 / 32.1; 256 of 17 29.5 / 21.3, of 33
    // 45.7 / 42.1.  With four: 320 of 9 27.2 / 18.6, of 17 32.0 / 30.5, of 33
    // 52.5 / 62.0; 512 of 17 48.5 / 41.3, of 33 76.0 / 76.6.  Chunks of many
    // rows have many items of one length and stay whole.
    // A tile's number exists for every sequence, one without rows too: with
    // many of these the workgroups of eight waves could pass a launch's limit
    // (those of four cannot: the limit on q_heads is theirs), and stay four.
    const bool chunk = items >= 2 * round && b.T * group >= 64 * seqs;
    const int64_t tiles = b.T * group / 16 + b.B;
    const bool eight = !(c.head_dim == 256 && c.format == QMV_KV_F16) && items <= (c.head_dim == 64 ? 512 : 256) &&
                       tiles * c.kv_heads * 8 * kWaveThreads <= kMaxThreads;
    p.split = !chunk && (eight ? steps * 8 > 36 + items : steps * 20 > 80 + items);
    if (!p.split) {
        // Two row tiles share the keys' and values' loads and conversions.
        // Two prompts of 1024 new tokens over 6000, 8 heads of 128: 260 us
        // against 375-397 us (float16: 298 against 505-516); with fewer items
        // than a round (256 new tokens of one prompt over 2048) 32.8 against
        // 32.3.  In an earlier state of the kernel 64-wide heads took 129 us
        // with two against 126 with one, 256-wide ones 176 against 130
        // (registers), in a smaller case.
        p.r = c.head_dim == 128 && items_of(32) >= kRound && b.T * group >= 64 * seqs ? 2 : 1;
        p.waves = eight && steps > kAttnWaves ? 8 : kAttnWaves;
        p.tiles = b.T * group / (16 * p.r) + b.B;
        return p;
    }
    p.tiles = tiles;
    p.workgroups = round;
    // unit numbers fit 31 bits whatever the lengths
    while (items * ((keys >> p.unit_shift) + 1) >= (int64_t{1} << 31)) ++p.unit_shift;
    p.part_bytes = static_cast<size_t>(2 * p.workgroups) * static_cast<size_t>(16 * (c.head_dim + 2)) * sizeof(float);
    p.owner_bytes = static_cast<size_t>(p.tiles * c.kv_heads) * kOwnerBytes;
    return p;
}

}  // namespace qmv
