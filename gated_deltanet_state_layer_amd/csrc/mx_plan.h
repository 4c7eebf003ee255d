// Which kernels a projection with 4-bit weights launches, by its sizes alone.
// Host code without HIP, so that tests can ask it.
#pragma once
#include <algorithm>
#include <cstdint>

namespace gdn {

constexpr int kMxTileTokens = 128, kMxWorkgroup = 512;   // every kernel has 512 threads
// A launch holds fewer than 2^32 threads.
constexpr int64_t kMxMaxWorkgroups = ((int64_t)1 << 32) / kMxWorkgroup - 1;

// One launch: workgroups of `tokens` by `channels` over the channels [c0, c1).
struct MxLaunch {
    bool tile;   // the tile kernel or the skinny one
    int tokens, channels, c0, c1;
    int64_t workgroups;
};
struct MxPlan {
    MxLaunch launch[2];
    int n;
};

inline int64_t mx_tiles(int64_t n_tok, int64_t n_out, int tt, int cc) {
    return ((n_tok + tt - 1) / tt) * ((n_out + cc - 1) / cc);
}
inline int64_t mx_rounds(int64_t tiles) { return (tiles + 255) / 256; }

inline MxLaunch mx_launch(bool tile, int64_t n_tok, int tokens, int channels, int c0, int c1) {
    return {tile, tokens, channels, c0, c1, mx_tiles(n_tok, c1 - c0, tokens, channels)};
}

// The calls that are taken: 32 tokens by 64 channels, the largest skinny shape,
// are then fewer than 2^23 workgroups.
inline bool mx_proj_fits(int64_t n_tok, int64_t n_out) {
    const int64_t t = n_tok / 64 + 1, c = n_out / 64 + 1;
    return t < (1 << 22) && t * c < (1 << 22);
}

// Times in 1/1024 us, from which a call's kernels are picked.  A round of 256
// skinny workgroups of 32 tokens by 64 channels takes about 2.5 us and 1.6 more
// per 1024 inputs; of tiles about 4 us and, per 1024 inputs, 8.8 (128x128) or
// 12.2 (128x192).  Fitted to 19 token counts of 24 to 8192 for each of eleven
// pairs of 128 to 8192 inputs and 1001 to 16384 channels: what is picked takes
// 0.5 % longer than the fastest way on average, 17 % at worst.
inline int64_t mx_skinny_time(int64_t n_tok, int32_t n_in, int64_t n_out) {
    return mx_rounds(mx_tiles(n_tok, n_out, 32, 64)) * (2560 + (int64_t)n_in * 8 / 5);
}

// Tiles of 128 tokens by `channels` for the channels below n_main.  Where the
// last column of tiles would cost a round for few channels, these are a skinny
// call of their own (500 x 2048 -> 12352: 64 columns in one round and a strip
// 39.0 us, 65 columns in two 61.0).
struct MxTiles {
    int channels, n_main;
    int64_t time;
};
constexpr int kMxTiles[2][2] = {{192, 12 * 1024 + 205}, {128, 8 * 1024 + 819}};

inline MxTiles mx_plan_tiles(int64_t n_tok, int32_t n_in, int64_t n_out) {
    MxTiles best{0, (int)n_out, INT64_MAX};
    for (const auto& t : kMxTiles) {
        const int cc = t[0];
        const int64_t round = 4 * 1024 + (int64_t)n_in * t[1] / 1024;
        const int64_t whole = n_out / cc * cc;
        const int64_t all = mx_rounds(mx_tiles(n_tok, n_out, kMxTileTokens, cc)) * round;
        if (all < best.time) best = {cc, (int)n_out, all};
        if (whole == 0 || whole == n_out || n_in < 128) continue;
        const int64_t strip = mx_rounds(mx_tiles(n_tok, whole, kMxTileTokens, cc)) * round + 2048 +
                              mx_skinny_time(n_tok, n_in, n_out - whole);
        if (strip < best.time) best = {cc, (int)whole, strip};
    }
    return best;
}

// The skinny kernel's shape for a call of its own: by the bytes that the busiest
// CU takes in, the tile's tokens and weights, the measure that separates the
// shapes where the axis is not the limit.
inline MxLaunch mx_plan_skinny(int64_t n_tok, int64_t n_out) {
    constexpr int shapes[][2] = {{4, 16}, {4, 32}, {16, 16}, {16, 32}, {16, 64}, {32, 64}};
    const int first = n_tok <= 4 ? 0 : 2, last = n_tok <= 4 ? 2 : 6;
    int best = first;
    int64_t least = INT64_MAX;
    for (int i = first; i < last; ++i) {
        const int r = shapes[i][0], cc = shapes[i][1];
        const int64_t wgs = mx_tiles(n_tok, n_out, r, cc);
        if (wgs > kMxMaxWorkgroups) continue;
        const int64_t c = mx_rounds(wgs) * (std::min<int64_t>(n_tok, r) * 4 + cc);
        if (c < least) { least = c; best = i; }
    }
    return mx_launch(false, n_tok, shapes[best][0], shapes[best][1], 0, (int)n_out);
}

// The skinny kernel takes the call, or the tile kernel (2048 -> 12352: 96 tokens
// 20.4 against 23.6 us, 128 tokens 26.3 against 23.6; 4096 -> 2048: 1000 tokens
// 34.7 against 42.3 us, 1536 tokens 51.1 against 42.6).
inline MxPlan mx_plan(int64_t n_tok, int32_t n_in, int64_t n_out) {
    const MxTiles t = mx_plan_tiles(n_tok, n_in, n_out);
    if (n_in >= 128 && (n_tok <= 16 || mx_skinny_time(n_tok, n_in, n_out) <= t.time))
        return {{mx_plan_skinny(n_tok, n_out), {}}, 1};
    MxPlan p{{mx_launch(true, n_tok, kMxTileTokens, t.channels, 0, t.n_main), {}}, 1};
    if (t.n_main < n_out) p.launch[p.n++] = mx_launch(false, n_tok, 32, 64, t.n_main, (int)n_out);
    return p;
}

}  // namespace gdn
