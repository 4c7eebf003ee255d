// Projections with 4-bit weights: y = x W^T, x bf16, W in the format of
// mx_format.hip, fp32 accumulation on the matrix cores.
//
// Few tokens are bound by the weights' bytes and one trip to memory, many by
// the matrix units' feed.  A code times its scale is exact in bf16, so codes are
// expanded in registers and multiplied in bf16: products are exact and sums
// hold 32 bits.  The scaled matrix instructions would take codes as they are
// beside tokens in two 8-bit parts, at the same matrix cycles (8192 x 2048 ->
// 12352 338 us against 496), but drop what lies 2^-13 below the largest product
// of a group: next to one value 2^16 above the others, 88 % of the bf16 results
// came out wrong.
#include <algorithm>
#include <type_traits>

#include "gdn_common.h"
#include "lds_load.h"
#include "mfma_split.h"
#include "mx_plan.h"

namespace gdn {
namespace {

// Where the output channels go: [0, end[0]) to seg[0], [end[0], end[1]) to
// seg[1], and so on, ld elements between tokens; from end[3] on, fp32 gates a
// and b of h_v channels each.  A plain projection has one segment.
struct MxOut {
    void* seg[4];
    int64_t ld[4];
    int end[4];
    float *a, *b;
    int h_v, n_out;
    int vec4, vec16;   // segment starts, strides and ends are multiples of 4 elements / 16 bytes
};

// The segments' values are picked lane by lane: an index would read them from
// memory again.
template <typename T>
__device__ __forceinline__ T* mx_at(const MxOut& o, int64_t t, int n) {
    void* p = o.seg[0];
    int64_t ld = o.ld[0];
    int base = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const bool past = n >= o.end[i];
        p = past ? o.seg[i + 1] : p;
        ld = past ? o.ld[i + 1] : ld;
        base = past ? o.end[i] : base;
    }
    return static_cast<T*>(p) + t * ld + n - base;
}

template <typename T>
__device__ __forceinline__ void mx_put(const MxOut& o, int64_t t, int n, float y) {
    if (n < o.end[3]) {
        Io<T>::store(mx_at<T>(o, t, n), 0, y);
        return;
    }
    const int g = n - o.end[3];
    const bool is_b = g >= o.h_v;
    (is_b ? o.b - o.h_v : o.a)[t * o.h_v + g] = 1.0f / (1.0f + expf(is_b ? -y : y));
}

__device__ __forceinline__ u32x2 pack4(f32x4 y) {
    return u32x2{f32_to_bf16(y[0]) | (uint32_t)f32_to_bf16(y[1]) << 16,
                 f32_to_bf16(y[2]) | (uint32_t)f32_to_bf16(y[3]) << 16};
}

// Channels n .. n+3 (n a multiple of four) of token t.
template <typename T>
__device__ __forceinline__ void mx_put4(const MxOut& o, int64_t t, int n, f32x4 y) {
    if (o.vec4 && n < o.end[3]) {
        T* p = mx_at<T>(o, t, n);
        if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2*>(p) = pack4(y);
        else *reinterpret_cast<f32x4*>(p) = y;
        return;
    }
    const int end = min(4, o.n_out - n);
#pragma unroll 1
    for (int i = 0; i < end; ++i) {
        mx_put<T>(o, t, n + i, y[0]);
        y = f32x4{y[1], y[2], y[3], 0.f};
    }
}

// Eight codes (one register) times their group's scale, in bf16.  A weight
// (code times a power of two) is exact in bf16, so products with bf16 tokens
// are exact in fp32.
__device__ __forceinline__ bf16x8 mx_expand(uint32_t c, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// A low-rank adapter per token beside the weights: token t's h[t] (scale x A^T of
// its adapter, in three bf16 pieces by blocks of 16 ranks: see lora.hip) times the
// rows of its adapter's B is added to the sums.  MxNoLora: none, and no code for it.
// In-projections 2048 -> 12352 at rank 16, without adapters and with, of the h before
// them: 1 token 4.5 and 7.3 us, 64 tokens with one each 9.8 and 16.7 (25 MB of B),
// 500 tokens with eight in runs 40 and 49, 8192 tokens 476 and 502 (526 at rank 32).
struct MxLora {
    const uint16_t* h;   // [n_tok][blocks][3][16]
    const uint16_t* b;   // [n_adapters][n_out][rank]
    const int32_t* ids;  // [n_tok]
    int n_adapters, rank, blocks;
};
// The same for so little work that every workgroup makes its own h, from A in the L2
// caches, and the call is one launch.  Two launches and one: 1 x 4096 -> 2048 at rank
// 16 6.7 and 6.1 us (from Python 11.5 and 8.8), 1 x 2048 -> 12352 7.0 and 7.3 (11.4 and
// 8.7), 4 x 1024 -> 1024 6.0 and 6.1; past the limit 1 x 4096 -> 2048 at rank 32 7.2
// and 8.0, 2 x 4096 -> 4096 6.9 and 8.5.
struct MxLoraHere {
    static constexpr int kTokens = 4, kBlocks = 2;
    static bool takes(int64_t n_tok, int n_in, int blocks) {
        return n_tok <= kTokens && blocks <= kBlocks && n_tok * blocks * n_in <= 4096;
    }
    const uint16_t *a, *b;   // [n_adapters][rank][n_in], [n_adapters][n_out][rank]
    const float* scale;
    const int32_t* ids;
    int n_adapters, rank, blocks;
};
struct MxNoLora {
    MxNoLora() = default;
    __device__ __forceinline__ MxNoLora(const MxNoLora&, int64_t, int) {}
};
// Up to this rank the first adapter's rows of B have LDS of their own in the tile
// kernel, at most 24 KiB beside the stages, and arrive during the main loop; else they
// go into the stages behind it (8192 tokens at rank 16, one adapter 504 us for 511).
constexpr int kLoraAhead = 64;
__device__ __forceinline__ int lora_ranks(const MxLora& l) { return l.rank; }
__device__ __forceinline__ int lora_ranks(const MxNoLora&) { return 0; }

__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(high_bf16(a[i]), high_bf16(b[i]), fmaf(low_bf16(a[i]), low_bf16(b[i]), s));
    return s;
}

// A thread's part of what token t's adapter adds to a tile's 16 NC channels: thread j
// of the token's TPT takes half the ranks of each 16, and channels i TPT / 2 + j / 2,
// so that neighbouring lanes read B side by side.  G blocks of 16 ranks at a time, of
// 16 / G channels: a row's 32 G bytes are one thread's loads behind each other, and
// come as one line (64 tokens with an adapter each, 2048 -> 12352: at rank 64 45 us for
// 66 with 16 ranks of all channels first, 32 tokens 21 for 32).
template <int TPT, int E, int G>
__device__ __forceinline__ void lora_share(const MxLora& l, const uint16_t* h, const uint16_t* b, int ranks, int j,
                                           int last, float (&y)[E]) {
    constexpr int C = E < 16 / G ? E : 16 / G;
    static_assert(E % C == 0, "whole groups of channels");
    float v[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        u32x4 p[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
            p[i] = 16 * g < ranks ? *reinterpret_cast<const u32x4*>(h + 48 * g + 16 * i) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // the pieces' sum is exact
            v[g][2 * k] = low_bf16(p[0][k]) + (low_bf16(p[1][k]) + low_bf16(p[2][k]));
            v[g][2 * k + 1] = high_bf16(p[0][k]) + (high_bf16(p[1][k]) + high_bf16(p[2][k]));
        }
    }
#pragma unroll
    for (int i0 = 0; i0 < E; i0 += C) {
        u32x4 w[C][G];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g)
                w[i][g] = 16 * g < ranks ? *reinterpret_cast<const u32x4*>(
                                               b + min((i0 + i) * (TPT / 2) + j / 2, last) * l.rank + 16 * g)
                                         : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < C; ++i)
                    y[i0 + i] = fmaf(high_bf16(w[i][g][k]), v[g][2 * k + 1],
                                     fmaf(low_bf16(w[i][g][k]), v[g][2 * k], y[i0 + i]));
        __builtin_amdgcn_sched_barrier(0);   // one group's loads in registers at a time
    }
}

template <int TPT, int E>
__device__ __forceinline__ void lora_share(const MxLora& l, int64_t t, int n0, int n_out, int j, float (&y)[E]) {
    const int id = l.ids[t];
    if ((unsigned)id >= (unsigned)l.n_adapters) return;
    const int r0 = 8 * (j & 1), last = n_out - 1 - n0;   // rows past the end repeat the last one
    const uint16_t* b = l.b + ((int64_t)id * n_out + n0) * l.rank + r0;
    const uint16_t* h = l.h + t * l.blocks * 48 + r0;
    constexpr int kMost = E > 8 ? 2 : 4;   // four of 16 channels each spill
    if (l.blocks == 1) {
        lora_share<TPT, E, 1>(l, h, b, l.rank - r0, j, last, y);
    } else if (l.blocks == 2) {
        lora_share<TPT, E, 2>(l, h, b, l.rank - r0, j, last, y);
    } else {
#pragma unroll 1
        for (int r = 0; r < l.rank; r += 16 * kMost)
            lora_share<TPT, E, kMost>(l, h + 3 * r, b + r, l.rank - r0 - r, j, last, y);
    }
}

// h of a workgroup's few tokens and the thread's part of the rows of B (see lora_share).
struct LoraHere {
    u32x4 w[MxLoraHere::kBlocks];
    __device__ __forceinline__ static float* h() {   // [token][rank]
        __shared__ float v[MxLoraHere::kTokens * MxLoraHere::kBlocks * 16];
        return v;
    }
    __device__ __forceinline__ void load(const MxLoraHere& l, bool in, int t, int row, int n_out, int j) {
        const int id = in ? l.ids[t] : -1;
#pragma unroll
        for (int k = 0; k < MxLoraHere::kBlocks; ++k) {
            const int r = 16 * k + 8 * (j & 1);
            w[k] = u32x4{0u, 0u, 0u, 0u};
            if ((unsigned)id < (unsigned)l.n_adapters && r < l.rank)
                w[k] = *reinterpret_cast<const u32x4*>(l.b + ((int64_t)id * n_out + row) * l.rank + r);
        }
    }
    // Two ranks of every 16 to a wave.  Two steps at a time: of four at a time, which all
    // workgroups read at once, 1 x 4096 -> 2048 takes 7.2 us for 6.1.
    __device__ __forceinline__ void shrink(const MxLoraHere& l, const uint16_t* x, int64_t ld_x, int n_in, int toks,
                                           int wave) {
        const int lane = threadIdx.x & 63;
        for (int i = 0; i < toks * l.blocks; ++i) {
            const int t = i / l.blocks, r = i % l.blocks * 16 + wave;
            const int id = l.ids[t];
            float s0 = 0.f, s1 = 0.f;
            if ((unsigned)id < (unsigned)l.n_adapters) {
                // ranks are a multiple of 8: the first of the two is there for every wave or for none
                const uint16_t* a = l.a + ((int64_t)id * l.rank + r) * n_in;
                const bool second = r + 8 < l.rank;
                const uint16_t* a1 = second ? a + 8 * (int64_t)n_in : a;
#pragma unroll 2
                for (int c = lane * 8; c < n_in; c += 512) {
                    const u32x4 v = *reinterpret_cast<const u32x4*>(x + t * ld_x + c);
                    s0 = dot8(v, *reinterpret_cast<const u32x4*>(a + c), s0);
                    s1 = dot8(v, *reinterpret_cast<const u32x4*>(a1 + c), s1);
                }
                s0 = l.scale[id] * wave_sum(s0);
                s1 = second ? l.scale[id] * wave_sum(s1) : 0.f;
            }
            if (lane == 0) {
                h()[i * 16 + wave] = s0;
                h()[i * 16 + wave + 8] = s1;
            }
        }
    }
    // Behind a barrier.
    __device__ __forceinline__ float expand(const MxLoraHere& l, int t, int j) const {
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < MxLoraHere::kBlocks; ++k) {
            if (k >= l.blocks) continue;
            const float* v = h() + (t * l.blocks + k) * 16 + 8 * (j & 1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y = fmaf(high_bf16(w[k][i]), v[2 * i + 1], fmaf(low_bf16(w[k][i]), v[2 * i], y));
        }
        return y;
    }
};

struct MxIn {
    const uint16_t* x;
    const uint8_t *codes, *scales;
    int64_t n_tok, ld_x;
    int n_in, n_out;
};

// Few tokens, and a strip of channels that the tile kernel leaves.  One
// workgroup of 8 waves per R tokens and 16 NC channels; each wave multiplies
// the whole tile over its eighth of the input axis, in steps of 128, and the
// eight partial tiles are added in LDS.  Operands go through LDS of the wave's
// own (no barrier), D steps ahead, by loads that store straight into it: they
// read rows in whole pieces of 64 and 256 bytes from neighbouring lanes, where
// loads in the matrix operands' layout would take every lane's 16 bytes from
// another row, at a quarter of the rate.  Lane l = 16 q + m holds row m's group
// q of a step; MFMA j of the four (16x16x32) takes values 8j .. 8j+7 of all
// four groups, so one scale serves a lane's four.  W is the A operand: a lane's
// four results are consecutive channels of one token.  With R = 4 the tokens'
// lanes repeat, and what repeats is left out at the end.  A row's last step may
// reach past it: its tokens read zeros there and its scales are 0, so whatever
// the codes are adds nothing.  At least four groups of 32 (the scale bytes of a
// step come as one word).  One token 2048 -> 12352 5.7 us (13.4 MB of weights at
// 5.0 TB/s would take 2.7, a launch takes 1.9), 64 tokens 4096 -> 2048 5.9 us;
// operand-order loads 7.7 and 9.8.  D = 1 where two steps do not fit: 32 tokens
// by 64 channels of LDS would be 192 KiB; 64 by 64 take all 160 with one.
constexpr int kSkinnyThreads = kMxWorkgroup, kSkinnyWaves = kSkinnyThreads / 64;

template <int R, int NC, int D>
struct SkinnyShape {
    static constexpr int NT = (R + 15) / 16, XL = R / 4, kW = NC * 1024, kStage = kW + R * 256;
    static constexpr int LD = 16 * NC + 4;
    static constexpr int kLoads = kSkinnyWaves * D * kStage, kSums = kSkinnyWaves * R * LD * 4;
    static constexpr int kBytes = kLoads > kSums ? kLoads : kSums;
    static constexpr int kLoraSums = kSums + R * LD * 4, kLoraBytes = kLoads > kLoraSums ? kLoads : kLoraSums;
    static constexpr int kAhead = (D - 1) * (1 + NC + XL);   // loads of the steps behind the present one
    static_assert((R == 4 || R % 16 == 0) && NC <= 4 && D <= 2 && kAhead < 64, "the schedule");
};

template <typename T, int R, int NC, int D, typename L>
__global__ __launch_bounds__(kSkinnyThreads, 2) void mx_skinny_kernel(MxIn p, MxOut o, int c0, int cols, L lora) {
    using S = SkinnyShape<R, NC, D>;
    constexpr int NT = S::NT;
    extern __shared__ __align__(16) uint8_t lds[];
    const int64_t t0 = (int64_t)(blockIdx.x / cols) * R;
    const int n0 = c0 + (int)(blockIdx.x % cols) * (16 * NC);
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int toks = (int)min((int64_t)R, p.n_tok - t0), rows = min(16 * NC, p.n_out - n0);
    const int half = p.n_in / 2, groups = p.n_in / 32;
    const int steps = (groups + 3) / 4, per = (steps + kSkinnyWaves - 1) / kSkinnyWaves;
    const int s_begin = wave * per, s_end = min(steps, s_begin + per);
    const auto x_rs = buf_rsrc(p.x + t0 * p.ld_x, ((toks - 1) * p.ld_x + p.n_in) * 2);
    const auto w_rs = buf_rsrc(p.codes + (int64_t)n0 * half, (int64_t)rows * half);
    // Slot s of a token's 16 holds chunk s ^ row % 16, of a weight row's four
    // chunk s ^ (row / 4) % 4, so the 16 rows of a fragment read spread over all
    // banks.
    int wo[NC], xo[S::XL], xchunk[S::XL];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int r = c * 16 + (lane >> 2);
        wo[c] = offset_if(r < rows, r * half + ((lane & 3) ^ ((r >> 2) & 3)) * 16);
    }
#pragma unroll
    for (int i = 0; i < S::XL; ++i) {
        const int r = i * 4 + q;
        xchunk[i] = m ^ (r & 15);
        xo[i] = offset_if(r < toks, (int)(r * p.ld_x) * 2 + xchunk[i] * 16);
    }
    // The scale bytes of groups 4 st .. 4 st + 3 of row `lane`, the first lowest.
    // The load may be unaligned; where the row ends inside the four it starts
    // earlier, by past() bytes that are shifted out once it has arrived.
    const auto past = [&](int st) { return max(0, st * 4 + 4 - groups); };
    const uint8_t* sc = p.scales + (int64_t)n0 * groups;
    const uint32_t so = (uint32_t)min(lane, rows - 1) * (uint32_t)groups;
    uint8_t* mine = lds + wave * (D * S::kStage);
    uint32_t ss[D];
    const auto fetch = [&](int st, int b) {
        uint8_t* base = mine + b * S::kStage;
        __builtin_memcpy(&ss[b], sc + (st * 4 - past(st)) + so, 4);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < NC; ++c) load_lds16(w_rs, base + c * 1024, wo[c], st * 64);
#pragma unroll
        for (int i = 0; i < S::XL; ++i)
            load_lds16(x_rs, base + S::kW + i * 1024, offset_if(st * 128 + xchunk[i] * 8 < p.n_in, xo[i]), st * 256);
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 acc[NT][NC];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int mx = m & (R < 16 ? R - 1 : 15);
    const int w_at = m * 64 + ((q ^ (m >> 2)) & 3) * 16, x_at = S::kW + mx * 256;
    const auto step = [&](int st, int b) __attribute__((always_inline)) {
        constexpr int kVm0 = 0x0f70, kVmAhead = 0x0f70 | (S::kAhead & 15) | (S::kAhead >> 4) << 14;
        if (st + D - 1 < s_end) __builtin_amdgcn_s_waitcnt(kVmAhead);
        else __builtin_amdgcn_s_waitcnt(kVm0);
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t* base = mine + b * S::kStage;
        const uint32_t s = ss[b] >> (8 * past(st));
        u32x4 w[NC], x[NT][4];
#pragma unroll
        for (int c = 0; c < NC; ++c) w[c] = *reinterpret_cast<const u32x4*>(base + c * 1024 + w_at);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[t][j] = *reinterpret_cast<const u32x4*>(base + t * 4096 + x_at + ((q * 4 + j) ^ mx) * 16);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint32_t sr = (uint32_t)__builtin_amdgcn_ds_bpermute((c * 16 + m) * 4, (int)s);
            const float scale = __uint_as_float((sr >> (8 * q) & 0xffu) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 wf = mx_expand(w[c][j], scale);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        wf, __builtin_bit_cast(bf16x8, x[t][j]), acc[t][c], 0, 0, 0);
            }
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): the stage is read
        __builtin_amdgcn_sched_barrier(0);
        if (st + D < s_end) fetch(st + D, b);
    };
#pragma unroll
    for (int i = 0; i < D; ++i)
        if (s_begin + i < s_end) fetch(s_begin + i, i);
    // The adapters' share, while the first steps arrive: every thread has a token.
    constexpr bool kHere = std::is_same_v<L, MxLoraHere>, kLora = std::is_same_v<L, MxLora> || kHere;
    constexpr int kPerToken = kSkinnyThreads / R, kShare = (32 * NC + kPerToken - 1) / kPerToken;
    const int share_t = threadIdx.x / kPerToken, share_j = threadIdx.x % kPerToken;
    const bool share_in = share_t < toks && share_j < 32 * NC;
    [[maybe_unused]] float share[kShare] = {};
    [[maybe_unused]] std::conditional_t<kHere, LoraHere, MxNoLora> here;
    if constexpr (kHere) {
        static_assert(R == MxLoraHere::kTokens && kShare == 1, "a thread has half a row of B");
        here.load(lora, share_in, (int)t0 + share_t, n0 + min(share_j / 2, rows - 1), p.n_out, share_j);
        here.shrink(lora, p.x, p.ld_x, p.n_in, toks, wave);
    } else if constexpr (kLora) {
        if (share_in) lora_share<kPerToken>(lora, t0 + share_t, n0, p.n_out, share_j, share);
    }
#pragma unroll 1
    for (int st = s_begin; st < s_end; st += D) {
        step(st, 0);
        if constexpr (D == 2)
            if (st + 1 < s_end) step(st + 1, 1);
    }
    __syncthreads();   // every wave is done with its stages
    float* red = reinterpret_cast<float*>(lds);   // [8 waves][R tokens][16 NC + 4 channels]
    if (R >= 16 || m < R)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<f32x4*>(&red[(wave * R + t * 16 + m) * S::LD + c * 16 + 4 * q]) = acc[t][c];
    if constexpr (kHere) share[0] = here.expand(lora, share_t, share_j);
    if constexpr (kLora) {
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            const float both = group_sum<2>(share[i]);
            if (share_in && !(share_j & 1))
                red[(kSkinnyWaves * R + share_t) * S::LD + i * (kPerToken / 2) + share_j / 2] = both;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < R * 4 * NC; i += kSkinnyThreads) {
        const int t = i / (4 * NC), c = (i % (4 * NC)) * 4;
        if (t >= toks || n0 + c >= p.n_out) continue;
        f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kSkinnyWaves + (kLora ? 1 : 0); ++w)
            y += *reinterpret_cast<const f32x4*>(&red[(w * R + t) * S::LD + c]);
        mx_put4<T>(o, t0 + t, n0 + c, y);
    }
}

// Many tokens.  Eight waves, four along the tokens and two along the channels,
// each 32 tokens x 16 NC channels, so a tile of 128 tokens x CC channels per
// workgroup.  The input axis goes by in blocks of 64 through LDS, written by
// loads that store straight into LDS: the tokens' 128 bytes of a block through
// four stages, the weights' 64 bytes of a pair of blocks, codes as they are,
// through three.  The four scale bytes of a pair go through a register to a
// two-stage area ordered so that a lane reads those of its rows side by side.
// Lane q of MFMA j (16x16x32) takes k = 16 q + 8 j ..: one 8-byte read of codes
// serves both MFMAs, expanded in registers.
//
// A wave keeps its tokens' fragments of a block in registers and takes its
// channels in two halves, all of a half times one token fragment after the
// other; the next half's codes arrive meanwhile.  The block's one barrier
// stands between the halves.  It says that the next block has arrived and this
// one's stage is read out, to be filled with the block four ahead.  Behind it
// the next block's token fragments are read into a second set of registers.
//
// Expanding codes bounds the kernel: each expansion serves two token fragments,
// and the vector units are busy 44 % of the cycles, the matrix units 34 %, at two
// waves a SIMD.  8192 x 2048 -> 12288 in 128x192 tiles 480 us, 0.86 PFLOP/s; 4096
// x 4096 -> 2048 in 128x128 ones 81 us, 0.85.  The shapes divide by rounds: see
// the rule.  With 256x256 a wave's expanded codes do not fit its registers.
constexpr int kTileTokens = kMxTileTokens, kTileThreads = kMxWorkgroup, kStages = 4, kWeightStages = 3;

template <int NC>
struct TileShape {
    static constexpr int NT = 2, WC = 2, CC = 16 * NC * WC, WAVES = 8;
    static constexpr int XL = kTileTokens / 8 / WAVES;             // loads per wave and block
    static constexpr int WL = (CC / 16 + WAVES - 1) / WAVES;       // loads per wave and pair
    static constexpr int kX = kTileTokens * 128, kW = WL * WAVES * 1024, kWeights = kStages * kX;
    static constexpr int HC = NC / 2, HP = HC <= 2 ? 2 : 4;        // channels of a half; their scale words' places
    static constexpr int kWS = WC * 16 * 2 * HP * 4;
    static constexpr int kScale = kWeights + kWeightStages * kW, kBytes = kScale + 2 * kWS;
    static_assert(NC % 2 == 0 && CC % 64 == 0 && CC <= 256, "halves; a scale word per thread of whole waves");
    static_assert(WL + (kStages - 1) * XL < 16, "the schedule");
    // the epilogue's rows (fp32, 16 bytes apart) in the stages
    static constexpr int kRow = 16 * NC * 4 + 16;
    static_assert(WAVES * 16 * kRow <= kScale && kBytes <= 160 * 1024, "fits");
};

// The adapters among a tile's tokens, one after the other.  Every wave holds all the
// tile's ids, two to a lane, and so comes to the same order by itself.
struct LoraOrder {
    int id[2];
    uint64_t left[2];
    __device__ __forceinline__ LoraOrder(const MxLora& l, int64_t t0, int toks) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < 2; ++i) id[i] = i * 64 + lane < toks ? l.ids[t0 + i * 64 + lane] : -1;
#pragma unroll
        for (int i = 0; i < 2; ++i) left[i] = __ballot((unsigned)id[i] < (unsigned)l.n_adapters);
    }
    // The next adapter, -1 behind the last.
    __device__ __forceinline__ int next() {
        if (!(left[0] | left[1])) return -1;
        const int cur = left[0] ? __builtin_amdgcn_readlane(id[0], __builtin_ctzll(left[0]))
                                : __builtin_amdgcn_readlane(id[1], __builtin_ctzll(left[1]));
#pragma unroll
        for (int i = 0; i < 2; ++i) left[i] &= ~__ballot(id[i] == cur);
        return cur;
    }
};

// An adapter's rows of B for a tile's channels into LDS, as they lie; zeros past the
// last row.
__device__ __forceinline__ void lora_stage(const MxLora& l, int cur, int n0, int n_out, int rows, int channels,
                                           uint8_t* dst) {
    const auto rs = buf_rsrc(l.b + ((int64_t)cur * n_out + n0) * l.rank, (int64_t)rows * l.rank * 2);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int loads = channels * l.rank / 512;   // of 1 KiB; channels are a multiple of 64
    for (int i = wave; i < loads; i += kMxWorkgroup / 64) load_lds16(rs, dst + i * 1024, i * 1024 + lane * 16, 0);
}

// The pieces of h of a wave's tokens for 16 ranks, the first two pieces as one operand
// and the third as another.  Tokens without an adapter bring what lies there.
template <int NT>
struct LoraPieces {
    u32x4 v[NT][2];
    __device__ __forceinline__ void load(const MxLora& l, int64_t t0, int64_t n_tok, int k) {
        const int m = threadIdx.x & 15, q = threadIdx.x >> 4 & 3;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint16_t* h = l.h + (min(t0 + t * 16 + m, n_tok - 1) * l.blocks + k) * 48;
            v[t][0] = *reinterpret_cast<const u32x4*>(h + 8 * q);
            const u32x4 third = *reinterpret_cast<const u32x4*>(h + 32 + 8 * (q & 1));
            v[t][1] = q < 2 ? third : u32x4{0u, 0u, 0u, 0u};
        }
    }
};

// Adds adapter cur's share to the sums of a wave's 16 NT tokens by 16 NC channels:
// lane (q, m) holds channels c * 16 + 4q .. of token m of each 16.  Sixteen ranks are
// two MFMAs of 32 beside the same rows of B.  A token takes its own adapter's alone,
// summed apart from the others', so that its result does not depend on theirs.  (As
// what the sums begin with, the first adapter's share would make it depend.)
template <int NT, int NC>
__device__ __forceinline__ void lora_add(const MxLora& l, int cur, const int (&ids)[NT], int64_t t0, int64_t n_tok,
                                         const LoraPieces<NT>& first, const uint8_t* b, f32x4 (&acc)[NT][NC]) {
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    bool any = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) any |= __any(ids[t] == cur);
    if (!any) return;
    f32x4 d[NT][NC];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) d[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    LoraPieces<NT> h = first;
    for (int k = 0; k < l.blocks; ++k) {
        const LoraPieces<NT> now = h;
        if (k + 1 < l.blocks) h.load(l, t0, n_tok, k + 1);
        const bool in = 16 * k + 8 * (q & 1) < l.rank;
        u32x4 w[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(b + (c * 16 + m) * l.rank * 2 + (in ? 32 * k + 16 * (q & 1) : 0));
            w[c] = in ? v : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    d[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[c]),
                                                                      __builtin_bit_cast(bf16x8, now.v[t][j]), d[t][c],
                                                                      0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][c][j] = ids[t] == cur ? acc[t][c][j] + d[t][c][j] : acc[t][c][j];
}

template <typename T, int NC, typename L>
__global__ __launch_bounds__(kTileThreads, 2) void mx_tile_kernel(MxIn p, MxOut o, int tiles_t, int n_end, L lora) {
    using S = TileShape<NC>;
    constexpr int NT = S::NT;
    constexpr bool kLora = std::is_same_v<L, MxLora>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wt = wave / S::WC, wc = wave % S::WC;
    // Consecutive tiles share their channels.  Workgroups go to the eight XCDs
    // in turn: with up to eight tiles along the tokens each XCD takes a run of
    // tiles, so that it reads the run's weights into its own cache once (2048 ->
    // 12352: 500 tokens 39.3 us in turn, 38.2 in runs, 1000 tokens 69.7 and 66.1);
    // with more, every eighth shares its tokens (4096 -> 4096: 4096 tokens 155.0
    // us in turn, 171.7 in runs; at 16 tiles either may win by 3 %).
    unsigned idx = blockIdx.x;
    if (tiles_t <= 8) {
        const unsigned xcd = idx % 8, per = gridDim.x / 8, rest = gridDim.x % 8;
        idx = xcd * per + min(xcd, rest) + idx / 8;
    }
    const int64_t t0 = (int64_t)(idx % tiles_t) * kTileTokens;
    const int n0 = (int)(idx / tiles_t) * S::CC;
    const int toks = (int)min((int64_t)kTileTokens, p.n_tok - t0), rows = min(S::CC, n_end - n0);
    const int half = p.n_in / 2, groups = p.n_in / 32, blocks = (groups + 1) / 2, pairs = (groups + 3) / 4;
    const auto x_rs = buf_rsrc(p.x + t0 * p.ld_x, ((toks - 1) * p.ld_x + p.n_in) * 2);
    const auto w_rs = buf_rsrc(p.codes + (int64_t)n0 * half, (int64_t)rows * half);
    [[maybe_unused]] std::conditional_t<kLora, LoraOrder, MxNoLora> order(lora, t0, toks);
    [[maybe_unused]] std::conditional_t<kLora, LoraPieces<NT>, MxNoLora> pieces;

    // Loads into LDS: lane l of a wave's load writes 16 bytes at 16 l, i.e.
    // eight rows of tokens or 16 rows of weights.  Slot s of a token row holds
    // chunk s ^ (row / 2) % 8, of a weight row s ^ (row / 4) % 4, so the 16
    // rows of a fragment read spread over all banks.
    int gx[S::XL], xchunk[S::XL], gw[S::WL];
#pragma unroll
    for (int i = 0; i < S::XL; ++i) {
        const int r = (wave * S::XL + i) * 8 + (lane >> 3);
        xchunk[i] = (lane & 7) ^ ((r >> 1) & 7);
        gx[i] = offset_if(r < toks, (int)(r * p.ld_x * 2) + xchunk[i] * 16);
    }
#pragma unroll
    for (int i = 0; i < S::WL; ++i) {
        const int r = (wave * S::WL + i) * 16 + (lane >> 2);
        gw[i] = offset_if(r < rows, r * half + ((lane & 3) ^ ((r >> 2) & 3)) * 16);
    }
    // Past a row's end the tokens are zeros and the scales 0, so the codes there
    // may be anything; past the last block it is loaded again and not used.
    // Scalar offsets stay inside the descriptors: their range is checked on what
    // is left behind that offset.
    const auto issue_x = [&](int k, int st) {
        const int kb = min(k, blocks - 1);
#pragma unroll
        for (int i = 0; i < S::XL; ++i)
            load_lds16(x_rs, lds + st * S::kX + (wave * S::XL + i) * 1024,
                       offset_if(kb * 64 + xchunk[i] * 8 < p.n_in, gx[i]), kb * 128);
    };
    const auto issue_w = [&](int k, int wb) {
#pragma unroll
        for (int i = 0; i < S::WL; ++i)
            load_lds16(w_rs, lds + S::kWeights + wb * S::kW + (wave * S::WL + i) * 1024, gw[i],
                       min(k, pairs - 1) * 64);
    };
    // Scale words: a weight row's per thread, in the first CC / 64 waves.  The
    // word may be unaligned; where the row ends inside it, it starts earlier, by
    // past() bytes that are shifted out.
    const bool carries = wave < S::CC / 64;
    const int rr = tid >> 4;
    const auto past = [&](int kp) { return max(0, kp * 4 + 4 - groups); };
    const uint8_t* s_at = p.scales + (int64_t)(n0 + min(tid, rows - 1)) * groups;
    const int s_to = ((rr / NC * 16 + (tid & 15)) * 2 * S::HP + rr % NC / S::HC * S::HP + rr % NC % S::HC) * 4;
    uint32_t s_in = 0;
    const auto issue_scales = [&](int k) {
        const int kp = min(k, pairs - 1);
        if (carries) {
            if (groups >= 4) {
                __builtin_memcpy(&s_in, s_at + kp * 4 - past(kp), 4);
            } else {
                s_in = 0;
#pragma unroll 1
                for (int j = 0; j < groups; ++j) s_in |= (uint32_t)s_at[j] << (8 * j);
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // before the pair's other loads: the waits count on it
    };
    const auto put_scales = [&](int kp) {
        if (carries)
            *reinterpret_cast<uint32_t*>(lds + S::kScale + (kp & 1) * S::kWS + s_to) =
                groups >= 4 ? s_in >> (8 * past(min(kp, pairs - 1))) : s_in;
    };

    // Fragment reads; b is the block's place in its pair.
    const int xkey = (m >> 1) & 7, wkey = (m >> 2) & 3;
    const int xr = (wt * 16 * NT + m) * 128, xo0 = xr + 16 * ((2 * q) ^ xkey), xo1 = xr + 16 * ((2 * q + 1) ^ xkey);
    const int wo0 = S::kWeights + (wc * 16 * NC + m) * 64 + 16 * ((q >> 1) ^ wkey) + 8 * (q & 1), wo1 = wo0 ^ 32;
    const int s_shift = 8 * (q >> 1);
    u32x4 xf[2][NT][2];
    u32x2 wf[2][S::HC];
    bf16x8 we[S::HC][2];   // a half's weights, expanded
    uint32_t sw[2][S::HC];
    const auto read_x = [&](int st, int t, int to) {
        const uint8_t* base = lds + st * S::kX + t * 2048;
        xf[to][t][0] = *reinterpret_cast<const u32x4*>(base + xo0);
        xf[to][t][1] = *reinterpret_cast<const u32x4*>(base + xo1);
    };
    const auto read_w = [&](int wb, int b, int h) {
#pragma unroll
        for (int i = 0; i < S::HC; ++i)
            wf[h][i] = *reinterpret_cast<const u32x2*>(lds + wb * S::kW + (h * S::HC + i) * 1024 + (b ? wo1 : wo0));
    };
    const auto read_sw = [&](int kp, int h) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(lds + S::kScale + (kp & 1) * S::kWS) +
                            (wc * 16 + m) * 2 * S::HP + h * S::HP;
#pragma unroll
        for (int i = 0; i < S::HC; ++i) sw[h][i] = s[i] >> s_shift;
    };
    f32x4 acc[NT][NC];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    constexpr int kVm = 0x0f70, kLgkm0 = 0xc07f;   // wait for all but the low bits' vector loads; for all of LDS
    // the order in which the waits count: what follows a block's tokens
    issue_scales(0);
    issue_w(0, 0);
    issue_w(1, 1);
    issue_x(0, 0);
    __builtin_amdgcn_sched_barrier(0);
    issue_x(1, 1);
    __builtin_amdgcn_sched_barrier(0);
    issue_w(2, 2);
    issue_x(2, 2);
    issue_x(3, 3);
    __builtin_amdgcn_sched_barrier(0);
    // Ranks up to kLoraAhead: the first adapter's rows arrive beside the first blocks.
    // The waits that count loads then wait for these as well.
    [[maybe_unused]] int lora_cur = -1;
    [[maybe_unused]] const bool ahead = lora_ranks(lora) <= kLoraAhead;
    if constexpr (kLora) {
        lora_cur = order.next();
        if (ahead && lora_cur >= 0) lora_stage(lora, lora_cur, n0, p.n_out, rows, S::CC, lds + S::kBytes);
        pieces.load(lora, t0 + wt * 16 * NT, p.n_tok, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(kVm | (S::WL + 3 * S::XL));
    put_scales(0);
    __builtin_amdgcn_s_waitcnt(kLgkm0);
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int t = 0; t < NT; ++t) read_x(0, t, 0);
    read_w(0, 0, 0);
    read_sw(0, 0);

    // The next pair's scales are loaded in a pair's first block, before that
    // block's tokens, and put down in its second one, where the weights three
    // pairs ahead are loaded.
    int st = 0, wb = 0;
    // P is kb % 2 (a constant once inlined)
    const auto block = [&](int kb, const int P) __attribute__((always_inline)) {
        const int nx = st + 1 == kStages ? 0 : st + 1, nw = wb + 1 == kWeightStages ? 0 : wb + 1, kp = kb >> 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 0) {
                read_w(wb, P, 1);
                if (P == 0) read_sw(kp, 1);
            } else {
                if (P == 0) __builtin_amdgcn_s_waitcnt(kVm | (S::WL + 2 * S::XL));
                else __builtin_amdgcn_s_waitcnt(kVm | S::XL);
                if (P == 1) put_scales(kp + 1);
                __builtin_amdgcn_s_waitcnt(kLgkm0);
                asm volatile("s_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                read_w(P ? nw : wb, 1 - P, 0);
                if (P == 1) read_sw(kp + 1, 0);
#pragma unroll
                for (int t = 0; t < NT; ++t) read_x(nx, t, 1 - P);
                if (P == 0) issue_scales(kp + 1);
                else issue_w(kp + kWeightStages, wb);
                __builtin_amdgcn_sched_barrier(0);
                issue_x(kb + kStages, st);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < S::HC; ++i) {
                    const int c = h * S::HC + i;
                    if (t == 0) {
                        const float scale = __uint_as_float((sw[h][i] >> (16 * P) & 0xffu) << 23);
                        we[i][0] = mx_expand(wf[h][i][0], scale);
                        we[i][1] = mx_expand(wf[h][i][1], scale);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            we[i][j], __builtin_bit_cast(bf16x8, xf[P][t][j]), acc[t][c], 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (P == 1) wb = nw;
        st = nx;
    };
    for (int kb = 0; kb < blocks; kb += 2) {
        block(kb, 0);
        if (kb + 1 == blocks) break;
        block(kb + 1, 1);
    }
    // the loads past the last block are done before their stages are used again
    __builtin_amdgcn_s_waitcnt(0x0070);                          // vmcnt(0) lgkmcnt(0)
    __syncthreads();

    // The adapters' share, the next one's rows of B on their way meanwhile.
    if constexpr (kLora) {
        int ids[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = (wt * NT + t) * 16 + m;
            ids[t] = __shfl(order.id[r >= 64], r & 63);
        }
        constexpr int kHalf = S::CC * GDN_LORA_MAX_RANK * 2;
        static_assert(2 * kHalf <= S::kScale, "two adapters' rows in the stages");
        const auto place = [&](int i) { return lds + (i == 0 && ahead ? S::kBytes : (i & 1) * kHalf); };
        if (!ahead && lora_cur >= 0) {
            lora_stage(lora, lora_cur, n0, p.n_out, rows, S::CC, place(0));
            __builtin_amdgcn_s_waitcnt(0x0f70);                  // vmcnt(0)
            __syncthreads();
        }
        for (int i = 0; lora_cur >= 0; ++i) {
            const int then = order.next();
            if (then >= 0) lora_stage(lora, then, n0, p.n_out, rows, S::CC, place(i + 1));
            lora_add<NT, NC>(lora, lora_cur, ids, t0 + wt * 16 * NT, p.n_tok, pieces, place(i) + wc * 16 * NC * lora.rank * 2,
                             acc);
            __builtin_amdgcn_s_waitcnt(0x0f70);                  // vmcnt(0): the next rows are there
            __syncthreads();
            lora_cur = then;
        }
    }

    // 16 tokens at a time through LDS, each wave its own rows, so that a token's
    // channels leave in 16-byte pieces side by side
    constexpr int V = 16 / (int)sizeof(T), PIECES = 16 * NC / V;
    const int64_t tw = t0 + wt * 16 * NT;
    const int nw = n0 + wc * 16 * NC;
    const int end = min(n_end, o.end[3]);   // from here on gates
    uint8_t* eb = lds + wave * (16 * S::kRow);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            *reinterpret_cast<f32x4*>(eb + m * S::kRow + (c * 16 + 4 * q) * 4) = acc[t][c];
        if (!o.vec16) {   // element by element, neighbours in neighbouring lanes
#pragma unroll 1
            for (int i = lane; i < 16 * 16 * NC; i += 64) {
                const int r = i / (16 * NC), c = i % (16 * NC);
                const int64_t tok = tw + t * 16 + r;
                if (tok >= p.n_tok || nw + c >= n_end) continue;
                mx_put<T>(o, tok, nw + c, reinterpret_cast<const float*>(eb + r * S::kRow)[c]);
            }
            continue;
        }
#pragma unroll 1
        for (int i = lane; i < 16 * PIECES; i += 64) {
            const int r = i / PIECES, piece = (i % PIECES) * V;
            const float* src = reinterpret_cast<const float*>(eb + r * S::kRow) + piece;
            const int64_t tok = tw + t * 16 + r;
            const int n = nw + piece;
            if (tok >= p.n_tok || n >= n_end) continue;
            if (n + V <= end) {
                const f32x4 y0 = *reinterpret_cast<const f32x4*>(src);
                T* d = mx_at<T>(o, tok, n);
                if constexpr (V == 8) {
                    const u32x2 a = pack4(y0), b = pack4(*reinterpret_cast<const f32x4*>(src + 4));
                    *reinterpret_cast<u32x4*>(d) = u32x4{a[0], a[1], b[0], b[1]};
                } else {
                    *reinterpret_cast<f32x4*>(d) = y0;
                }
                continue;
            }
            const int last = min(V, n_end - n);
#pragma unroll 1
            for (int j = 0; j < last; ++j) mx_put<T>(o, tok, n + j, src[j]);
        }
    }
}

bool fits(const void* p, int64_t ld, int elem, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (vec * elem) == 0 && ld % vec == 0;
}

template <typename T, int R, int NC, int D = 2, typename L>
hipError_t skinny(const MxIn& p, const MxOut& o, const MxLaunch& l, const L& lora, hipStream_t stream) {
    constexpr int lds = std::is_same_v<L, MxNoLora> ? SkinnyShape<R, NC, D>::kBytes : SkinnyShape<R, NC, D>::kLoraBytes;
    static_assert(lds <= 160 * 1024, "fits");
    if (lds > 65536) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_dynamic_lds(&mx_skinny_kernel<T, R, NC, D, L>, lds, &done);
        if (e != hipSuccess) return e;
    }
    const int cols = (l.c1 - l.c0 + 16 * NC - 1) / (16 * NC);
    hipLaunchKernelGGL((mx_skinny_kernel<T, R, NC, D, L>), dim3((unsigned)l.workgroups), dim3(kSkinnyThreads), lds,
                       stream, p, o, l.c0, cols, lora);
    return hipGetLastError();
}

template <typename T, int NC, typename L>
hipError_t tile(const MxIn& p, const MxOut& o, const MxLaunch& l, const L& lora, hipStream_t stream) {
    using S = TileShape<NC>;
    constexpr int lds = S::kBytes + (std::is_same_v<L, MxLora> ? S::CC * kLoraAhead * 2 : 0);
    static_assert(lds <= 160 * 1024, "fits");
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_dynamic_lds(&mx_tile_kernel<T, NC, L>, lds, &done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((mx_tile_kernel<T, NC, L>), dim3((unsigned)l.workgroups), dim3(kTileThreads), lds, stream,
                       p, o, (int)((p.n_tok + kTileTokens - 1) / kTileTokens), l.c1, lora);
    return hipGetLastError();
}

template <typename T, typename L>
hipError_t launch_one(const MxIn& p, const MxOut& o, const MxLaunch& l, const L& lora, hipStream_t stream) {
    if (l.tile) return l.channels == 192 ? tile<T, 6>(p, o, l, lora, stream) : tile<T, 4>(p, o, l, lora, stream);
    switch (l.tokens * 256 + l.channels) {
        case 4 * 256 + 16: return skinny<T, 4, 1>(p, o, l, lora, stream);
        case 4 * 256 + 32: return skinny<T, 4, 2>(p, o, l, lora, stream);
        case 16 * 256 + 16: return skinny<T, 16, 1>(p, o, l, lora, stream);
        case 16 * 256 + 32: return skinny<T, 16, 2>(p, o, l, lora, stream);
        case 16 * 256 + 64: return skinny<T, 16, 4>(p, o, l, lora, stream);
        case 32 * 256 + 64: return skinny<T, 32, 4, 1>(p, o, l, lora, stream);
        case 64 * 256 + 64: return skinny<T, 64, 4, 1>(p, o, l, lora, stream);
        default: return hipErrorInvalidValue;   // a shape without a kernel
    }
}

template <typename T, typename L>
hipError_t launch_typed(const MxIn& p, const MxOut& o, const L& lora, hipStream_t stream) {
    const MxPlan plan = mx_plan(p.n_tok, p.n_in, p.n_out);
    for (int i = 0; i < plan.n; ++i) {
        const hipError_t e = launch_one<T>(p, o, plan.launch[i], lora, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename L>
hipError_t launch_any(gdn_dtype out, const MxIn& p, const MxOut& o, const L& lora, hipStream_t stream) {
    return out == GDN_BF16 ? launch_typed<uint16_t>(p, o, lora, stream) : launch_typed<float>(p, o, lora, stream);
}

template <typename T>
hipError_t launch_here(const MxIn& p, const MxOut& o, const MxLaunch& m, const MxLoraHere& lora, hipStream_t stream) {
    return m.channels == 16 ? skinny<T, 4, 1>(p, o, m, lora, stream) : skinny<T, 4, 2>(p, o, m, lora, stream);
}

hipError_t launch_with(gdn_dtype out, const MxIn& p, const MxOut& o, const LoraArgs& l, hipStream_t stream) {
    const int blocks = (l.rank + 15) / 16;
    if (MxLoraHere::takes(p.n_tok, p.n_in, blocks)) {
        const MxPlan plan = mx_plan(p.n_tok, p.n_in, p.n_out);
        const MxLaunch& m = plan.launch[0];
        if (plan.n == 1 && !m.tile && m.tokens == 4 && (m.channels == 16 || m.channels == 32)) {
            const MxLoraHere lora{static_cast<const uint16_t*>(l.a), static_cast<const uint16_t*>(l.b), l.scale, l.ids,
                                  l.n_adapters, l.rank, blocks};
            return out == GDN_BF16 ? launch_here<uint16_t>(p, o, m, lora, stream)
                                   : launch_here<float>(p, o, m, lora, stream);
        }
    }
    const hipError_t e = launch_lora_shrink(p.n_tok, p.n_in, p.x, p.ld_x, l, stream);
    if (e != hipSuccess) return e;
    const MxLora lora{static_cast<const uint16_t*>(l.h), static_cast<const uint16_t*>(l.b), l.ids,
                      l.n_adapters, l.rank, blocks};
    return launch_any(out, p, o, lora, stream);
}

MxOut proj_out(int32_t n_out, gdn_dtype y_dtype, void* y, int64_t ld_y) {
    MxOut o{};
    o.seg[0] = y;
    o.ld[0] = ld_y;
    for (int i = 0; i < 4; ++i) o.end[i] = n_out;
    o.n_out = n_out;
    const int elem = y_dtype == GDN_BF16 ? 2 : 4;
    o.vec4 = n_out % 4 == 0 && fits(y, ld_y, elem, 4);
    o.vec16 = n_out % (16 / elem) == 0 && fits(y, ld_y, elem, 16 / elem);
    return o;
}

MxOut in_proj_out(const gdn_pool* pool, void* q, void* k, void* v, void* z, float* a, float* b) {
    const PoolView& P = pool->view;
    const int hkd = P.h_k * P.d, hvd = P.h_v * P.d;
    MxOut o{};
    void* seg[4] = {q, k, v, z};
    const int width[4] = {hkd, hkd, hvd, z ? hvd : 0};
    const int elem = pool->io_size;
    int end = 0;
    o.vec4 = o.vec16 = 1;
    for (int i = 0; i < 4; ++i) {
        o.seg[i] = seg[i];
        o.ld[i] = width[i];
        o.end[i] = end += width[i];
        o.vec4 = o.vec4 && fits(seg[i], width[i], elem, 4);
        o.vec16 = o.vec16 && fits(seg[i], width[i], elem, 16 / elem);
    }
    o.a = a;
    o.b = b;
    o.h_v = P.h_v;
    o.n_out = end + 2 * P.h_v;
    return o;
}

}  // namespace

hipError_t launch_mx_proj(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t ld_x,
                          const void* codes, const uint8_t* scales, gdn_dtype y_dtype, void* y,
                          int64_t ld_y, hipStream_t stream) {
    const MxIn p{static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(codes), scales,
                 n_tok, ld_x, n_in, n_out};
    return launch_any(y_dtype, p, proj_out(n_out, y_dtype, y, ld_y), MxNoLora{}, stream);
}

hipError_t launch_mx_proj_lora(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t ld_x,
                               const void* codes, const uint8_t* scales, const LoraArgs& l, gdn_dtype y_dtype,
                               void* y, int64_t ld_y, hipStream_t stream) {
    const MxIn p{static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(codes), scales,
                 n_tok, ld_x, n_in, n_out};
    return launch_with(y_dtype, p, proj_out(n_out, y_dtype, y, ld_y), l, stream);
}

hipError_t launch_mx_in_proj(const gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x,
                             const void* codes, const uint8_t* scales, void* q, void* k, void* v,
                             void* z, float* a, float* b, hipStream_t stream) {
    const MxOut o = in_proj_out(pool, q, k, v, z, a, b);
    const MxIn p{static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(codes), scales,
                 n_tok, hidden, hidden, o.n_out};
    return launch_any(pool->desc.io_dtype, p, o, MxNoLora{}, stream);
}

hipError_t launch_mx_in_proj_lora(const gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x,
                                  const void* codes, const uint8_t* scales, const LoraArgs& l, void* q, void* k,
                                  void* v, void* z, float* a, float* b, hipStream_t stream) {
    const MxOut o = in_proj_out(pool, q, k, v, z, a, b);
    const MxIn p{static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(codes), scales,
                 n_tok, hidden, hidden, o.n_out};
    return launch_with(pool->desc.io_dtype, p, o, l, stream);
}

}  // namespace gdn
