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

#include "gdn_common.h"
#include "mfma_split.h"
#include "mx_plan.h"

namespace gdn {
namespace {

constexpr int kRsrcWord3 = 0x00020000;
constexpr int kOffOOB = 0x7ffffff0;   // past every descriptor: loads return zeros

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
using lds_ptr = __attribute__((address_space(3))) void*;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, kRsrcWord3);
}

// 16 bytes per lane from base + offset + soffset straight into LDS, lane l's at
// dst + 16 l.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t rs, void* dst, int offset, int soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)dst, 16, offset, soffset, 0, 0);
}

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

// An offset, or one past every descriptor.  Opaque to the compiler, which would
// otherwise split the load into two branches with a wait between them.
__device__ __forceinline__ int offset_if(bool in, int offset) {
    int v = in ? offset : kOffOOB;
    asm("" : "+v"(v));
    return v;
}

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
// by 64 channels of LDS would be 192 KiB.
constexpr int kSkinnyThreads = kMxWorkgroup, kSkinnyWaves = kSkinnyThreads / 64;

template <int R, int NC, int D>
struct SkinnyShape {
    static constexpr int NT = (R + 15) / 16, XL = R / 4, kW = NC * 1024, kStage = kW + R * 256;
    static constexpr int LD = 16 * NC + 4;
    static constexpr int kLoads = kSkinnyWaves * D * kStage, kSums = kSkinnyWaves * R * LD * 4;
    static constexpr int kBytes = kLoads > kSums ? kLoads : kSums;
    static constexpr int kAhead = (D - 1) * (1 + NC + XL);   // loads of the steps behind the present one
    static_assert((R == 4 || R % 16 == 0) && NC <= 4 && D <= 2 && kAhead < 64, "the schedule");
};

template <typename T, int R, int NC, int D>
__global__ __launch_bounds__(kSkinnyThreads, 2) void mx_skinny_kernel(MxIn p, MxOut o, int c0, int cols) {
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
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < R * 4 * NC; i += kSkinnyThreads) {
        const int t = i / (4 * NC), c = (i % (4 * NC)) * 4;
        if (t >= toks || n0 + c >= p.n_out) continue;
        f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kSkinnyWaves; ++w)
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

template <typename T, int NC>
__global__ __launch_bounds__(kTileThreads, 2) void mx_tile_kernel(MxIn p, MxOut o, int tiles_t, int n_end) {
    using S = TileShape<NC>;
    constexpr int NT = S::NT;
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

template <typename T, int R, int NC, int D = 2>
hipError_t skinny(const MxIn& p, const MxOut& o, const MxLaunch& l, hipStream_t stream) {
    constexpr int lds = SkinnyShape<R, NC, D>::kBytes;
    static_assert(lds <= 160 * 1024, "fits");
    if (lds > 65536) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_dynamic_lds(&mx_skinny_kernel<T, R, NC, D>, lds, &done);
        if (e != hipSuccess) return e;
    }
    const int cols = (l.c1 - l.c0 + 16 * NC - 1) / (16 * NC);
    hipLaunchKernelGGL((mx_skinny_kernel<T, R, NC, D>), dim3((unsigned)l.workgroups), dim3(kSkinnyThreads), lds, stream,
                       p, o, l.c0, cols);
    return hipGetLastError();
}

template <typename T, int NC>
hipError_t tile(const MxIn& p, const MxOut& o, const MxLaunch& l, hipStream_t stream) {
    using S = TileShape<NC>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_dynamic_lds(&mx_tile_kernel<T, NC>, S::kBytes, &done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((mx_tile_kernel<T, NC>), dim3((unsigned)l.workgroups), dim3(kTileThreads), S::kBytes, stream, p,
                       o, (int)((p.n_tok + kTileTokens - 1) / kTileTokens), l.c1);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_one(const MxIn& p, const MxOut& o, const MxLaunch& l, hipStream_t stream) {
    if (l.tile) return l.channels == 192 ? tile<T, 6>(p, o, l, stream) : tile<T, 4>(p, o, l, stream);
    switch (l.tokens * 256 + l.channels) {
        case 4 * 256 + 16: return skinny<T, 4, 1>(p, o, l, stream);
        case 4 * 256 + 32: return skinny<T, 4, 2>(p, o, l, stream);
        case 16 * 256 + 16: return skinny<T, 16, 1>(p, o, l, stream);
        case 16 * 256 + 32: return skinny<T, 16, 2>(p, o, l, stream);
        case 16 * 256 + 64: return skinny<T, 16, 4>(p, o, l, stream);
        case 32 * 256 + 64: return skinny<T, 32, 4, 1>(p, o, l, stream);
        default: return hipErrorInvalidValue;   // a shape without a kernel
    }
}

template <typename T>
hipError_t launch_typed(const MxIn& p, const MxOut& o, hipStream_t stream) {
    const MxPlan plan = mx_plan(p.n_tok, p.n_in, p.n_out);
    for (int i = 0; i < plan.n; ++i) {
        const hipError_t e = launch_one<T>(p, o, plan.launch[i], stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_mx_proj(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t ld_x,
                          const void* codes, const uint8_t* scales, gdn_dtype y_dtype, void* y,
                          int64_t ld_y, hipStream_t stream) {
    const MxIn p{static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(codes), scales,
                 n_tok, ld_x, n_in, n_out};
    MxOut o{};
    o.seg[0] = y;
    o.ld[0] = ld_y;
    for (int i = 0; i < 4; ++i) o.end[i] = n_out;
    o.n_out = n_out;
    const int elem = y_dtype == GDN_BF16 ? 2 : 4;
    o.vec4 = n_out % 4 == 0 && fits(y, ld_y, elem, 4);
    o.vec16 = n_out % (16 / elem) == 0 && fits(y, ld_y, elem, 16 / elem);
    return y_dtype == GDN_BF16 ? launch_typed<uint16_t>(p, o, stream)
                               : launch_typed<float>(p, o, stream);
}

hipError_t launch_mx_in_proj(const gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x,
                             const void* codes, const uint8_t* scales, void* q, void* k, void* v,
                             void* z, float* a, float* b, hipStream_t stream) {
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
    const MxIn p{static_cast<const uint16_t*>(x), static_cast<const uint8_t*>(codes), scales,
                 n_tok, hidden, hidden, o.n_out};
    return pool->desc.io_dtype == GDN_BF16 ? launch_typed<uint16_t>(p, o, stream)
                                           : launch_typed<float>(p, o, stream);
}

}  // namespace gdn
