// Projections with 4-bit weights: y = x W^T, x bf16, W in the format of
// mx_format.hip, fp32 accumulation on the matrix cores.
//
// Few tokens are bound by the weights' bytes and one trip to memory, many by
// the matrix units' feed.  A code times its scale is exact in bf16, so the plain
// way is to expand codes in registers and multiply in bf16.  For bf16 results of
// many tokens the tokens are split into two 8-bit floats instead, and codes go
// into the scaled matrix instructions as they are: as many matrix cycles, none
// for expanding (8192 x 2048 -> 12288 with gates 320-345 us against 487; a
// library product of that size on bf16 weights takes 358).  The 8-bit
// instructions' sums are less exact than the bf16 ones': of 2048 -> 4096, 4 bf16
// results in 1000 differ from the float64 sum's rounding, 4 in 100000 the plain
// way.  So fp32 results take the plain way, and gates do.
#include <algorithm>
#include <type_traits>

#include "gdn_common.h"
#include "mfma_split.h"

namespace gdn {
namespace {

constexpr int kRsrcWord3 = 0x00020000;
constexpr int kOffOOB = 0x7ffffff0;   // past every descriptor: loads return zeros

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
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

// Tokens split into two 8-bit floats (e4m3) with a power-of-two scale for 32
// values: x = (hi + lo / 32) 2^(s - 127), hi and lo rounded to nearest.  With
// the largest magnitude of the 32 in [128, 256) steps of the scale, hi's error
// is at most half of its last of four bits, a multiple of x's own last bit and
// so exact in lo: values down to 2^-14 of the largest are split without error,
// and smaller ones to within 2^-22 of the largest.
// Blocks of 64 values lie token by token, so that a tile's share of a block is
// one piece of memory: rows a power of two apart would all come from the same
// few channels of the cache.
struct MxSplit {
    uint8_t* data;     // [2 pairs][n_tok][128]: 64 hi bytes, then 64 lo bytes
    uint8_t* scales;   // [pairs][n_tok][4], one byte per 32 values; 255: not all finite
    uint8_t* flags;    // [n_tok]: bit 0 an infinity, bit 1 a NaN
    int pairs;         // of blocks, the last padded with zeros
};

// Few tokens, and the strip of gates that the tile kernel leaves.  One
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
constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyThreads = 64 * kSkinnyWaves;

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
__device__ __forceinline__ void skinny_tile(const MxIn& p, const MxOut& o, int64_t t0, int n0) {
    using S = SkinnyShape<R, NC, D>;
    constexpr int NT = S::NT;
    extern __shared__ __align__(16) uint8_t lds[];
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

template <typename T, int R, int NC, int D>
__global__ __launch_bounds__(kSkinnyThreads, 2) void mx_skinny_kernel(MxIn p, MxOut o, int c0, int cols) {
    skinny_tile<T, R, NC, D>(p, o, (int64_t)(blockIdx.x / cols) * R, c0 + (int)(blockIdx.x % cols) * (16 * NC));
}

// The split of the tokens, one wave per token, 16 values per lane and round;
// and in the first gate_wgs workgroups of the same launch the gates, which keep
// fp32's accuracy: the skinny product over the strip of channels from c0 on.
// 8192 tokens of 2048 12.7 us (5.3 TB/s), with 64 gates 21.7; 500 tokens 3.8
// and 4.6.  As further columns of the tiles the gates would cost a round of
// their own.
constexpr int kGateTokens = 16, kGateChannels = 2;   // channels in 16s
using GateShape = SkinnyShape<kGateTokens, kGateChannels, 1>;

__global__ __launch_bounds__(kSkinnyThreads, 4) void mx_split_kernel(MxIn p, MxOut o, int c0, int cols,
                                                                     unsigned gate_wgs, MxSplit sp) {
    if (blockIdx.x < gate_wgs) {
        skinny_tile<uint16_t, kGateTokens, kGateChannels, 1>(p, o, (int64_t)(blockIdx.x / cols) * kGateTokens,
                                                             c0 + (int)(blockIdx.x % cols) * (16 * kGateChannels));
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, values = sp.pairs * 128;
    const int64_t stride = (int64_t)(gridDim.x - gate_wgs) * kSkinnyWaves;
    for (int64_t t = (int64_t)(blockIdx.x - gate_wgs) * kSkinnyWaves + wave; t < p.n_tok; t += stride) {
        const uint16_t* x = p.x + t * p.ld_x;
        uint32_t flag = 0;
        u32x4 next[2];
        const auto load = [&](int v) {
            next[0] = next[1] = u32x4{0, 0, 0, 0};
            if (v < p.n_in) {
                next[0] = *reinterpret_cast<const u32x4*>(x + v);
                next[1] = *reinterpret_cast<const u32x4*>(x + v + 8);
            }
        };
        load(lane * 16);
        for (int v0 = 0; v0 < values; v0 += 64 * 16) {
            const int v = v0 + lane * 16;
            const u32x4 in[2] = {next[0], next[1]};
            load(v + 64 * 16);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max(top, max(in[i / 4][i % 4] << 16 & 0x7fff0000u, in[i / 4][i % 4] & 0x7fff0000u));
            // two lanes hold a group
            top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));
            // the largest magnitude to [128, 256), scale bytes from 5 on (lo's is 5 less)
            int e;
            (void)frexpf(__uint_as_float(top), &e);   // top in [2^(e-1), 2^e)
            const int s = top == 0 ? 127 : max(e - 8 + 127, 5);
            const bool finite = top < 0x7f800000u;
            u32x4 hi, lo;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = ldexpf(__uint_as_float(in[i / 4][i % 4] << 16), 127 - s);
                const float b = ldexpf(__uint_as_float(in[i / 4][i % 4] & 0xffff0000u), 127 - s);
                const int h = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
                const f32x2 f = __builtin_amdgcn_cvt_pk_f32_fp8(h, false);
                const int l = __builtin_amdgcn_cvt_pk_fp8_f32((a - f[0]) * 32.0f, (b - f[1]) * 32.0f, 0, false);
                if (i & 1) { hi[i / 2] |= (uint32_t)h << 16; lo[i / 2] |= (uint32_t)l << 16; }
                else { hi[i / 2] = (uint32_t)h & 0xffffu; lo[i / 2] = (uint32_t)l & 0xffffu; }
            }
            if (v < values) {
                uint8_t* d = sp.data + ((v >> 6) * p.n_tok + t) * 128 + (v & 63);
                const u32x4 zero = {0, 0, 0, 0};
                *reinterpret_cast<u32x4*>(d) = finite ? hi : zero;
                *reinterpret_cast<u32x4*>(d + 64) = finite ? lo : zero;
                if ((lane & 1) == 0) sp.scales[((v >> 7) * p.n_tok + t) * 4 + (v >> 5 & 3)] = (uint8_t)(finite ? s : 255);
            }
            flag |= finite ? 0u : top > 0x7f800000u ? 2u : 1u;
        }
        const bool inf = __ballot(flag & 1) != 0, nan = __ballot(flag & 2) != 0;
        if (lane == 0) sp.flags[t] = (uint8_t)((inf ? 1 : 0) | (nan ? 2 : 0));
    }
}

// Many tokens.  Eight waves, WT x WC, each 16 NT tokens x 16 NC channels, so a
// tile of TT tokens x CC channels per workgroup.  The input axis goes by in
// blocks of 64 through LDS, written by loads that store straight into LDS: the
// tokens' 128 bytes of a block (64 bf16, or the 64 hi and 64 lo bytes of the
// split) through STAGES stages, the weights' 64 bytes of a pair of blocks,
// codes as they are, through STAGES - 1.  The four scale bytes of a pair go
// through a register to a two-stage area ordered so that a lane reads those of
// its rows side by side.  What bounds the kernel is this feed, not the matrix
// units, so each load takes as much of a row at once as LDS holds: 8192 x 2048
// -> 12288 took 309 us, 255 without the loads, 259 without the products, before
// loads went one block further ahead (300 us; the matrix units are then busy
// 57 % of the time, at 2.0 GHz).  Four waves of twice the area read LDS less but
// hide less: 360 for 321 us with the split, and 500 tokens 38.2 for 34.0.
//
// bf16 (F8 false): lane q of MFMA j (16x16x32) takes k = 16 q + 8 j ..: one
// 8-byte read of codes serves both MFMAs, expanded in registers.
// Split (F8 true): one scaled MFMA (16x16x128) takes codes as they are times
// hi in its lower and lo in its upper half of k, the same codes in both.  It
// holds lane q's 32 codes for k = 32 q .., but 8-bit operands as k = 16 q ..
// and 64 + 16 q ..; the scale of lane q is that of k = 32 q .. for both.
//
// A wave keeps its tokens' fragments of a block in registers and takes its
// channels in two halves, all of a half times one token fragment after the
// other; the next half's codes arrive meanwhile.  The block's one barrier
// stands between the halves.  It says that the next block has arrived and this
// one's stage is read out, to be filled with the block STAGES ahead.
// Behind it the next block's token fragments are read, each as soon as the
// second half is through with its predecessor, or where registers allow
// (kDouble) all of them into a second set.
template <bool F8, int NT, int NC, int WT, int WC, int STAGES>
struct TileShape {
    static constexpr int TT = 16 * NT * WT, CC = 16 * NC * WC, WAVES = WT * WC, TH = 64 * WAVES;
    static constexpr int XL = TT / 8 / WAVES;                      // loads per wave and block
    static constexpr int WL = (CC / 16 + WAVES - 1) / WAVES;       // loads per wave and pair
    static constexpr int WB = STAGES - 1;
    static constexpr int kX = TT * 128, kW = WL * WAVES * 1024, kWeights = STAGES * kX;
    static constexpr int HC = NC / 2, HP = HC <= 2 ? 2 : 4;        // channels of a half; their scale words' places
    static constexpr int kWS = WC * 16 * 2 * HP * 4, kXS = WT * 16 * NT * 4;
    static constexpr int kScale = kWeights + WB * kW, kBytes = kScale + 2 * (kWS + kXS);
    static constexpr bool kDouble = NT <= 2;
    static_assert(WAVES == 8 && TT <= 256 && CC <= 256 && TT % 64 == 0, "a scale word per thread; whole loads");
    static_assert(NC % 2 == 0 && (STAGES == 3 || STAGES == 4) && WL + (STAGES - 1) * XL < 16, "the schedule");
    // the epilogue's rows (fp32, 16 bytes apart) in the stages
    static constexpr int kRow = 16 * NC * 4 + 16;
    static_assert(WAVES * 16 * kRow <= kScale && kBytes <= 160 * 1024, "fits");
};

// Byte 2 p of sw and of sx scale the operands (p a constant once inlined).
__device__ __forceinline__ f32x4 mfma_f8(int p, i32x8 w, i32x8 x, f32x4 c, int sw, int sx) {
    return p ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, 0, 2, sw, 2, sx)
             : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, 0, 0, sw, 0, sx);
}

// One output by the definition, for tokens that hold an infinity.
__device__ __forceinline__ float mx_dot(const MxIn& p, int64_t t, int n) {
    const uint16_t* x = p.x + t * p.ld_x;
    const uint8_t* c = p.codes + (int64_t)n * (p.n_in / 2);
    const uint8_t* s = p.scales + (int64_t)n * (p.n_in / 32);
    float y = 0.f;
#pragma unroll 1
    for (int k = 0; k < p.n_in; k += 2) {
        const bf16x2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c[k >> 1],
                                                                   __uint_as_float((uint32_t)s[k >> 5] << 23), 0);
        y = fmaf(bf16_to_f32(x[k]), (float)w[0], y);
        y = fmaf(bf16_to_f32(x[k + 1]), (float)w[1], y);
    }
    return y;
}

template <typename T, bool F8, int NT, int NC, int WT, int WC, int STAGES>
__global__ __launch_bounds__(64 * WT * WC, 2) void mx_tile_kernel(MxIn p, MxOut o, MxSplit sp, int tiles_t,
                                                                  int n_end) {
    using S = TileShape<F8, NT, NC, WT, WC, STAGES>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wt = wave / WC, wc = wave % WC;
    // Consecutive tiles share their channels.  Workgroups go to the eight XCDs
    // in turn: with fewer than eight tiles along the tokens each XCD takes a run
    // of tiles, so that it reads the run's weights into its own cache once
    // (500 x 2048 -> 12288 with gates 32.9 -> 31.9 us); with more, every eighth
    // shares its tokens (8192 tokens 331 us, in runs 362).
    unsigned idx = blockIdx.x;
    if (tiles_t < 8) {
        const unsigned xcd = idx % 8, per = gridDim.x / 8, rest = gridDim.x % 8;
        idx = xcd * per + min(xcd, rest) + idx / 8;
    }
    const int64_t t0 = (int64_t)(idx % tiles_t) * S::TT;
    const int n0 = (int)(idx / tiles_t) * S::CC;
    const int toks = (int)min((int64_t)S::TT, p.n_tok - t0), rows = min(S::CC, n_end - n0);
    const int half = p.n_in / 2, groups = p.n_in / 32, blocks = (groups + 1) / 2, pairs = (groups + 3) / 4;
    const auto x_rs = buf_rsrc(F8 ? nullptr : p.x + t0 * p.ld_x, ((toks - 1) * p.ld_x + p.n_in) * 2);
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
        gx[i] = offset_if(r < toks, (F8 ? r * 128 : (int)(r * p.ld_x * 2)) + xchunk[i] * 16);
    }
#pragma unroll
    for (int i = 0; i < S::WL; ++i) {
        const int r = (wave * S::WL + i) * 16 + (lane >> 2);
        gw[i] = offset_if(r < rows, r * half + ((lane & 3) ^ ((r >> 2) & 3)) * 16);
    }
    // Past a row's end the tokens are zeros (or the split's padding) and the
    // scales 0, so the codes there may be anything; past the last block it is
    // loaded again and not used.  Scalar offsets stay inside the descriptors:
    // their range is checked on what is left behind that offset.
    const auto issue_x = [&](int k, int st) {
        const int kb = min(k, blocks - 1);
        const auto rs = F8 ? buf_rsrc(sp.data + (kb * p.n_tok + t0) * 128, toks * 128) : x_rs;
#pragma unroll
        for (int i = 0; i < S::XL; ++i)
            load_lds16(rs, lds + st * S::kX + (wave * S::XL + i) * 1024,
                       F8 ? gx[i] : offset_if(kb * 64 + xchunk[i] * 8 < p.n_in, gx[i]), F8 ? 0 : kb * 128);
    };
    const auto issue_w = [&](int k, int wb) {
#pragma unroll
        for (int i = 0; i < S::WL; ++i)
            load_lds16(w_rs, lds + S::kWeights + wb * S::kW + (wave * S::WL + i) * 1024, gw[i],
                       min(k, pairs - 1) * 64);
    };
    // Scale words: the first four waves carry a weight row's per thread, the
    // others a token's.  A weight row's word may be unaligned; where the row ends
    // inside it, it starts earlier, by past() bytes that are shifted out.
    const bool of_x = wave >= 4;
    const int srow = tid & 255, rr = srow >> 4;
    const auto past = [&](int kp) { return of_x ? 0 : max(0, kp * 4 + 4 - groups); };
    const uint8_t* s_at = of_x ? sp.scales + (t0 + min(srow, toks - 1)) * 4
                               : p.scales + (int64_t)(n0 + min(srow, rows - 1)) * groups;
    const int64_t s_step = of_x ? p.n_tok * 4 : 4;
    const int s_to = of_x ? S::kWS + ((rr / NT * 16 + (srow & 15)) * NT + rr % NT) * 4
                          : ((rr / NC * 16 + (srow & 15)) * 2 * S::HP + rr % NC / S::HC * S::HP + rr % NC % S::HC) * 4;
    uint32_t s_in = 0;
    const auto issue_scales = [&](int k) {
        const int kp = min(k, pairs - 1);
        if (F8 || !of_x) {
            if (groups >= 4) {
                __builtin_memcpy(&s_in, s_at + kp * s_step - past(kp), 4);
            } else {
                s_in = 0;
#pragma unroll 1
                for (int j = 0; j < groups; ++j) s_in |= (uint32_t)s_at[j] << (8 * j);
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // before the pair's other loads: the waits count on it
    };
    const auto put_scales = [&](int kp) {
        if (srow < (of_x ? F8 ? S::TT : 0 : S::CC))
            *reinterpret_cast<uint32_t*>(lds + S::kScale + (kp & 1) * (S::kWS + S::kXS) + s_to) =
                groups >= 4 ? s_in >> (8 * past(min(kp, pairs - 1))) : s_in;
    };

    // Fragment reads; b is the block's place in its pair.
    const int xkey = (m >> 1) & 7, wkey = (m >> 2) & 3;
    const int xc0 = F8 ? q : 2 * q, xc1 = F8 ? 4 + q : 2 * q + 1;
    const int xr = (wt * 16 * NT + m) * 128, xo0 = xr + 16 * (xc0 ^ xkey), xo1 = xr + 16 * (xc1 ^ xkey);
    const int wr = S::kWeights + (wc * 16 * NC + m) * 64;
    const int wo0 = wr + (F8 ? 16 * ((q & 1) ^ wkey) : 16 * ((q >> 1) ^ wkey) + 8 * (q & 1)), wo1 = wo0 ^ 32;
    const int s_shift = 8 * (F8 ? q & 1 : q >> 1);
    u32x4 xf[S::kDouble ? 2 : 1][NT][2];
    using Codes = std::conditional_t<F8, u32x4, u32x2>;
    Codes wf[2][S::HC];
    bf16x8 we[F8 ? 1 : S::HC][2];   // a half's weights, expanded
    uint32_t sw[2][S::HC], sx[2][NT];
    const auto read_x = [&](int st, int t, int to) {
        const uint8_t* base = lds + st * S::kX + t * 2048;
        xf[to][t][0] = *reinterpret_cast<const u32x4*>(base + xo0);
        xf[to][t][1] = *reinterpret_cast<const u32x4*>(base + xo1);
    };
    const auto read_w = [&](int wb, int b, int h) {
#pragma unroll
        for (int i = 0; i < S::HC; ++i)
            wf[h][i] = *reinterpret_cast<const Codes*>(lds + wb * S::kW + (h * S::HC + i) * 1024 + (b ? wo1 : wo0));
    };
    const auto read_sw = [&](int kp, int h) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(lds + S::kScale + (kp & 1) * (S::kWS + S::kXS)) +
                            (wc * 16 + m) * 2 * S::HP + h * S::HP;
#pragma unroll
        for (int i = 0; i < S::HC; ++i) sw[h][i] = s[i] >> s_shift;
    };
    const auto read_sx = [&](int kp, int to) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(lds + S::kScale + (kp & 1) * (S::kWS + S::kXS) + S::kWS) +
                            (wt * 16 + m) * NT;
        if constexpr (F8)
#pragma unroll
            for (int t = 0; t < NT; ++t) sx[to][t] = (s[t] - (q >> 1) * 0x05050505u) >> s_shift;
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
    if constexpr (STAGES == 4) issue_w(1, 1);
    issue_x(0, 0);
    __builtin_amdgcn_sched_barrier(0);
    issue_x(1, 1);
    __builtin_amdgcn_sched_barrier(0);
    issue_w(S::WB - 1, S::WB - 1);
    issue_x(2, 2);
    if constexpr (STAGES == 4) issue_x(3, 3);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kVm | (S::WL + (STAGES - 1) * S::XL));
    put_scales(0);
    __builtin_amdgcn_s_waitcnt(kLgkm0);
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int t = 0; t < NT; ++t) read_x(0, t, 0);
    read_w(0, 0, 0);
    read_sw(0, 0);
    read_sx(0, 0);

    // The next pair's scales are loaded in a pair's first block, before that
    // block's tokens, and put down in its second one, where the weights WB pairs
    // ahead are loaded.
    int st = 0, wb = 0;
    // P is kb % 2 (a constant once inlined)
    const auto block = [&](int kb, const int P) __attribute__((always_inline)) {
        const int D = S::kDouble ? P : 0, N = S::kDouble ? 1 - P : 0;
        const int nx = st + 1 == STAGES ? 0 : st + 1, nw = wb + 1 == S::WB ? 0 : wb + 1, kp = kb >> 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 0) {
                read_w(wb, P, 1);
                if (P == 0) read_sw(kp, 1);
            } else {
                if (P == 0) __builtin_amdgcn_s_waitcnt(kVm | (S::WL + (STAGES - 2) * S::XL));
                else __builtin_amdgcn_s_waitcnt(kVm | S::XL);
                if (P == 1) put_scales(kp + 1);
                __builtin_amdgcn_s_waitcnt(kLgkm0);
                asm volatile("s_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                read_w(P ? nw : wb, 1 - P, 0);
                if (P == 1) {
                    read_sw(kp + 1, 0);
                    read_sx(kp + 1, 1);
                }
                if constexpr (S::kDouble)
#pragma unroll
                    for (int t = 0; t < NT; ++t) read_x(nx, t, N);
                if (P == 0) issue_scales(kp + 1);
                else issue_w(kp + S::WB, wb);
                __builtin_amdgcn_sched_barrier(0);
                issue_x(kb + STAGES, st);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < S::HC; ++i) {
                    const int c = h * S::HC + i;
                    const Codes w = wf[h][i];
                    if constexpr (F8) {
                        const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
                        const u32x4 hi = xf[D][t][0], lo = xf[D][t][1];
                        const i32x8 b = {(int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3],
                                         (int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3]};
                        acc[t][c] = mfma_f8(P, a, b, acc[t][c], (int)sw[h][i], (int)sx[0][t]);
                    } else {
                        if (t == 0) {
                            const float scale = __uint_as_float((sw[h][i] >> (16 * P) & 0xffu) << 23);
                            we[i][0] = mx_expand(w[0], scale);
                            we[i][1] = mx_expand(w[1], scale);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                we[i][j], __builtin_bit_cast(bf16x8, xf[D][t][j]), acc[t][c], 0, 0, 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (!S::kDouble)
                    if (h == 1) read_x(nx, t, 0);
            }
        }
        if (P == 1) {
            if constexpr (F8)
#pragma unroll
                for (int t = 0; t < NT; ++t) sx[0][t] = sx[1][t];
            wb = nw;
        }
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
                float y = reinterpret_cast<const float*>(eb + r * S::kRow)[c];
                if constexpr (F8)
                    if (y != y && sp.flags[tok] == 1) y = mx_dot(p, tok, nw + c);
                mx_put<T>(o, tok, nw + c, y);
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
            const f32x4 y0 = *reinterpret_cast<const f32x4*>(src);
            const f32x4 y1 = *reinterpret_cast<const f32x4*>(src + V - 4);
            const bool whole = n + V <= end;
            // A token with an infinity (and no NaN) has no split: its results
            // are infinite or NaN, as the definition has them.
            bool again = false;
            if constexpr (F8) {
                bool nan = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) nan |= (y0[j] != y0[j]) | (y1[j] != y1[j]);
                again = nan && sp.flags[tok] == 1;
            }
            if (whole && !again) {
                T* d = mx_at<T>(o, tok, n);
                if constexpr (V == 8) {
                    const u32x2 a = pack4(y0), b = pack4(y1);
                    *reinterpret_cast<u32x4*>(d) = u32x4{a[0], a[1], b[0], b[1]};
                } else {
                    *reinterpret_cast<f32x4*>(d) = y0;
                }
                continue;
            }
            const int last = min(V, n_end - n);
#pragma unroll 1
            for (int j = 0; j < last; ++j) {
                float y = src[j];
                if constexpr (F8)
                    if (again && y != y) y = mx_dot(p, tok, n + j);
                mx_put<T>(o, tok, n + j, y);
            }
        }
    }
}

bool fits(const void* p, int64_t ld, int elem, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (vec * elem) == 0 && ld % vec == 0;
}

// The channels from c0 on.
template <typename T, int R, int NC, int D = 2>
hipError_t skinny(const MxIn& p, const MxOut& o, hipStream_t stream, int c0 = 0) {
    constexpr int lds = SkinnyShape<R, NC, D>::kBytes;
    static_assert(lds <= 160 * 1024, "fits");
    if (lds > 65536) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_dynamic_lds(&mx_skinny_kernel<T, R, NC, D>, lds, &done);
        if (e != hipSuccess) return e;
    }
    const int cols = (p.n_out - c0 + 16 * NC - 1) / (16 * NC);
    const dim3 grid((unsigned)(cols * ((p.n_tok + R - 1) / R)));
    hipLaunchKernelGGL((mx_skinny_kernel<T, R, NC, D>), grid, dim3(kSkinnyThreads), lds, stream, p, o, c0, cols);
    return hipGetLastError();
}

// The tokens' split and the channels from c0 on.
hipError_t split(const MxIn& p, const MxOut& o, int c0, const MxSplit& sp, hipStream_t stream) {
    constexpr int lds = GateShape::kBytes;
    const int cols = (p.n_out - c0 + 16 * kGateChannels - 1) / (16 * kGateChannels);
    const int64_t gates = cols * ((p.n_tok + kGateTokens - 1) / kGateTokens);
    const int64_t tokens = std::min<int64_t>((p.n_tok + kSkinnyWaves - 1) / kSkinnyWaves, 1 << 20);
    if (gates && lds > 65536) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_dynamic_lds(&mx_split_kernel, lds, &done);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(mx_split_kernel, dim3((unsigned)(gates + tokens)), dim3(kSkinnyThreads), gates ? lds : 0,
                       stream, p, o, c0, cols, (unsigned)gates, sp);
    return hipGetLastError();
}

template <typename T, bool F8, int NT, int NC, int WT, int WC, int STAGES>
hipError_t tile(const MxIn& p, const MxOut& o, const MxSplit& sp, int n_end, hipStream_t stream) {
    using S = TileShape<F8, NT, NC, WT, WC, STAGES>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_dynamic_lds(&mx_tile_kernel<T, F8, NT, NC, WT, WC, STAGES>, S::kBytes, &done);
    if (e != hipSuccess) return e;
    const int tiles_t = (int)((p.n_tok + S::TT - 1) / S::TT), tiles_c = (n_end + S::CC - 1) / S::CC;
    hipLaunchKernelGGL((mx_tile_kernel<T, F8, NT, NC, WT, WC, STAGES>), dim3((unsigned)tiles_t * tiles_c), dim3(S::TH),
                       S::kBytes, stream, p, o, sp, tiles_t, n_end);
    return hipGetLastError();
}

int64_t tiles_of(int64_t n_tok, int64_t n_out, int tt, int cc) {
    return ((n_tok + tt - 1) / tt) * ((n_out + cc - 1) / cc);
}
int64_t rounds_of(int64_t tiles) { return (tiles + 255) / 256; }

// Times in 1/1024 us, from which a call's kernels are picked.  A round of 256
// skinny workgroups of 32 tokens by 64 channels takes about 2 us and 1.8 more
// per 1024 inputs; of tiles about 5 us and, per 1024 inputs, 8 (128x128), 11.5
// (128x192) or 23 (256x256).
int64_t skinny_time(int64_t n_tok, int32_t n_in, int64_t n_out) {
    return rounds_of(tiles_of(n_tok, n_out, 32, 64)) * (2048 + (int64_t)n_in * 9 / 5);
}

// Tiles of one shape for the channels below n_main.  Where the last column of
// tiles would cost a round for few channels, these are a skinny call of their
// own (4096 x 2048 -> 12352: 12288 channels in 3 rounds, not 49 columns in 4).
struct TilePlan {
    int shape, n_main;
    int64_t time;
};
constexpr int kTiles[3][3] = {{256, 256, 23 * 1024}, {128, 192, 11 * 1024 + 512}, {128, 128, 8 * 1024}};

TilePlan plan_tiles(int64_t n_tok, int32_t n_in, int64_t n_out, bool large) {
    TilePlan best{0, (int)n_out, INT64_MAX};
    for (int i = large ? 0 : 1; i < 3; ++i) {
        const int tt = kTiles[i][0], cc = kTiles[i][1];
        const int64_t round = 5 * 1024 + (int64_t)n_in * kTiles[i][2] / 1024;
        const int64_t whole = n_out / cc * cc;
        const int64_t all = rounds_of(tiles_of(n_tok, n_out, tt, cc)) * round;
        if (all < best.time) best = {i, (int)n_out, all};
        if (whole == 0 || whole == n_out || n_in < 128) continue;
        const int64_t strip = rounds_of(tiles_of(n_tok, whole, tt, cc)) * round + 2048 +
                              skinny_time(n_tok, n_in, n_out - whole);
        if (strip < best.time) best = {i, (int)whole, strip};
    }
    return best;
}

// Tiles for the channels below n_end; with expanded weights (no split) the
// largest shape's registers spill.
template <typename T, bool F8>
hipError_t launch_tiles(const MxIn& p, const MxOut& o, const MxSplit& sp, int n_end, hipStream_t stream) {
    const TilePlan plan = plan_tiles(p.n_tok, p.n_in, n_end, F8);
    if (plan.n_main < n_end) {
        MxIn rest = p;
        rest.n_out = n_end;
        const hipError_t e = skinny<T, 32, 4, 1>(rest, o, stream, plan.n_main);
        if (e != hipSuccess) return e;
    }
    if constexpr (F8)
        if (plan.shape == 0) return tile<T, F8, 4, 8, 4, 2, 3>(p, o, sp, plan.n_main, stream);
    if (plan.shape == 1) return tile<T, F8, 2, 6, 4, 2, 4>(p, o, sp, plan.n_main, stream);
    return tile<T, F8, 2, 4, 4, 2, 4>(p, o, sp, plan.n_main, stream);
}

// The skinny kernel takes the call, or the tile kernel (2048 -> 12352: 96 tokens
// 19.9 against 24.3 us, 128 tokens 25.5 against 24.2; 4096 -> 2048: 256 tokens
// 10.0 against 39.8 us, 1500 tokens 48.9 against 43.1).
bool use_skinny(int64_t n_tok, int32_t n_in, int64_t n_out) {
    if (n_in < 128) return false;
    // the split takes about 3 us, and its reads and writes
    return n_tok <= 16 || skinny_time(n_tok, n_in, n_out) <=
                              plan_tiles(n_tok, n_in, n_out, true).time + 3072 + n_tok * n_in / 1660;
}

bool use_split(int64_t n_tok, int32_t n_in, int64_t n_out, gdn_dtype out) {
    return out == GDN_BF16 && n_in >= 512 && !use_skinny(n_tok, n_in, n_out);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

MxSplit split_of(int64_t n_tok, int32_t n_in, void* workspace, size_t* bytes) {
    MxSplit s;
    s.pairs = (n_in + 127) / 128;
    const size_t data = (size_t)n_tok * s.pairs * 256, scales = up256((size_t)n_tok * s.pairs * 4);
    s.data = static_cast<uint8_t*>(workspace);
    s.scales = s.data + data;
    s.flags = s.scales + scales;
    *bytes = data + scales + up256((size_t)n_tok);
    return s;
}

template <typename T>
hipError_t launch_few(const MxIn& p, const MxOut& o, hipStream_t stream) {
    // Bytes that the busiest CU takes in, the tile's tokens and weights: the
    // measure that separates the shapes where the axis is not the limit.
    const auto cost = [&](int r, int nc) {
        const int64_t wgs = ((p.n_tok + r - 1) / r) * ((p.n_out + 16 * nc - 1) / (16 * nc));
        return (wgs + 255) / 256 * (std::min<int64_t>(p.n_tok, r) * 4 + 16 * nc);
    };
    if (p.n_tok <= 4) return cost(4, 1) <= cost(4, 2) ? skinny<T, 4, 1>(p, o, stream) : skinny<T, 4, 2>(p, o, stream);
    int best = 0;
    int64_t least = INT64_MAX;
    constexpr int shapes[][2] = {{16, 1}, {16, 2}, {16, 4}, {32, 4}};
    for (int i = 0; i < 4; ++i) {
        const int64_t c = cost(shapes[i][0], shapes[i][1]);
        if (c < least) { least = c; best = i; }
    }
    switch (best) {
        case 0: return skinny<T, 16, 1>(p, o, stream);
        case 1: return skinny<T, 16, 2>(p, o, stream);
        case 2: return skinny<T, 16, 4>(p, o, stream);
        default: return skinny<T, 32, 4, 1>(p, o, stream);
    }
}

template <typename T>
hipError_t launch_typed(const MxIn& p, const MxOut& o, void* workspace, hipStream_t stream) {
    if (use_skinny(p.n_tok, p.n_in, p.n_out)) return launch_few<T>(p, o, stream);
    if constexpr (sizeof(T) == 2) {
        if (use_split(p.n_tok, p.n_in, p.n_out, GDN_BF16)) {
            size_t bytes;
            const MxSplit sp = split_of(p.n_tok, p.n_in, workspace, &bytes);
            const int n_end = o.end[3];
            const hipError_t e = split(p, o, n_end, sp, stream);
            if (e != hipSuccess) return e;
            return launch_tiles<T, true>(p, o, sp, n_end, stream);
        }
    }
    const MxSplit none{};
    return launch_tiles<T, false>(p, o, none, p.n_out, stream);
}

}  // namespace

// Every launch stays below 2^32 threads: the most are 512 for each 16 tokens or
// so and the few channels of the gates, or each 32 by 64.
bool mx_proj_fits(int64_t n_tok, int64_t n_out) {
    const int64_t t = n_tok / 64 + 1, c = n_out / 64 + 1;
    return t < (1 << 22) && t * c < (1 << 22);
}

size_t mx_proj_workspace_bytes(int64_t n_tok, int32_t n_in, int32_t n_out) {
    size_t bytes = 0;
    // whichever type the results have
    if (use_split(n_tok, n_in, n_out, GDN_BF16)) split_of(n_tok, n_in, nullptr, &bytes);
    return bytes;
}

hipError_t launch_mx_proj(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t ld_x,
                          const void* codes, const uint8_t* scales, gdn_dtype y_dtype, void* y,
                          int64_t ld_y, void* workspace, hipStream_t stream) {
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
    return y_dtype == GDN_BF16 ? launch_typed<uint16_t>(p, o, workspace, stream)
                               : launch_typed<float>(p, o, workspace, stream);
}

hipError_t launch_mx_in_proj(const gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x,
                             const void* codes, const uint8_t* scales, void* q, void* k, void* v,
                             void* z, float* a, float* b, void* workspace, hipStream_t stream) {
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
    return pool->desc.io_dtype == GDN_BF16 ? launch_typed<uint16_t>(p, o, workspace, stream)
                                           : launch_typed<float>(p, o, workspace, stream);
}

}  // namespace gdn
