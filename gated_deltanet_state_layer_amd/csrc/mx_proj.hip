// Projections with 4-bit weights: y = x W^T, x bf16, W in the format of
// mx_format.hip, fp32 accumulation on the matrix cores.
#include <algorithm>

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

// Where the output channels go: [0, end[0]) to seg[0], [end[0], end[1]) to
// seg[1], and so on, ld elements between tokens; from end[3] on, fp32 gates a
// and b of h_v channels each.  A plain projection has one segment.
struct MxOut {
    void* seg[4];
    int64_t ld[4];
    int end[4];
    float *a, *b;
    int h_v, n_out;
    int vec4, vec8;   // segment starts, strides and ends are multiples of 4 / 8 elements
};

template <typename T>
__device__ __forceinline__ T* mx_at(const MxOut& o, int64_t t, int n) {
    int s = 0, base = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (n >= o.end[i]) { s = i + 1; base = o.end[i]; }
    return static_cast<T*>(o.seg[s]) + t * o.ld[s] + n - base;
}

template <typename T>
__device__ __forceinline__ void mx_put(const MxOut& o, int64_t t, int n, float y) {
    if (n < o.end[3]) Io<T>::store(mx_at<T>(o, t, n), 0, y);
    else if (n < o.end[3] + o.h_v) o.a[t * o.h_v + n - o.end[3]] = 1.0f / (1.0f + expf(y));
    else o.b[t * o.h_v + n - o.end[3] - o.h_v] = 1.0f / (1.0f + expf(-y));
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
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < o.n_out) mx_put<T>(o, t, n + i, y[i]);
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
struct MxSplit {
    uint8_t* data;     // [n_tok][row]: per 64 values 64 hi bytes, then 64 lo bytes
    uint8_t* scales;   // [n_tok][row / 64], one byte per 32 values; 255: not all finite
    uint8_t* flags;    // [n_tok]: bit 0 an infinity, bit 1 a NaN
    int row;           // bytes of a token's data, a multiple of 128
};

// The four codes' dwords of four lanes 16 apart, transposed: lane row q gets
// dword q of lane rows 0..3 in w[0..3].
__device__ __forceinline__ void transpose4(u32x4& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4{c[0], c[1], d[0], d[1]};
}

// Largest over the four lanes 16 apart, in all four.
__device__ __forceinline__ uint32_t max_over_rows(uint32_t x) {
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return max((uint32_t)b[0], (uint32_t)b[1]);
}

// The scale bytes of groups 4 st .. 4 st + 3 of a row, the first lowest.  The
// load may be unaligned; where the row ends inside the four it starts earlier,
// by scales_past() bytes that the caller shifts out once it has arrived.
__device__ __forceinline__ int scales_past(int st, int groups) {
    return groups < 4 ? 0 : max(0, st * 4 + 4 - groups);
}
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, int st, int groups) {
    uint32_t v = 0;
    if (groups >= 4) {
        __builtin_memcpy(&v, row + st * 4 - scales_past(st, groups), 4);
    } else {
#pragma unroll 1
        for (int j = 0; j < groups; ++j) v |= (uint32_t)row[j] << (8 * j);
    }
    return v;
}

// Few tokens, and the strip of channels that the tile kernel leaves.  One
// workgroup of 8 waves per 16 NT tokens and 16 NC channels; each wave
// multiplies the whole tile over its eighth of the input axis, operands
// straight from memory, D steps of 128 in flight, and the eight partial tiles
// are added in LDS.  Lane l = 16 q + m loads row m's group q of a step as 16
// bytes (32 codes); transposed over q, MFMA j of the four (16x16x32) takes
// group j, lane q its codes 8q .. 8q+7, so tokens are read 64 bytes at a time.
// W is the A operand: a lane's four results are consecutive channels of one
// token.  With SPLIT the workgroups of channel block 0 also write the tokens'
// 8-bit split (NC = 0: nothing else).
constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyThreads = 64 * kSkinnyWaves;

constexpr size_t skinny_lds(int nt, int nc) {
    return (size_t)kSkinnyWaves * 16 * nt * (16 * nc + 4) * sizeof(float);
}

template <typename T, int NT, int NC, bool SPLIT>
__global__ __launch_bounds__(kSkinnyThreads, NT * 16 + NC * 5 > 40 ? 2 : 4) void mx_skinny_kernel(MxIn p, MxOut o, int c0,
                                                                                       MxSplit sp) {
    constexpr int D = 2;
    extern __shared__ __align__(16) float red[];   // [8 waves][16 NT tokens][16 NC + 4 channels]
    __shared__ uint32_t flags[16 * NT];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.y * (16 * NT);
    const int n0 = c0 + blockIdx.x * (16 * NC);
    const int toks = (int)min((int64_t)(16 * NT), p.n_tok - t0), rows = min(16 * NC, p.n_out - n0);
    const int half = p.n_in / 2, groups = p.n_in / 32;
    const int steps = (groups + 3) / 4, per = (steps + kSkinnyWaves - 1) / kSkinnyWaves;
    const int s_begin = wave * per, s_end = min(steps, s_begin + per);
    const bool split = SPLIT && blockIdx.x == 0;
    const auto x_rs = buf_rsrc(p.x + t0 * p.ld_x, ((toks - 1) * p.ld_x + p.n_in) * 2);
    const auto w_rs = buf_rsrc(p.codes + (int64_t)n0 * half, (int64_t)rows * half);
    if constexpr (SPLIT) {
        if (threadIdx.x < 16 * NT) flags[threadIdx.x] = 0;
        __syncthreads();
    }
    u32x4 xs[D][NT][4], ws[D][NC > 0 ? NC : 1];
    uint32_t ss[D][NC > 0 ? NC : 1];
    const auto fetch = [&](int st, int b) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int r = c * 16 + m;
            const bool in = st < s_end && r < rows;
            ws[b][c] = __builtin_amdgcn_raw_buffer_load_b128(
                w_rs, in && st * 4 + q < groups ? r * half + (st * 4 + q) * 16 : kOffOOB, 0, 0);
            ss[b][c] = load_scales(p.scales + (int64_t)(n0 + min(r, rows - 1)) * groups, min(st, steps - 1), groups);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = t * 16 + m;
                const bool in = st < s_end && st * 4 + j < groups && r < toks;
                xs[b][t][j] = __builtin_amdgcn_raw_buffer_load_b128(
                    x_rs, in ? (int)(r * p.ld_x + st * 128 + j * 32 + q * 8) * 2 : kOffOOB, 0, 0);
            }
    };
    f32x4 acc[NT][NC > 0 ? NC : 1];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto multiply = [&](int st, int b) {
        const int past = 8 * scales_past(st, groups);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            transpose4(ws[b][c]);
            const uint32_t s = ss[b][c] >> past;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 wf = mx_expand(ws[b][c][j], __uint_as_float((s >> (8 * j) & 0xffu) << 23));
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        wf, __builtin_bit_cast(bf16x8, xs[b][t][j]), acc[t][c], 0, 0, 0);
            }
        }
    };
    // The split of step st: lane (m, q) holds values 8q .. 8q+7 of group 4 st + j of token m.
    const auto write_split = [&](int st, int b) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = t * 16 + m;
            uint32_t packed = 0, flag = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = max(top, max(xs[b][t][j][i] << 16 & 0x7fff0000u, xs[b][t][j][i] & 0x7fff0000u));
                top = max_over_rows(top);
                // the largest magnitude to [128, 256), scale bytes from 5 on (lo's is 5 less)
                int e;
                (void)frexpf(__uint_as_float(top), &e);   // top in [2^(e-1), 2^e)
                const int s = top == 0 ? 127 : max(e - 8 + 127, 5);
                const int up = 127 - s;
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v0 = ldexpf(__uint_as_float(xs[b][t][j][i] << 16), up);
                    const float v1 = ldexpf(__uint_as_float(xs[b][t][j][i] & 0xffff0000u), up);
                    const int h = __builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
                    const f32x2 f = __builtin_amdgcn_cvt_pk_f32_fp8(h, false);
                    const int l = __builtin_amdgcn_cvt_pk_fp8_f32((v0 - f[0]) * 32.0f, (v1 - f[1]) * 32.0f, 0, false);
                    if (i & 1) { hi[i / 2] |= (uint32_t)h << 16; lo[i / 2] |= (uint32_t)l << 16; }
                    else { hi[i / 2] = (uint32_t)h & 0xffffu; lo[i / 2] = (uint32_t)l & 0xffffu; }
                }
                const bool finite = top < 0x7f800000u;
                packed |= (finite ? (uint32_t)s : 255u) << (8 * j);
                flag |= finite ? 0u : top > 0x7f800000u ? 2u : 1u;
                const int g = st * 4 + j;
                if (r < toks && g * 64 < sp.row) {
                    uint8_t* d = sp.data + (t0 + r) * sp.row + (g >> 1) * 128 + (g & 1) * 32 + q * 8;
                    *reinterpret_cast<u32x2*>(d) = finite ? u32x2{hi[0], hi[1]} : u32x2{0, 0};
                    *reinterpret_cast<u32x2*>(d + 64) = finite ? u32x2{lo[0], lo[1]} : u32x2{0, 0};
                }
            }
            if (r < toks && q == 0) {
                // rows hold an even number of groups
                uint16_t* d = reinterpret_cast<uint16_t*>(sp.scales + (t0 + r) * (sp.row / 64)) + st * 2;
                d[0] = (uint16_t)packed;
                if (st * 4 + 2 < sp.row / 64) d[1] = (uint16_t)(packed >> 16);
                if (flag) atomicOr(&flags[r], flag);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < D; ++i) fetch(s_begin + i, i);
    __builtin_amdgcn_sched_barrier(0);
    int st = s_begin;
    for (; st + D < s_end; st += D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (split) write_split(st + i, i);
            multiply(st + i, i);
            fetch(st + D + i, i);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int i = 0; i < D; ++i)
        if (st + i < s_end) {
            if (split) write_split(st + i, i);
            multiply(st + i, i);
        }
    if constexpr (NC > 0) {
        constexpr int LD = 16 * NC + 4;
        float* mine = red + wave * (16 * NT * LD);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<f32x4*>(&mine[(t * 16 + m) * LD + c * 16 + 4 * q]) = acc[t][c];
    }
    __syncthreads();
    if constexpr (SPLIT) {
        if (split && threadIdx.x < toks) sp.flags[t0 + threadIdx.x] = (uint8_t)flags[threadIdx.x];
    }
    if constexpr (NC > 0) {
        constexpr int LD = 16 * NC + 4;
        for (int i = threadIdx.x; i < 16 * NT * 4 * NC; i += kSkinnyThreads) {
            const int t = i / (4 * NC), c = (i % (4 * NC)) * 4;
            if (t >= toks || n0 + c >= p.n_out) continue;
            f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kSkinnyWaves; ++w)
                y += *reinterpret_cast<const f32x4*>(&red[w * (16 * NT * LD) + t * LD + c]);
            mx_put4<T>(o, t0 + t, n0 + c, y);
        }
    }
}

// Many tokens.  WT x WC waves, each 16 NT tokens x 16 NC channels, so a tile
// of TT tokens x CC channels per workgroup; the input axis goes by in blocks
// of 64 through three LDS stages, written by loads that store straight into
// LDS two blocks ahead.  A stage holds the tokens' 128 bytes (64 bf16, or the
// 64 hi and 64 lo bytes of the split) and the weights' 32 bytes of codes as
// they are; scale bytes go through registers to a two-stage area ordered so
// that a lane reads the scales of all its rows at once.
//
// bf16 (F8 false): lane q of MFMA j (16x16x32) takes k = 16 q + 8 j ..: one
// 8-byte read of codes serves both MFMAs, expanded in registers.
// Split (F8 true): one scaled MFMA (16x16x128) takes codes as they are times
// hi in its lower and lo in its upper half of k, the same codes in both.  It
// holds lane q's 32 codes for k = 32 q .., but 8-bit operands as k = 16 q ..
// and 64 + 16 q ..; the scale of lane q is that of k = 32 q .. for both.
//
// A wave keeps its tokens' fragments of a block in registers and walks the
// channels, so the next channels' codes arrive while the present ones
// multiply; in the last step of a block each token fragment is replaced by the
// next block's, and the barrier stands before that step, so no wave runs dry
// at it.
template <bool F8, int NT, int NC, int WT, int WC>
struct TileShape {
    static constexpr int TT = 16 * NT * WT, CC = 16 * NC * WC, TH = 64 * WT * WC;
    static constexpr int kX = TT * 128, kW = CC * 32, kStage = kX + kW;
    static constexpr int kScale = 3 * kStage;            // two stages of CC * 2 + TT * 2 bytes
    static constexpr int kBytes = kScale + 2 * 2 * (CC + TT);
    static_assert(TT * 2 == TH && CC * 2 == TH, "per thread one scale byte of each operand, and 4 + 1 loads");
    // the epilogue's rows (bf16, 16 bytes apart) in the stages
    static constexpr int kRow = 16 * NC * 2 + 16;
    static_assert(WT * WC * 16 * kRow <= 3 * kStage, "epilogue rows fit");
};

template <int OA, int OB>
__device__ __forceinline__ f32x4 mfma_f8(i32x8 w, i32x8 x, f32x4 c, int sw, int sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, 0, OA, sw, OB, sx);
}
template <int OA>
__device__ __forceinline__ f32x4 mfma_f8(int ob, i32x8 w, i32x8 x, f32x4 c, int sw, int sx) {
    switch (ob) {
        case 0: return mfma_f8<OA, 0>(w, x, c, sw, sx);
        case 1: return mfma_f8<OA, 1>(w, x, c, sw, sx);
        case 2: return mfma_f8<OA, 2>(w, x, c, sw, sx);
        default: return mfma_f8<OA, 3>(w, x, c, sw, sx);
    }
}
// Byte oa of sw and ob of sx scale the operands (constants once unrolled).
__device__ __forceinline__ f32x4 mfma_f8(int oa, int ob, i32x8 w, i32x8 x, f32x4 c, int sw, int sx) {
    switch (oa) {
        case 0: return mfma_f8<0>(ob, w, x, c, sw, sx);
        case 1: return mfma_f8<1>(ob, w, x, c, sw, sx);
        case 2: return mfma_f8<2>(ob, w, x, c, sw, sx);
        default: return mfma_f8<3>(ob, w, x, c, sw, sx);
    }
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

template <typename T, bool F8, int NT, int NC, int WT, int WC>
__global__ __launch_bounds__(64 * WT * WC, 2) void mx_tile_kernel(MxIn p, MxOut o, MxSplit sp, int tiles_t,
                                                                  int n_end) {
    using S = TileShape<F8, NT, NC, WT, WC>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
    const int wt = wave / WC, wc = wave % WC;
    // consecutive tiles share their channels
    const int64_t t0 = (int64_t)(blockIdx.x % tiles_t) * S::TT;
    const int n0 = (int)(blockIdx.x / tiles_t) * S::CC;
    const int toks = (int)min((int64_t)S::TT, p.n_tok - t0), rows = min(S::CC, n_end - n0);
    const int half = p.n_in / 2, groups = p.n_in / 32, blocks = (groups + 1) / 2;
    const void* xp = F8 ? static_cast<const void*>(sp.data + t0 * sp.row) : p.x + t0 * p.ld_x;
    const auto x_rs = buf_rsrc(xp, F8 ? (int64_t)toks * sp.row : ((toks - 1) * p.ld_x + p.n_in) * 2);
    const auto w_rs = buf_rsrc(p.codes + (int64_t)n0 * half, (int64_t)rows * half);
    const auto s_rs = buf_rsrc(p.scales + (int64_t)n0 * groups, (int64_t)rows * groups);
    const auto e_rs = buf_rsrc(F8 ? sp.scales + t0 * (sp.row / 64) : sp.scales, F8 ? (int64_t)toks * (sp.row / 64) : 0);

    // Loads into LDS: lane l of a wave's load writes 16 bytes at 16 l, i.e.
    // eight rows of tokens or 32 rows of weights.  Slot s of a token row holds
    // chunk s ^ (row / 2) % 8, of a weight row s ^ (row / 8) % 2, so the 16
    // rows of a fragment read spread over all banks.
    int gx[4], xchunk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = wave * 32 + i * 8 + (lane >> 3);
        xchunk[i] = (lane & 7) ^ ((r >> 1) & 7);
        gx[i] = r < toks ? (F8 ? r * sp.row : (int)(r * p.ld_x * 2)) + xchunk[i] * 16 : kOffOOB;
    }
    const int wrow = wave * 32 + (lane >> 1), wchunk = (lane & 1) ^ ((wrow >> 3) & 1);
    const int gw = wrow < rows ? wrow * half + wchunk * 16 : kOffOOB;
    const auto issue = [&](int kb, int st) {
        uint8_t* base = lds + st * S::kStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = gx[i] != kOffOOB && (F8 ? kb < blocks : kb * 64 + xchunk[i] * 8 < p.n_in);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x_rs, (lds_ptr)(base + (wave * 4 + i) * 1024), 16,
                                                     in ? gx[i] + kb * 128 : kOffOOB, 0, 0, 0);
        }
        const bool in = gw != kOffOOB && kb * 2 + wchunk < groups;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rs, (lds_ptr)(base + S::kX + wave * 1024), 16,
                                                 in ? gw + kb * 32 : kOffOOB, 0, 0, 0);
    };
    // Scale bytes: thread tid carries group tid % 2 of row tid / 2.
    const int srow = tid >> 1, sgrp = tid & 1;
    uint32_t sw_in, sx_in = 0;
    const auto issue_scales = [&](int kb) {
        const int g = kb * 2 + sgrp;
        sw_in = __builtin_amdgcn_raw_buffer_load_b8(s_rs, srow < rows && g < groups ? srow * groups + g : kOffOOB, 0, 0);
        if constexpr (F8)
            sx_in = __builtin_amdgcn_raw_buffer_load_b8(
                e_rs, srow < toks && kb < blocks ? srow * (sp.row / 64) + g : kOffOOB, 0, 0);
    };
    const int sw_at = ((srow / (16 * NC) * 16 + (srow & 15)) * 2 + sgrp) * NC + (srow >> 4) % NC;
    const int sx_at = 2 * S::CC + ((srow / (16 * NT) * 16 + (srow & 15)) * 2 + sgrp) * NT + (srow >> 4) % NT;
    const auto put_scales = [&](int kb) {
        uint8_t* base = lds + S::kScale + (kb & 1) * (2 * (S::CC + S::TT));
        base[sw_at] = (uint8_t)sw_in;
        if constexpr (F8) base[sx_at] = (uint8_t)sx_in;
    };

    // Fragment reads.
    const int xkey = (m >> 1) & 7, wkey = (m >> 3) & 1;
    const int xc0 = F8 ? q : 2 * q, xc1 = F8 ? 4 + q : 2 * q + 1;
    const int xr = (wt * 16 * NT + m) * 128, xo0 = xr + 16 * (xc0 ^ xkey), xo1 = xr + 16 * (xc1 ^ xkey);
    const int wo = S::kX + (wc * 16 * NC + m) * 32 +
                   (F8 ? 16 * ((q & 1) ^ wkey) : 16 * ((q >> 1) ^ wkey) + 8 * (q & 1));
    const int swo = ((wc * 16 + m) * 2 + (F8 ? q & 1 : q >> 1)) * NC;
    const int sxo = 2 * S::CC + ((wt * 16 + m) * 2 + (q & 1)) * NT;
    u32x4 xf[NT][2];
    using Codes = std::conditional_t<F8, u32x4, u32x2>;
    Codes wf[2];
    uint32_t sw[2][NC / 4], sx[2];
    const auto read_x = [&](int st, int t) {
        const uint8_t* base = lds + st * S::kStage + t * 2048;
        xf[t][0] = *reinterpret_cast<const u32x4*>(base + xo0);
        xf[t][1] = *reinterpret_cast<const u32x4*>(base + xo1);
    };
    const auto read_w = [&](int st, int c, Codes& w) {
        w = *reinterpret_cast<const Codes*>(lds + st * S::kStage + c * 512 + wo);
    };
    const auto read_scales = [&](int kb, int to) {
        const uint8_t* base = lds + S::kScale + (kb & 1) * (2 * (S::CC + S::TT));
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) sw[to][i] = *reinterpret_cast<const uint32_t*>(base + swo + 4 * i);
        if constexpr (F8) sx[to] = *reinterpret_cast<const uint32_t*>(base + sxo) - (q >> 1) * 0x05050505u;
    };
    f32x4 acc[NT][NC];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    const auto barrier = [&](int kb) {
        // every wave's loads of block kb are done, and its reads of block kb - 1
        // (the last of them before this point)
        __builtin_amdgcn_s_waitcnt(0x0f75);                      // vmcnt(5): one block's loads in flight
        put_scales(kb);
        __builtin_amdgcn_s_waitcnt(0xc07f);                      // lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
    };
    issue_scales(0);
    __builtin_amdgcn_sched_barrier(0);
    issue(0, 0);
    issue(1, 1);
    barrier(0);
    issue_scales(1);
    __builtin_amdgcn_sched_barrier(0);   // the scales' loads come first: the wait counts on it
    issue(2, 2);
#pragma unroll
    for (int t = 0; t < NT; ++t) read_x(0, t);
    read_w(0, 0, wf[0]);
    read_scales(0, 0);

    int st = 0;
    for (int kb = 0; kb < blocks; ++kb) {
        const int nx = st == 2 ? 0 : st + 1;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (c == NC - 1) {
                barrier(kb + 1);
                issue_scales(kb + 2);
                __builtin_amdgcn_sched_barrier(0);
                issue(kb + 3, st);
                read_w(nx, 0, wf[(c + 1) & 1]);
                read_scales(kb + 1, 1);
            } else {
                read_w(st, c + 1, wf[(c + 1) & 1]);
            }
            if constexpr (F8) {
                const Codes& w = wf[c & 1];
                const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const u32x4 h = xf[t][0], l = xf[t][1];
                    const i32x8 b = {(int)h[0], (int)h[1], (int)h[2], (int)h[3],
                                     (int)l[0], (int)l[1], (int)l[2], (int)l[3]};
                    acc[t][c] = mfma_f8(c & 3, t & 3, a, b, acc[t][c], (int)sw[0][c / 4], (int)sx[0]);
                    if (c == NC - 1) read_x(nx, t);
                }
            } else {
                const Codes w = wf[c & 1];
                const float scale = __uint_as_float((sw[0][c / 4] >> (8 * (c & 3)) & 0xffu) << 23);
                const bf16x8 w0 = mx_expand(w[0], scale), w1 = mx_expand(w[1], scale);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        w0, __builtin_bit_cast(bf16x8, xf[t][0]), acc[t][c], 0, 0, 0);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        w1, __builtin_bit_cast(bf16x8, xf[t][1]), acc[t][c], 0, 0, 0);
                    if (c == NC - 1) read_x(nx, t);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) sw[0][i] = sw[1][i];
        sx[0] = sx[1];
        st = nx;
    }
    // the loads past the last block are done before their stages are used again
    __builtin_amdgcn_s_waitcnt(0x0070);                          // vmcnt(0) lgkmcnt(0)
    __syncthreads();

    const int64_t tw = t0 + wt * 16 * NT;
    const int nw = n0 + wc * 16 * NC;
    if constexpr (sizeof(T) == 2) {
        // 16 tokens at a time through LDS, each wave its own rows, so that a
        // token's channels leave in 16-byte pieces side by side
        uint8_t* eb = lds + wave * (16 * S::kRow);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int n = nw + c * 16 + 4 * q;
                if (F8 || n < o.end[3])
                    *reinterpret_cast<u32x2*>(eb + m * S::kRow + (c * 16 + 4 * q) * 2) = pack4(acc[t][c]);
                else if (n < n_end && tw + t * 16 + m < p.n_tok)
                    mx_put4<T>(o, tw + t * 16 + m, n, acc[t][c]);   // gates: fp32
            }
#pragma unroll
            for (int i = lane; i < 32 * NC; i += 64) {
                const int r = i / (2 * NC), c8 = (i % (2 * NC)) * 8;
                const u32x4 v = *reinterpret_cast<const u32x4*>(eb + r * S::kRow + c8 * 2);
                const int64_t tok = tw + t * 16 + r;
                const int n = nw + c8;
                const int end = F8 ? n_end : min(n_end, o.end[3]);
                if (tok >= p.n_tok || n >= end) continue;
                uint32_t nan = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    nan |= (uint32_t)((v[j / 2] >> (16 * (j & 1)) & 0x7fffu) > 0x7f80u) << j;
                if (o.vec8 && n + 8 <= end) {
                    *reinterpret_cast<u32x4*>(mx_at<T>(o, tok, n)) = v;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < end) mx_put<T>(o, tok, n + j, __uint_as_float(v[j / 2] >> (16 * (j & 1)) << 16));
                }
                // A token with an infinity (and no NaN) has no split: its
                // results are infinite or NaN, as the definition has them.
                if constexpr (F8) {
                    if (nan && sp.flags[tok] == 1) {
#pragma unroll 1
                        for (; nan; nan &= nan - 1) {
                            const int j = __ffs((int)nan) - 1;
                            if (n + j < n_end) mx_put<T>(o, tok, n + j, mx_dot(p, tok, n + j));
                        }
                    }
                }
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int64_t tok = tw + t * 16 + m;
                const int n = nw + c * 16 + 4 * q;
                if (tok < p.n_tok && n < n_end) mx_put4<T>(o, tok, n, acc[t][c]);
            }
    }
}

bool fits(const void* p, int64_t ld, int elem, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (vec * elem) == 0 && ld % vec == 0;
}

template <typename T, int NT, int NC, bool SPLIT>
hipError_t skinny(const MxIn& p, const MxOut& o, int c0, const MxSplit& sp, hipStream_t stream) {
    constexpr size_t lds = NC > 0 ? skinny_lds(NT, NC) : 0;
    if (lds > 65536) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_dynamic_lds(&mx_skinny_kernel<T, NT, NC, SPLIT>, lds, &done);
        if (e != hipSuccess) return e;
    }
    const int cols = NC > 0 ? (p.n_out - c0 + 16 * NC - 1) / (16 * NC) : 1;
    const dim3 grid((unsigned)cols, (unsigned)((p.n_tok + 16 * NT - 1) / (16 * NT)));
    hipLaunchKernelGGL((mx_skinny_kernel<T, NT, NC, SPLIT>), grid, dim3(kSkinnyThreads), lds, stream, p, o, c0, sp);
    return hipGetLastError();
}

template <typename T, bool F8, int NT, int NC, int WT, int WC>
hipError_t tile(const MxIn& p, const MxOut& o, const MxSplit& sp, int n_end, hipStream_t stream) {
    using S = TileShape<F8, NT, NC, WT, WC>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_dynamic_lds(&mx_tile_kernel<T, F8, NT, NC, WT, WC>, S::kBytes, &done);
    if (e != hipSuccess) return e;
    const int tiles_t = (int)((p.n_tok + S::TT - 1) / S::TT), tiles_c = (n_end + S::CC - 1) / S::CC;
    hipLaunchKernelGGL((mx_tile_kernel<T, F8, NT, NC, WT, WC>), dim3((unsigned)tiles_t * tiles_c), dim3(S::TH),
                       S::kBytes, stream, p, o, sp, tiles_t, n_end);
    return hipGetLastError();
}

constexpr int64_t kSkinnyTokens = 64;   // up to here the skinny kernel takes all channels

bool use_split(int64_t n_tok, int32_t n_in, gdn_dtype out) {
    return out == GDN_BF16 && n_tok > kSkinnyTokens && n_in >= 512;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

MxSplit split_of(int64_t n_tok, int32_t n_in, void* workspace, size_t* bytes) {
    MxSplit s;
    s.row = (n_in + 63) / 64 * 128;
    const size_t data = up256((size_t)n_tok * s.row), scales = up256((size_t)n_tok * (s.row / 64));
    s.data = static_cast<uint8_t*>(workspace);
    s.scales = s.data + data;
    s.flags = s.scales + scales;
    *bytes = data + scales + up256((size_t)n_tok);
    return s;
}

template <typename T>
hipError_t launch_few(const MxIn& p, const MxOut& o, hipStream_t stream) {
    const MxSplit none{};
    // Bytes that the busiest CU takes in, the tile's tokens and weights: the
    // measure that separates the shapes where the axis is not the limit.
    const auto cost = [&](int nt, int nc) {
        const int64_t wgs = ((p.n_tok + 16 * nt - 1) / (16 * nt)) * ((p.n_out + 16 * nc - 1) / (16 * nc));
        const int64_t toks = std::min<int64_t>(p.n_tok, 16 * nt);
        return std::max<int64_t>(wgs, 256) * (toks * 4 + 16 * nc);
    };
    int best = 0;
    int64_t least = INT64_MAX;
    constexpr int shapes[][2] = {{1, 1}, {1, 2}, {1, 4}, {2, 2}, {2, 4}, {4, 4}};
    for (int i = 0; i < 6; ++i) {
        const int64_t c = cost(shapes[i][0], shapes[i][1]);
        if (c < least) { least = c; best = i; }
    }
    switch (best) {
        case 0: return skinny<T, 1, 1, false>(p, o, 0, none, stream);
        case 1: return skinny<T, 1, 2, false>(p, o, 0, none, stream);
        case 2: return skinny<T, 1, 4, false>(p, o, 0, none, stream);
        case 3: return skinny<T, 2, 2, false>(p, o, 0, none, stream);
        case 4: return skinny<T, 2, 4, false>(p, o, 0, none, stream);
        default: return skinny<T, 4, 4, false>(p, o, 0, none, stream);
    }
}

template <typename T>
hipError_t launch_typed(const MxIn& p, const MxOut& o, void* workspace, hipStream_t stream) {
    if (p.n_tok <= kSkinnyTokens) return launch_few<T>(p, o, stream);
    const bool large = ((p.n_tok + 255) / 256) * ((p.n_out + 255) / 256) >= 256;
    if constexpr (sizeof(T) == 2) {
        if (use_split(p.n_tok, p.n_in, GDN_BF16)) {
            size_t bytes;
            const MxSplit sp = split_of(p.n_tok, p.n_in, workspace, &bytes);
            // the gates keep fp32's accuracy: they go with the split's pass over the tokens
            const int n_end = o.end[3];
            const hipError_t e = n_end < p.n_out ? skinny<T, 2, 4, true>(p, o, n_end, sp, stream)
                                                 : skinny<T, 2, 0, true>(p, o, n_end, sp, stream);
            if (e != hipSuccess) return e;
            return large ? tile<T, true, 4, 8, 4, 2>(p, o, sp, n_end, stream)
                         : tile<T, true, 4, 4, 2, 2>(p, o, sp, n_end, stream);
        }
    }
    const MxSplit none{};
    return large ? tile<T, false, 4, 8, 4, 2>(p, o, none, p.n_out, stream)
                 : tile<T, false, 4, 4, 2, 2>(p, o, none, p.n_out, stream);
}

}  // namespace

// Tiles of one launch (of 256 threads) stay below 2^32 threads.
bool mx_proj_fits(int64_t n_tok, int64_t n_out) {
    return ((n_tok + 63) / 64) * ((n_out + 63) / 64) < (1 << 23);
}

size_t mx_proj_workspace_bytes(int64_t n_tok, int32_t n_in, int32_t n_out) {
    size_t bytes = 0;
    // whichever type the results have
    if (use_split(n_tok, n_in, GDN_BF16)) split_of(n_tok, n_in, nullptr, &bytes);
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
    o.vec8 = n_out % 8 == 0 && fits(y, ld_y, elem, 8);
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
    o.vec4 = o.vec8 = 1;
    for (int i = 0; i < 4; ++i) {
        o.seg[i] = seg[i];
        o.ld[i] = width[i];
        o.end[i] = end += width[i];
        o.vec4 = o.vec4 && fits(seg[i], width[i], elem, 4);
        o.vec8 = o.vec8 && fits(seg[i], width[i], elem, 8);
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
