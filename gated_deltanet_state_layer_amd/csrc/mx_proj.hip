// Projections with 4-bit weights: y = x W^T, x bf16, W in the format of
// mx_format.hip, fp32 accumulation on the bf16 matrix cores.  A weight (code
// times a power of two) is exact in bf16, so products are exact in fp32 and
// no rounding is added to the weights.
//
// Operand layout.  A step covers 128 of the input axis (four groups).  Lane
// l = 16 q + m of a wave holds row m's group q as one 16-byte load (32 codes,
// one scale byte); MFMA j of the four (16x16x32) takes codes 8j .. 8j+7, so
// the k index of lane q, element i is 32 q + 8 j + i, and the x operand reads
// the same k: 16 bytes at 32 q + 8 j of token m.  W is the A operand, so a
// lane's four results are consecutive channels of one token.
#include <algorithm>

#include "gdn_common.h"
#include "mfma_split.h"

namespace gdn {
namespace {

constexpr int kRsrcWord3 = 0x00020000;
constexpr int kOffOOB = 0x7ffffff0;   // past every descriptor: loads return zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, kRsrcWord3);
}

// Where the output channels go: [0, end[0]) to seg[0], [end[0], end[1]) to
// seg[1], and so on, ld elements between tokens; from gate_begin on, fp32
// gates a and b of h_v channels each.  A plain projection has one segment.
struct MxOut {
    void* seg[4];
    int64_t ld[4];
    int end[4];
    float *a, *b;
    int h_v, n_out;
    int vec4;   // segment starts, strides and ends are multiples of four elements
};

template <typename T>
__device__ __forceinline__ void mx_put(const MxOut& o, int64_t t, int n, float y) {
    int s = 0, base = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (n >= o.end[i]) { s = i + 1; base = o.end[i]; }
    if (n < o.end[3]) Io<T>::store(static_cast<T*>(o.seg[s]), t * o.ld[s] + n - base, y);
    else if (n < o.end[3] + o.h_v) o.a[t * o.h_v + n - o.end[3]] = 1.0f / (1.0f + expf(y));
    else o.b[t * o.h_v + n - o.end[3] - o.h_v] = 1.0f / (1.0f + expf(-y));
}

// Channels n .. n+3 (n a multiple of four) of token t.
template <typename T>
__device__ __forceinline__ void mx_put4(const MxOut& o, int64_t t, int n, f32x4 y) {
    if (o.vec4 && n < o.end[3]) {
        int s = 0, base = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (n >= o.end[i]) { s = i + 1; base = o.end[i]; }
        T* p = static_cast<T*>(o.seg[s]) + t * o.ld[s] + n - base;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint2*>(p) =
                make_uint2(f32_to_bf16(y[0]) | (uint32_t)f32_to_bf16(y[1]) << 16,
                           f32_to_bf16(y[2]) | (uint32_t)f32_to_bf16(y[3]) << 16);
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < o.n_out) mx_put<T>(o, t, n + i, y[i]);
}

// Eight codes (one register) times their group's scale, in bf16.
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

// Four waves, 64 channels x 64 tokens: wave w holds channels 16 w .. 16 w + 15
// of the tile and all its tokens, operands straight from memory.
constexpr int kTileThreads = 256;

template <typename T>
__global__ __launch_bounds__(kTileThreads) void mx_proj_tile_kernel(MxIn p, MxOut o, int tiles_n) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    const int64_t t0 = (int64_t)(blockIdx.x / tiles_n) * 64;
    const int n0 = (blockIdx.x % tiles_n) * 64 + wave * 16;
    if (n0 >= p.n_out) return;
    const int rows = min(16, p.n_out - n0), toks = (int)min((int64_t)64, p.n_tok - t0);
    const int half = p.n_in / 2, groups = p.n_in / 32;
    const auto w_rs = buf_rsrc(p.codes + (int64_t)n0 * half, (int64_t)rows * half);
    const auto s_rs = buf_rsrc(p.scales + (int64_t)n0 * groups, (int64_t)rows * groups);
    const auto x_rs = buf_rsrc(p.x + t0 * p.ld_x, ((toks - 1) * p.ld_x + p.n_in) * 2);
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int g0 = 0; g0 < groups; g0 += 4) {
        const int g = g0 + q;
        const bool in = g < groups;
        const auto w = __builtin_amdgcn_raw_buffer_load_b128(w_rs, in && m < rows ? m * half + g * 16 : kOffOOB, 0, 0);
        const uint32_t s = __builtin_amdgcn_raw_buffer_load_b8(s_rs, in && m < rows ? m * groups + g : kOffOOB, 0, 0);
        const float scale = __uint_as_float((s & 0xffu) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 wf = mx_expand(w[j], scale);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = i * 16 + m;
                const int off = in && t < toks ? (int)(t * p.ld_x + g * 32 + j * 8) * 2 : kOffOOB;
                const auto xf = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(x_rs, off, 0, 0));
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf, acc[i], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + i * 16 + m;
        const int n = n0 + 4 * q;
        if (t < p.n_tok && n < p.n_out) mx_put4<T>(o, t, n, acc[i]);
    }
}

template <typename T>
hipError_t launch_typed(const MxIn& p, const MxOut& o, hipStream_t stream) {
    const int tiles_n = (p.n_out + 63) / 64;
    const int64_t tiles = tiles_n * ((p.n_tok + 63) / 64);
    hipLaunchKernelGGL(mx_proj_tile_kernel<T>, dim3((unsigned)tiles), dim3(kTileThreads), 0, stream, p, o, tiles_n);
    return hipGetLastError();
}

bool fits4(const void* p, int64_t ld, int elem) {
    return reinterpret_cast<uintptr_t>(p) % (4 * elem) == 0 && ld % 4 == 0;
}

}  // namespace

// Tiles of one launch (of 256 threads) stay below 2^32 threads.
bool mx_proj_fits(int64_t n_tok, int64_t n_out) {
    return ((n_tok + 63) / 64) * ((n_out + 63) / 64) < (1 << 23);
}

size_t mx_proj_workspace_bytes(int64_t n_tok, int32_t n_in, int32_t n_out) { return 0; }

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
    o.vec4 = n_out % 4 == 0 && fits4(y, ld_y, y_dtype == GDN_BF16 ? 2 : 4);
    return y_dtype == GDN_BF16 ? launch_typed<uint16_t>(p, o, stream) : launch_typed<float>(p, o, stream);
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
    o.vec4 = 1;
    for (int i = 0; i < 4; ++i) {
        o.seg[i] = seg[i];
        o.ld[i] = width[i];
        o.end[i] = end += width[i];
        o.vec4 = o.vec4 && fits4(seg[i], width[i], elem);
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
