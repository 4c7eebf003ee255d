// The norms around the layer core.
//
// block_norm closes one block and opens the next: with the block's output y,
//     u  = y                 or   u = w_post * y / sqrt(mean(y^2) + eps)
//     r' = r + res_scale * u                     (stored in the residual type)
//     x  = (w_offset + w_pre) * r' / sqrt(mean(r'^2) + eps)
// over the hidden size, from one read of y and r.  The second norm uses the
// unrounded fp32 sum r', so its input does not depend on the residual type.
//
// gated_norm follows the core: per token and value head,
//     out = w * o / sqrt(mean(o^2) + eps) * z * sigmoid(z).
//
// Both are bound by memory: every element is read and written once, rows stay
// in registers between the sum of squares and the scaling, and all arithmetic
// is fp32 (squares of rows of 16384 elements included).  8192 tokens of 2048
// with an fp32 residual 38.3 us, 8192 x 32 heads of 128 in bf16 36.6 us: 5.3
// and 5.5 TB/s, where a large copy reaches 5.0.  One row 2.2 us, the launch
// alone 1.9.  Non-temporal stores took 38.3 to 36.1 us, but the next call reads
// what they would keep out of the cache.
#include <algorithm>

#include "gdn_common.h"

namespace gdn {
namespace {

// Eight consecutive elements as one (bf16) or two (fp32) 16-byte accesses.
__device__ __forceinline__ void load8(const uint16_t* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = f32_to_bf16(x[2 * i]) | (uint32_t)f32_to_bf16(x[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// fp32 elements at any address: 16-byte accesses need only four-byte alignment.
__device__ __forceinline__ void load8_any(const float* p, float* x) { __builtin_memcpy(x, p, 32); }
__device__ __forceinline__ void store8_any(float* p, const float* x) { __builtin_memcpy(p, x, 32); }

constexpr int kNormThreads = 256;
// A launch holds fewer than 2^32 threads; larger calls loop.
constexpr int64_t kMaxGrid = 1 << 20;

struct BlockNorm {
    const void *y, *r;
    const float *w_post, *w_pre;
    void *r_out, *x;
    int64_t n_tok, ld_y, ld_r, ld_ro, ld_x;
    int hidden;
    float res_scale, w_offset, inv_hidden, eps;
};

// How a row is read and written: in aligned 16-byte accesses; in unaligned ones
// with a ragged last vector (fp32 operands of odd widths and strides); element
// by element (where an operand is bf16, and fp32 rows of up to 2048).
enum class Rows { kAligned, kUnaligned, kElements };

// One workgroup of TPR threads per row.  Element j of vector i of thread t is
// column (i * TPR + t) * 8 + j, and column (8 i + j) * TPR + t by elements
// (neighbouring threads read neighbouring elements).
template <typename TIO, typename TR, int TPR, int NV, Rows ROWS>
__global__ __launch_bounds__(TPR) void block_norm_kernel(BlockNorm p) {
    __shared__ float red[2][TPR / 64];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const auto col = [&](int i, int j) { return ROWS != Rows::kElements ? (i * TPR + t) * 8 + j : (8 * i + j) * TPR + t; };
    const auto row_sum = [&](float s, int slot) {
        s = wave_sum(s);
        if (lane == 0) red[slot][wave] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) s += red[slot][w];
        return s;
    };
    const auto read = [&](const auto* src, float* v, int i) {
        if constexpr (ROWS == Rows::kAligned) {
            if (col(i, 0) < p.hidden) load8(src + col(i, 0), v);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.f;
        } else {
            if constexpr (ROWS == Rows::kUnaligned)
                if (col(i, 7) < p.hidden) return load8_any(src + col(i, 0), v);
            using T = std::remove_cv_t<std::remove_pointer_t<decltype(src)>>;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = col(i, j) < p.hidden ? Io<T>::load(src, col(i, j)) : 0.f;
        }
    };
    const auto write = [&](auto* dst, const float* v, int i) {
        if constexpr (ROWS == Rows::kAligned) {
            if (col(i, 0) < p.hidden) store8(dst + col(i, 0), v);
        } else {
            if constexpr (ROWS == Rows::kUnaligned)
                if (col(i, 7) < p.hidden) return store8_any(dst + col(i, 0), v);
            using T = std::remove_pointer_t<decltype(dst)>;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col(i, j) < p.hidden) Io<T>::store(dst, col(i, j), v[j]);
        }
    };
    for (int64_t row = blockIdx.x; row < p.n_tok; row += gridDim.x) {
    float h[NV][8];
    const auto* r = static_cast<const TR*>(p.r) + row * p.ld_r;
#pragma unroll
    for (int i = 0; i < NV; ++i) read(r, h[i], i);
    if (p.y) {
        float u[NV][8];
        const auto* y = static_cast<const TIO*>(p.y) + row * p.ld_y;
#pragma unroll
        for (int i = 0; i < NV; ++i) read(y, u[i], i);
        if (p.w_post) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(u[i][j], u[i][j], s);
            const float inv = 1.0f / sqrtf(row_sum(s, 0) * p.inv_hidden + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float w[8];
                read(p.w_post, w, i);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] *= inv * w[j];
            }
        }
        auto* ro = static_cast<TR*>(p.r_out) + row * p.ld_ro;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = fmaf(p.res_scale, u[i][j], h[i][j]);
            write(ro, h[i], i);
        }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
    const float inv = 1.0f / sqrtf(row_sum(s, 1) * p.inv_hidden + p.eps);
    auto* x = static_cast<TIO*>(p.x) + row * p.ld_x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[8];
        read(p.w_pre, w, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] *= inv * (p.w_offset + w[j]);
        write(x, h[i], i);
    }
    __syncthreads();   // red is free for the next row
    }
}

template <typename TIO, typename TR, Rows ROWS>
void launch_block_norm_rows(const BlockNorm& p, hipStream_t stream) {
    const dim3 grid((unsigned)std::min<int64_t>(p.n_tok, kMaxGrid));
    const int vecs = (p.hidden + 7) / 8;
    // A vector a thread as far as a workgroup reaches, and no fewer than 256
    // threads: with 256 at every width 3000 x 5003 (bf16, fp32 residual, element by
    // element) took 134.9 us, 78.5 so, and 64 x 4096 in fp32 3.6 us, 3.2 so.
    if (vecs <= 256)
        hipLaunchKernelGGL((block_norm_kernel<TIO, TR, 256, 1, ROWS>), grid, dim3(256), 0, stream, p);
    else if (vecs <= 512)
        hipLaunchKernelGGL((block_norm_kernel<TIO, TR, 512, 1, ROWS>), grid, dim3(512), 0, stream, p);
    else if (vecs <= 1024)
        hipLaunchKernelGGL((block_norm_kernel<TIO, TR, 1024, 1, ROWS>), grid, dim3(1024), 0, stream, p);
    else
        hipLaunchKernelGGL((block_norm_kernel<TIO, TR, 1024, 2, ROWS>), grid, dim3(1024), 0, stream, p);
}

template <typename TIO, typename TR>
void launch_block_norm_typed(const BlockNorm& p, bool aligned, hipStream_t stream) {
    if (aligned) return launch_block_norm_rows<TIO, TR, Rows::kAligned>(p, stream);
    // unaligned vectors pay above 2048 elements (fp32: 1237 x 1999 9.5 us by
    // elements, 10.1 so; 3000 x 5003 62.7 and 53.2)
    if constexpr (sizeof(TIO) == 4 && sizeof(TR) == 4)
        if (p.hidden > 2048) return launch_block_norm_rows<TIO, TR, Rows::kUnaligned>(p, stream);
    launch_block_norm_rows<TIO, TR, Rows::kElements>(p, stream);
}

struct GatedNorm {
    const void *o, *z;
    const float* w;
    void* out;
    int64_t n_heads, ld_o, ld_z, ld_out;   // heads in all; strides between tokens
    int h_v;
    float eps;
};

// bf16 outputs take the fast exponential and reciprocal, a few roundings of
// fp32 less exact: of 16.4 million, 225 differ from the float64 result's rounding
// and 170 with the accurate ones, which take 44.7 us for 36.7 (8192 x 32 x 128).
// fp32 outputs keep those roundings, and take the accurate ones.
__device__ __forceinline__ float silu_of(float z, uint16_t) { return silu(z); }
__device__ __forceinline__ float silu_of(float z, float) { return z / (1.0f + expf(-z)); }

// D / 8 lanes per (token, head), eight elements each.
template <typename TIO, typename TO, int D>
__global__ __launch_bounds__(kNormThreads) void gated_norm_kernel(GatedNorm p) {
    constexpr int L = D / 8;
    constexpr int G = kNormThreads / L;
    const int c = (threadIdx.x % L) * 8;
    for (int64_t g = (int64_t)blockIdx.x * G + threadIdx.x / L; g < p.n_heads; g += (int64_t)gridDim.x * G) {
    const int64_t tok = g / p.h_v;
    const int64_t off = (g - tok * p.h_v) * D + c;
    float o[8], z[8], w[8];
    load8(static_cast<const TIO*>(p.o) + tok * p.ld_o + off, o);
    load8(static_cast<const TIO*>(p.z) + tok * p.ld_z + off, z);
    load8(p.w + c, w);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(o[j], o[j], s);
    const float inv = 1.0f / sqrtf(group_sum<L>(s) * (1.0f / D) + p.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = o[j] * inv * w[j] * silu_of(z[j], TO());
    store8(static_cast<TO*>(p.out) + tok * p.ld_out + off, o);
    }
}

template <typename TIO, typename TO>
void launch_gated_norm_typed(const GatedNorm& p, int d, hipStream_t stream) {
    const auto grid = [&](int lanes) {
        return dim3((unsigned)std::min(kMaxGrid, (p.n_heads * lanes + kNormThreads - 1) / kNormThreads));
    };
    if (d == 32)
        hipLaunchKernelGGL((gated_norm_kernel<TIO, TO, 32>), grid(4), dim3(kNormThreads), 0, stream, p);
    else if (d == 64)
        hipLaunchKernelGGL((gated_norm_kernel<TIO, TO, 64>), grid(8), dim3(kNormThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((gated_norm_kernel<TIO, TO, 128>), grid(16), dim3(kNormThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_block_norm(int64_t n_tok, int32_t hidden, gdn_dtype io_dtype, gdn_dtype res_dtype,
                             const void* y, int64_t ld_y, const float* w_post, float res_scale,
                             const void* r, int64_t ld_r, void* r_out, int64_t ld_ro,
                             const float* w_pre, float w_offset, float eps, void* x, int64_t ld_x,
                             hipStream_t stream) {
    const BlockNorm p{y, r, w_post, w_pre, r_out, x, n_tok, ld_y, ld_r, ld_ro, ld_x, hidden,
                      res_scale, w_offset, 1.0f / (float)hidden, eps};
    // 16-byte accesses need whole vectors and aligned rows in every operand.
    const auto ok = [](const void* ptr, int64_t ld) {
        return ptr == nullptr || (((uintptr_t)ptr & 15) == 0 && ld % 8 == 0);
    };
    const bool vec = hidden % 8 == 0 && ok(y, ld_y) && ok(r, ld_r) && ok(r_out, ld_ro) && ok(x, ld_x) &&
                     ok(w_post, 0) && ok(w_pre, 0);
    const bool io16 = io_dtype == GDN_BF16, r16 = res_dtype == GDN_BF16;
    if (io16 && r16) launch_block_norm_typed<uint16_t, uint16_t>(p, vec, stream);
    else if (io16) launch_block_norm_typed<uint16_t, float>(p, vec, stream);
    else if (r16) launch_block_norm_typed<float, uint16_t>(p, vec, stream);
    else launch_block_norm_typed<float, float>(p, vec, stream);
    return hipGetLastError();
}

hipError_t launch_gated_norm(const gdn_pool* pool, int64_t n_tok, const void* o, int64_t ld_o,
                             const void* z, int64_t ld_z, const float* w, float eps,
                             gdn_dtype out_dtype, void* out, int64_t ld_out, hipStream_t stream) {
    const GatedNorm p{o, z, w, out, n_tok * pool->view.h_v, ld_o, ld_z, ld_out, pool->view.h_v, eps};
    const bool in16 = pool->desc.io_dtype == GDN_BF16, out16 = out_dtype == GDN_BF16;
    if (in16 && out16) launch_gated_norm_typed<uint16_t, uint16_t>(p, pool->view.d, stream);
    else if (in16) launch_gated_norm_typed<uint16_t, float>(p, pool->view.d, stream);
    else if (out16) launch_gated_norm_typed<float, uint16_t>(p, pool->view.d, stream);
    else launch_gated_norm_typed<float, float>(p, pool->view.d, stream);
    return hipGetLastError();
}

}  // namespace gdn
