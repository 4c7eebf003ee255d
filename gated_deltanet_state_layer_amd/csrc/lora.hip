// Low-rank adapters beside a projection, first half: h[t] = s (x[t] A^T) of each
// token's own adapter, for the projection's epilogue to multiply by B.
//
// h is summed in fp32 and left as three bf16 pieces of eight bits each, which hold its
// 24 bits, in the order in which matrix instructions take them: per token and 16
// ranks the 16 first pieces, the second ones, the third ones (96 bytes); ranks up to
// the next multiple of 16 are zeros.
#include <algorithm>

#include "gdn_common.h"
#include "mfma_split.h"

namespace gdn {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
        s = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), s);
    }
    return s;
}

// Rank r of token t; an infinity or NaN has no further pieces.
__device__ __forceinline__ void put_pieces(uint16_t* h, int64_t t, int blocks, int r, float x) {
    uint16_t* p = h + (t * blocks + r / 16) * 48 + r % 16;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint16_t b = f32_to_bf16(x);
        p[16 * i] = b;
        const float rest = x - bf16_to_f32(b);
        x = fabsf(rest) <= 3.0e38f ? rest : 0.0f;
    }
}

constexpr int kThreads = 256, kWaves = kThreads / 64;

// Few tokens: a wave per token and row of A, whose reads take one trip to memory.
__global__ __launch_bounds__(kThreads) void lora_rows_kernel(LoraArgs l, const uint16_t* x, int64_t ld_x, int n_in,
                                                            int blocks) {
    const int lane = threadIdx.x & 63;
    const int item = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
    const int64_t t = item / (16 * blocks);   // 16 blocks rows are a multiple of the waves: all of one token
    const int r = item % (16 * blocks);
    const int id = l.ids[t];
    if ((unsigned)id >= (unsigned)l.n_adapters) return;
    const uint16_t* xt = x + t * ld_x;
    const uint16_t* a = static_cast<const uint16_t*>(l.a) + ((int64_t)id * l.rank + r) * n_in;
    float s = 0.f;
    if (r < l.rank)
#pragma unroll 4
        for (int i = lane * 8; i < n_in; i += 512)
            s = dot8(*reinterpret_cast<const u32x4*>(xt + i), *reinterpret_cast<const u32x4*>(a + i), s);
    s = wave_sum(s);
    if (lane == 0) put_pieces(static_cast<uint16_t*>(l.h), t, blocks, r, l.scale[id] * s);
}

// Many tokens: 16 of them to a workgroup, the input axis split over its eight waves,
// on the matrix cores (A's rows times the tokens), the partial sums added in LDS.
// One pass per adapter among the 16 tokens; each token keeps its own.
constexpr int kTileWaves = 8, kTileThreads = kTileWaves * 64;

template <int RB>
__global__ __launch_bounds__(kTileThreads) void lora_tile_kernel(LoraArgs l, const uint16_t* x, int64_t ld_x,
                                                                int64_t n_tok, int n_in, int blocks, int r0) {
    __shared__ __align__(16) float part[kTileWaves][16][16 * RB + 4];   // [wave][token][rank]
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * 16, t = min(t0 + m, n_tok - 1);
    const int id = t0 + m < n_tok ? l.ids[t] : -1;
    const bool has = (unsigned)id < (unsigned)l.n_adapters;
    const int steps = n_in / 32, per = (steps + kTileWaves - 1) / kTileWaves;
    const int begin = wave * per, end = min(steps, begin + per);
    const uint16_t* xt = x + t * ld_x + 8 * q;
    uint64_t left = __ballot(has);
    while (left) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const bool mine = has && id == cur;
        left &= ~__ballot(mine);
        const uint16_t* a[RB];   // rows past the rank repeat the last one; what they give is dropped
#pragma unroll
        for (int b = 0; b < RB; ++b)
            a[b] = static_cast<const uint16_t*>(l.a) +
                   ((int64_t)cur * l.rank + min(r0 + 16 * b + m, l.rank - 1)) * n_in + 8 * q;
        f32x4 acc[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = begin; s < end; ++s) {
            const bf16x8 xv = *reinterpret_cast<const bf16x8*>(xt + s * 32);
#pragma unroll
            for (int b = 0; b < RB; ++b)
                acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(a[b] + s * 32), xv,
                                                                 acc[b], 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) *reinterpret_cast<f32x4*>(&part[wave][m][16 * b + 4 * q]) = acc[b];
        __syncthreads();
        const float scale = l.scale[cur];
        for (int i = threadIdx.x; i < 16 * 16 * RB; i += kTileThreads) {
            const int tok = i / (16 * RB), r = i % (16 * RB);
            if (__shfl(mine ? 1 : 0, tok) == 0) continue;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kTileWaves; ++w) sum += part[w][tok][r];
            if (r0 + r < 16 * blocks)
                put_pieces(static_cast<uint16_t*>(l.h), t0 + tok, blocks, r0 + r, r0 + r < l.rank ? scale * sum : 0.f);
        }
        __syncthreads();
    }
}

}  // namespace

size_t lora_workspace_bytes(int64_t n_tok, int32_t rank) { return (size_t)n_tok * ((rank + 15) / 16) * 96; }

hipError_t launch_lora_shrink(int64_t n_tok, int32_t n_in, const void* x, int64_t ld_x, const LoraArgs& l,
                              hipStream_t stream) {
    const int blocks = (l.rank + 15) / 16;
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    if (n_tok <= 128) {
        hipLaunchKernelGGL(lora_rows_kernel, dim3((unsigned)(n_tok * blocks * 16 / kWaves)), dim3(kThreads), 0, stream,
                           l, xp, ld_x, n_in, blocks);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((n_tok + 15) / 16));
    for (int b = 0; b < blocks;) {
        const int r0 = 16 * b, more = blocks - b;
        if (more >= 2) {
            hipLaunchKernelGGL(lora_tile_kernel<2>, grid, dim3(kTileThreads), 0, stream, l, xp, ld_x, n_tok, n_in,
                               blocks, r0);
            b += 2;
        } else {
            hipLaunchKernelGGL(lora_tile_kernel<1>, grid, dim3(kTileThreads), 0, stream, l, xp, ld_x, n_tok, n_in,
                               blocks, r0);
            b += 1;
        }
    }
    return hipGetLastError();
}

}  // namespace gdn
