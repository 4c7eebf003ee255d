// Low-rank adapters beside a projection, first half: h[t] = s (x[t] A^T) of each
// token's own adapter, for the projection's epilogue to multiply by B.
//
// h is summed in fp32 and left as three bf16 pieces of eight bits each, which hold its
// 24 bits, in the order in which matrix instructions take them: per token and 16
// ranks the 16 first pieces, the second ones, the third ones (96 bytes); ranks up to
// the next multiple of 16 are zeros.  One bf16 piece would round h to 8 bits; fp32
// would need these splits in every tile of the projection.
#include <algorithm>

#include "gdn_common.h"
#include "lds_load.h"
#include "mfma_split.h"

namespace gdn {
namespace {

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
// 2.7 us for one token of 4096 inputs, 3.5 for 64 of 2048: launch and trip.
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

// Many tokens: 16 of them by 16 RB ranks to a workgroup, on the matrix cores (A's rows
// times the tokens), the partial sums of its four waves added in LDS.  A wave takes
// every fourth 128 inputs, two steps of them through LDS of its own (no barrier) by
// loads that store straight into it: they read rows in pieces of 256 bytes from
// neighbouring lanes, where loads in the matrix operands' layout take 64 bytes each
// (8192 tokens of 2048 inputs at rank 16: 16 us, 34 MB at 2.1 TB/s; 25 in that layout).
// One pass per adapter among the 16 tokens, each token keeping its own; of several
// passes workgroup z takes every gridDim.z-th, where tokens alone leave CUs idle (a
// projection of 500 tokens at rank 32, eight adapters in turn: 61 us, 81 with z = 1).
constexpr int kTileWaves = 4, kTileThreads = kTileWaves * 64;

template <int RB>
__global__ __launch_bounds__(kTileThreads) void lora_tile_kernel(LoraArgs l, const uint16_t* x, int64_t ld_x,
                                                                int64_t n_tok, int n_in, int blocks) {
    constexpr int kRows = 16 * (1 + RB), kStage = kRows * 256, kLoads = kRows / 4, LD = 16 * RB + 4;
    extern __shared__ __align__(16) uint8_t lds[];   // [wave][2 steps][16 tokens, 16 RB rows of A][256]
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const int toks = (int)min((int64_t)16, n_tok - t0), r0 = blockIdx.y * (16 * RB), rows = min(16 * RB, l.rank - r0);
    const int id = m < toks ? l.ids[t0 + m] : -1;
    const bool has = (unsigned)id < (unsigned)l.n_adapters;
    const int steps = (n_in + 127) / 128;
    const auto x_rs = buf_rsrc(x + t0 * ld_x, ((toks - 1) * ld_x + n_in) * 2);
    uint8_t* mine = lds + wave * (2 * kStage);
    // Slot s of a row's 16 holds chunk s ^ row % 16, so the 16 rows of a fragment read
    // spread over all banks.
    int chunk[4], at[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = i * 4 + q;
        if (i < 4) chunk[i] = m ^ (r & 15);
        at[i] = i < 4 ? offset_if(r < toks, (int)(r * ld_x) * 2 + chunk[i] * 16)
                      : offset_if(r - 16 < rows, (r - 16) * n_in * 2 + chunk[i & 3] * 16);
    }
    uint64_t left = __ballot(has);
    for (unsigned pass = 0; left; ++pass) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t tokens = __ballot(has && id == cur);
        left &= ~tokens;
        if (pass % gridDim.z != blockIdx.z) continue;
        const auto a_rs = buf_rsrc(static_cast<const uint16_t*>(l.a) + ((int64_t)cur * l.rank + r0) * n_in,
                                   (int64_t)rows * n_in * 2);
        const auto fetch = [&](int s, int b) {   // past the row's end zeros
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_lds16(i < 4 ? x_rs : a_rs, mine + b * kStage + i * 1024,
                           offset_if(s * 128 + chunk[i & 3] * 8 < n_in, at[i]), s * 256);
        };
        f32x4 acc[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (wave < steps) fetch(wave, 0);
        if (wave + kTileWaves < steps) fetch(wave + kTileWaves, 1);
        for (int s = wave, b = 0; s < steps; s += kTileWaves, b ^= 1) {
            // this step's loads have arrived, the next one's may be on their way
            if (s + kTileWaves < steps) __builtin_amdgcn_s_waitcnt(0x0f70 | kLoads);
            else __builtin_amdgcn_s_waitcnt(0x0f70);
            __builtin_amdgcn_sched_barrier(0);
            const uint8_t* base = mine + b * kStage + m * 256;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int slot = ((q * 4 + j) ^ m) * 16;
                const bf16x8 xv = *reinterpret_cast<const bf16x8*>(base + slot);
#pragma unroll
                for (int c = 0; c < RB; ++c)
                    acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        *reinterpret_cast<const bf16x8*>(base + (1 + c) * 4096 + slot), xv, acc[c], 0, 0, 0);
            }
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): the stage is read
            __builtin_amdgcn_sched_barrier(0);
            if (s + 2 * kTileWaves < steps) fetch(s + 2 * kTileWaves, b);
        }
        __syncthreads();   // every wave is done with its stages
        float* part = reinterpret_cast<float*>(lds);   // [wave][token][LD]
#pragma unroll
        for (int c = 0; c < RB; ++c)
            *reinterpret_cast<f32x4*>(&part[(wave * 16 + m) * LD + 16 * c + 4 * q]) = acc[c];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            const int tok = threadIdx.x / 16, r = 16 * c + threadIdx.x % 16;
            if (!(tokens >> tok & 1) || r0 + r >= 16 * blocks) continue;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kTileWaves; ++w) sum += part[(w * 16 + tok) * LD + r];
            put_pieces(static_cast<uint16_t*>(l.h), t0 + tok, blocks, r0 + r, r < rows ? l.scale[cur] * sum : 0.f);
        }
        __syncthreads();
    }
}

template <int RB>
hipError_t tiles(int64_t n_tok, int32_t n_in, const uint16_t* x, int64_t ld_x, const LoraArgs& l, hipStream_t stream) {
    constexpr int lds = kTileWaves * 2 * 16 * (1 + RB) * 256;
    static std::atomic<uint64_t> done{0};
    if (lds > 65536) {
        const hipError_t e = allow_dynamic_lds(&lora_tile_kernel<RB>, lds, &done);
        if (e != hipSuccess) return e;
    }
    const int blocks = (l.rank + 15) / 16, y = (blocks + RB - 1) / RB;
    const int64_t n = (n_tok + 15) / 16, z = std::min<int64_t>(16, std::max<int64_t>(1, 256 / (n * y)));
    hipLaunchKernelGGL(lora_tile_kernel<RB>, dim3((unsigned)n, y, (unsigned)z), dim3(kTileThreads), lds, stream, l, x,
                       ld_x, n_tok, n_in, blocks);
    return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int64_t n_tok, int32_t rank) { return (size_t)n_tok * ((rank + 15) / 16) * 96; }

hipError_t launch_lora_shrink(int64_t n_tok, int32_t n_in, const void* x, int64_t ld_x, const LoraArgs& l,
                              hipStream_t stream) {
    const int blocks = (l.rank + 15) / 16;
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    // Rows up to here, which do not mind how many adapters there are.  Tiles and rows, with
    // a projection 2048 -> 256 behind them at rank 16: 64 tokens 8.2 and 6.9 us; 500 tokens
    // 9.3 and 9.8 with four adapters in turn, 11.9 and 9.8 with 64; 1000 tokens at rank 32
    // 13.1 and 19.2 with four.
    if (n_tok * blocks <= 768) {
        hipLaunchKernelGGL(lora_rows_kernel, dim3((unsigned)(n_tok * blocks * 16 / kWaves)), dim3(kThreads), 0, stream,
                           l, xp, ld_x, n_in, blocks);
        return hipGetLastError();
    }
    return blocks == 1 ? tiles<1>(n_tok, n_in, xp, ld_x, l, stream) : tiles<2>(n_tok, n_in, xp, ld_x, l, stream);
}

}  // namespace gdn
