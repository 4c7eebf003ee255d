// Low-rank adapters beside a projection, first half: h[t] = s (x[t] A^T) of each
// token's own adapter, in fp32, for the projection's epilogue to multiply by B.
#include <algorithm>

#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
        s = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), s);
    }
    return s;
}

// One workgroup per token in turn, a wave per row of A in turn.
__global__ __launch_bounds__(kThreads) void lora_token_kernel(LoraArgs l, const uint16_t* x, int64_t ld_x,
                                                             int64_t n_tok, int n_in, int ldh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x) {
        const int id = l.ids[t];
        if ((unsigned)id >= (unsigned)l.n_adapters) continue;
        const uint16_t* xt = x + t * ld_x;
        const uint16_t* a = static_cast<const uint16_t*>(l.a) + (int64_t)id * l.rank * n_in;
        const float scale = l.scale[id];
        for (int r = wave; r < ldh; r += kWaves) {
            float s = 0.f;
            if (r < l.rank)
                for (int i = lane * 8; i < n_in; i += 512)
                    s = dot8(*reinterpret_cast<const u32x4*>(xt + i),
                             *reinterpret_cast<const u32x4*>(a + (int64_t)r * n_in + i), s);
            s = wave_sum(s);
            if (lane == 0) l.h[t * ldh + r] = scale * s;
        }
    }
}

}  // namespace

size_t lora_workspace_bytes(int64_t n_tok, int32_t rank) { return (size_t)n_tok * ((rank + 15) / 16 * 16) * sizeof(float); }

hipError_t launch_lora_shrink(int64_t n_tok, int32_t n_in, const void* x, int64_t ld_x, const LoraArgs& l,
                              hipStream_t stream) {
    hipLaunchKernelGGL(lora_token_kernel, dim3((unsigned)std::min<int64_t>(n_tok, 1 << 20)), dim3(kThreads), 0,
                       stream, l, static_cast<const uint16_t*>(x), ld_x, n_tok, n_in, (l.rank + 15) / 16 * 16);
    return hipGetLastError();
}

}  // namespace gdn
