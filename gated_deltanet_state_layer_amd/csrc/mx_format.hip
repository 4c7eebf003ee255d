// The 4-bit weight format: groups of 32 consecutive weights of a row share a
// scale byte s, worth 2^(s - 127), and each weight is a 4-bit float (sign, two
// exponent bits, one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte,
// the even weight in the low half.  Every product of a code and a scale in
// range is exact in bf16, so a weight read back is the weight the projections
// multiply with.
//
// quantize: s - 127 = floor(log2(largest magnitude of the group)) - 2, so the
// group's largest magnitude falls in [4, 8) steps of the scale; codes round to
// nearest, ties to the even code, and saturate at 6.  Both directions are
// bound by memory (bytes read and written once): 12352 x 2048 from fp32 21.5
// us, back 19.6 us, 5.3 and 5.8 TB/s.
#include <algorithm>

#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kMxThreads = 256;
// A launch holds fewer than 2^32 threads; larger matrices loop.
constexpr int64_t kMaxGrid = 1 << 20;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight fp32 bit patterns of eight consecutive elements.
__device__ __forceinline__ void load8_bits(const uint16_t* p, uint32_t* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = w[i] << 16;
        x[2 * i + 1] = w[i] & 0xffff0000u;
    }
}
// An fp32 matrix comes from a checkpoint and is read once: past the caches
// (12352 x 2048 to codes and back 45.2 -> 41.1 us).  bf16 ones are half the
// size and were slower so (2048 x 4096 10.2 -> 11.2 us).
__device__ __forceinline__ void load8_bits(const float* p, uint32_t* x) {
    const auto* v = reinterpret_cast<const u32x4*>(p);
    const u32x4 a = __builtin_nontemporal_load(v), b = __builtin_nontemporal_load(v + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = a[i];
        x[4 + i] = b[i];
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false));
}

// Four lanes per group, eight weights each.  Magnitudes compare as integers:
// NaN patterns are above infinity's, infinity's above every number's, so a
// group's exponent field alone tells what it holds.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(const T* __restrict__ src, int64_t n8,
                                                                 uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
    // n8 is a multiple of 4: whole groups leave the loop
    for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < n8; i += (int64_t)gridDim.x * kMxThreads) {
    uint32_t w[8], top = 0;
    load8_bits(src + i * 8, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, w[j] & 0x7fffffffu);
    top = quad_max<0xB1>(top);
    top = quad_max<0x4E>(top);
    const uint32_t field = top >> 23;
    const uint32_t s = top == 0 ? 127u : field == 255 ? 255u : field < 2 ? 0u : field - 2;
    // A 255 group's codes mean nothing (the scale is NaN); 0 keeps them defined.
    const float scale = __uint_as_float(s << 23);
    uint32_t c = 0;
    if (s != 255) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[0]), __uint_as_float(w[1]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[2]), __uint_as_float(w[3]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[4]), __uint_as_float(w[5]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[6]), __uint_as_float(w[7]), scale, 3);
    }
    codes[i] = c;
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
}

// Eight weights per lane.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales,
                                                                   int64_t n8, T* __restrict__ dst) {
    for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < n8; i += (int64_t)gridDim.x * kMxThreads) {
    const uint32_t c = codes[i];
    const float scale = __uint_as_float((uint32_t)scales[i >> 2] << 23);
    if constexpr (sizeof(T) == 2) {
        uint4 v;
        v.x = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
        v.y = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
        v.z = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
        v.w = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
        reinterpret_cast<uint4*>(dst)[i] = v;
    } else {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
        const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
        reinterpret_cast<float4*>(dst)[2 * i] = make_float4(a[0], a[1], b[0], b[1]);
        reinterpret_cast<float4*>(dst)[2 * i + 1] = make_float4(d[0], d[1], e[0], e[1]);
    }
    }
}

}  // namespace

hipError_t launch_mx_quantize(int64_t rows, int32_t cols, gdn_dtype dtype, const void* src, void* codes,
                              uint8_t* scales, hipStream_t stream) {
    const int64_t n8 = rows * cols / 8;
    const dim3 grid((unsigned)std::min(kMaxGrid, (n8 + kMxThreads - 1) / kMxThreads));
    auto* c = static_cast<uint32_t*>(codes);
    if (dtype == GDN_BF16)
        hipLaunchKernelGGL(mx_quantize_kernel<uint16_t>, grid, dim3(kMxThreads), 0, stream,
                           static_cast<const uint16_t*>(src), n8, c, scales);
    else
        hipLaunchKernelGGL(mx_quantize_kernel<float>, grid, dim3(kMxThreads), 0, stream,
                           static_cast<const float*>(src), n8, c, scales);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(int64_t rows, int32_t cols, gdn_dtype dtype, const void* codes,
                                const uint8_t* scales, void* dst, hipStream_t stream) {
    const int64_t n8 = rows * cols / 8;
    const dim3 grid((unsigned)std::min(kMaxGrid, (n8 + kMxThreads - 1) / kMxThreads));
    const auto* c = static_cast<const uint32_t*>(codes);
    if (dtype == GDN_BF16)
        hipLaunchKernelGGL(mx_dequantize_kernel<uint16_t>, grid, dim3(kMxThreads), 0, stream, c, scales, n8,
                           static_cast<uint16_t*>(dst));
    else
        hipLaunchKernelGGL(mx_dequantize_kernel<float>, grid, dim3(kMxThreads), 0, stream, c, scales, n8,
                           static_cast<float*>(dst));
    return hipGetLastError();
}

}  // namespace gdn
