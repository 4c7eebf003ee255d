// Loads from a bounded buffer straight into LDS (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

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

// An offset, or one past every descriptor.  Opaque to the compiler, which would
// otherwise split the load into two branches with a wait between them.
__device__ __forceinline__ int offset_if(bool in, int offset) {
    int v = in ? offset : kOffOOB;
    asm("" : "+v"(v));
    return v;
}

}  // namespace gdn
