// Pool bookkeeping kernels: zero fill (pool creation, error-word clear) and
// slot reset.  Both write with 16-byte vector stores; no memset nodes are
// used, so the calls can be recorded into a HIP graph.
#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void fill_zero_kernel(float4* p, size_t n16) {
    const size_t stride = (size_t)gridDim.x * kThreads;
    for (size_t j = (size_t)blockIdx.x * kThreads + threadIdx.x; j < n16; j += stride)
        p[j] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// A reused request slot starts from zero: clear its state tiles and conv
// windows and empty its verify rings for every layer ("Project: adding the hybrid model Qwen3.5",
// "What to do", row "State").  grid = (blocks per slot, n entries).
__global__ __launch_bounds__(kThreads) void slot_reset_kernel(PoolView P, const int32_t* slot_ids,
                                                             size_t state16_per_slot,
                                                             size_t window16_per_slot) {
    const int slot = slot_ids[blockIdx.y];
    if (slot < 0) return;
    if (slot >= P.n_slots) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.err, kErrSlotRange);
        return;
    }
    float4* st = reinterpret_cast<float4*>(P.state) + (size_t)slot * state16_per_slot;
    float4* wn = reinterpret_cast<float4*>(P.window) + (size_t)slot * window16_per_slot;
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t stride = (size_t)gridDim.x * kThreads;
    for (size_t j = (size_t)blockIdx.x * kThreads + threadIdx.x; j < state16_per_slot; j += stride) st[j] = z;
    for (size_t j = (size_t)blockIdx.x * kThreads + threadIdx.x; j < window16_per_slot; j += stride) wn[j] = z;
    // an empty verify ring (its records need no clearing)
    if (P.ring_len > 0 && blockIdx.x == 0)
        for (int l = threadIdx.x; l < P.n_layers; l += kThreads) P.ring_cnt[(int64_t)slot * P.n_layers + l] = 0;
}

// Workgroup `block` of `blocks` copies its share of the state tiles, conv windows
// and verify rings of every layer of slot src to slot dst (a state "saved and
// copied whole": "Project: adding the hybrid model Qwen3.5", prefix-cache notes).
__device__ __forceinline__ void copy_slot(const PoolView& P, int src, int dst, unsigned block, unsigned blocks,
                                          size_t state16_per_slot, size_t window16_per_slot) {
    const float4* ss = reinterpret_cast<const float4*>(P.state) + (size_t)src * state16_per_slot;
    float4* sd = reinterpret_cast<float4*>(P.state) + (size_t)dst * state16_per_slot;
    const float4* ws = reinterpret_cast<const float4*>(P.window) + (size_t)src * window16_per_slot;
    float4* wd = reinterpret_cast<float4*>(P.window) + (size_t)dst * window16_per_slot;
    const size_t stride = (size_t)blocks * kThreads, first = (size_t)block * kThreads + threadIdx.x;
    for (size_t j = first; j < state16_per_slot; j += stride) sd[j] = ss[j];
    for (size_t j = first; j < window16_per_slot; j += stride) wd[j] = ws[j];
    if (P.ring_len > 0) {   // the verify ring: counts and records of every layer
        const size_t ring16 = (size_t)P.n_layers * P.ring_stride / 4;
        const float4* rs = reinterpret_cast<const float4*>(P.ring) + (size_t)src * ring16;
        float4* rd = reinterpret_cast<float4*>(P.ring) + (size_t)dst * ring16;
        for (size_t j = first; j < ring16; j += stride) rd[j] = rs[j];
        if (block == 0)
            for (int l = threadIdx.x; l < P.n_layers; l += kThreads)
                P.ring_cnt[(int64_t)dst * P.n_layers + l] = P.ring_cnt[(int64_t)src * P.n_layers + l];
    }
}

// Slot src_ids[i] to slot dst_ids[i].  grid = (blocks per slot, n).
__global__ __launch_bounds__(kThreads) void slot_copy_kernel(PoolView P, const int32_t* src_ids,
                                                            const int32_t* dst_ids,
                                                            size_t state16_per_slot,
                                                            size_t window16_per_slot) {
    const int src = src_ids[blockIdx.y], dst = dst_ids[blockIdx.y];
    if (src < 0 || dst < 0) return;
    if (src >= P.n_slots || dst >= P.n_slots) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.err, kErrSlotRange);
        return;
    }
    copy_slot(P, src, dst, blockIdx.x, gridDim.x, state16_per_slot, window16_per_slot);
}

// Beams after a selection.  A parent's first child keeps its slot, every other
// beam takes, in order, the slot of a beam without children: what is copied is a
// beam's second, third .. child, and no source is a destination.  Lane j of each
// wave holds beam j, so a beam's place in either order is a ballot.
struct Beams {
    int slot, from;   // this lane's beam: the slot it gets, the slot copied into it (-1: none)
    bool range;       // a slot of the copy is not in the pool
};

__device__ __forceinline__ Beams place_beams(const int32_t* slots, const int32_t* parents, int width, int n_slots) {
    const int lane = threadIdx.x & 63;
    const int slot = lane < width ? slots[lane] : -1;
    int parent = lane < width ? parents[lane] : -1;
    if (parent >= width) parent = -1;
    const uint64_t before = ((uint64_t)1 << lane) - 1;
    // beams that some beam continues, and beams that are not the first to continue theirs
    uint64_t continued = 0, later = 0;
    for (int j = 0; j < width; ++j) {
        const int p = __builtin_amdgcn_readlane(parent, j);
        const uint64_t bit = p < 0 ? 0 : (uint64_t)1 << p;
        if (p < 0 || (continued & bit)) later |= (uint64_t)1 << j;
        continued |= bit;
    }
    const uint64_t all = width == 64 ? ~(uint64_t)0 : ((uint64_t)1 << width) - 1;
    // the lane that holds the k-th childless beam, for this lane's place k among the later ones
    const uint64_t childless = all & ~continued;
    const int k = __popcll(later & before);
    uint64_t rest = childless;
    int spare = 0;
    for (int j = 0, n = 0; rest; ++n, rest &= rest - 1) {
        j = __builtin_ctzll(rest);
        if (n == k) spare = j;
    }
    const bool moves = lane < width && (later >> lane & 1);
    const int source = __shfl(slot, parent < 0 ? 0 : parent), target = __shfl(slot, spare);
    Beams b;
    b.slot = moves ? target : source;
    b.from = moves && parent >= 0 && source >= 0 && target >= 0 ? source : -1;
    b.range = b.from >= 0 && (source >= n_slots || target >= n_slots);
    if (b.range) b.from = -1;
    return b;
}

// grid = (blocks per slot, beams).  Every workgroup places its request's beams itself,
// from two loads.  16 x 8 beams that copy 824 MB in all: 147 us (5.6 TB/s), one beam
// of 8.6 MB 3.9 us, a launch being 1.9.
__global__ __launch_bounds__(kThreads) void slot_reorder_kernel(PoolView P, int width, const int32_t* slots,
                                                               const int32_t* parents, int32_t* slots_out,
                                                               size_t state16_per_slot, size_t window16_per_slot) {
    const int req = blockIdx.y / width, beam = blockIdx.y % width;
    const Beams b = place_beams(slots + (int64_t)req * width, parents + (int64_t)req * width, width, P.n_slots);
    const int dst = __builtin_amdgcn_readlane(b.slot, beam), src = __builtin_amdgcn_readlane(b.from, beam);
    if (slots_out && blockIdx.x == 0 && threadIdx.x == 0) slots_out[blockIdx.y] = dst;
    if (__builtin_amdgcn_readlane((int)b.range, beam) && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(P.err, kErrSlotRange);
    if (src >= 0) copy_slot(P, src, dst, blockIdx.x, gridDim.x, state16_per_slot, window16_per_slot);
}

// The table alone, one wave per request, in place (2 us beside the copies).
__global__ __launch_bounds__(64) void slot_table_kernel(int width, int32_t* slots, const int32_t* parents) {
    int32_t* mine = slots + (int64_t)blockIdx.x * width;
    const Beams b = place_beams(mine, parents + (int64_t)blockIdx.x * width, width, 0);
    if ((int)threadIdx.x < width) mine[threadIdx.x] = b.slot;
}

}  // namespace

hipError_t launch_slot_copy(const gdn_pool* pool, int32_t n, const int32_t* src_ids,
                            const int32_t* dst_ids, hipStream_t stream) {
    const PoolView& P = pool->view;
    const size_t state16 = (size_t)P.n_layers * P.h_v * P.d * P.d / 4;
    const size_t win16 = (size_t)P.n_layers * (P.conv_k - 1) * P.c_conv * pool->io_size / 16;
    size_t blocks = (state16 + kThreads * 4 - 1) / (kThreads * 4);
    blocks = blocks < 1 ? 1 : (blocks > 256 ? 256 : blocks);
    hipLaunchKernelGGL(slot_copy_kernel, dim3((unsigned)blocks, n), dim3(kThreads), 0, stream, P,
                       src_ids, dst_ids, state16, win16);
    return hipGetLastError();
}

hipError_t launch_slot_reorder(const gdn_pool* pool, int32_t n_req, int32_t width, const int32_t* slots,
                               const int32_t* parents, int32_t* slots_out, hipStream_t stream) {
    const PoolView& P = pool->view;
    const size_t state16 = (size_t)P.n_layers * P.h_v * P.d * P.d / 4;
    const size_t win16 = (size_t)P.n_layers * (P.conv_k - 1) * P.c_conv * pool->io_size / 16;
    size_t blocks = (state16 + kThreads * 4 - 1) / (kThreads * 4);
    blocks = blocks < 1 ? 1 : (blocks > 256 ? 256 : blocks);
    // In place the table is written behind the copies, which all read it.
    const bool in_place = slots_out == slots;
    hipLaunchKernelGGL(slot_reorder_kernel, dim3((unsigned)blocks, n_req * width), dim3(kThreads), 0, stream, P,
                       width, slots, parents, in_place ? nullptr : slots_out, state16, win16);
    if (in_place)
        hipLaunchKernelGGL(slot_table_kernel, dim3(n_req), dim3(64), 0, stream, width, slots_out, parents);
    return hipGetLastError();
}

hipError_t launch_fill_zero(void* ptr, size_t bytes, hipStream_t stream) {
    const size_t n16 = bytes / 16;  // callers pass multiples of 16 bytes
    if (n16 == 0) return hipSuccess;
    size_t blocks = (n16 + kThreads - 1) / kThreads;
    blocks = blocks > 4096 ? 4096 : blocks;
    hipLaunchKernelGGL(fill_zero_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream,
                       static_cast<float4*>(ptr), n16);
    return hipGetLastError();
}

hipError_t launch_slot_reset(const gdn_pool* pool, int32_t n, const int32_t* slot_ids,
                             hipStream_t stream) {
    const PoolView& P = pool->view;
    const size_t state16 = (size_t)P.n_layers * P.h_v * P.d * P.d / 4;
    const size_t win_bytes = (size_t)P.n_layers * (P.conv_k - 1) * P.c_conv * pool->io_size;
    const size_t win16 = win_bytes / 16;  // c_conv is a multiple of 32, so this is exact
    size_t blocks = (state16 + kThreads * 4 - 1) / (kThreads * 4);
    blocks = blocks < 1 ? 1 : (blocks > 256 ? 256 : blocks);
    hipLaunchKernelGGL(slot_reset_kernel, dim3((unsigned)blocks, n), dim3(kThreads), 0, stream, P,
                       slot_ids, state16, win16);
    return hipGetLastError();
}

}  // namespace gdn
