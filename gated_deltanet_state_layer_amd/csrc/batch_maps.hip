// The maps of a batch from its requests' lengths: starts of the requests, maps
// from tokens to requests, positions and adapters, and the checkpoint table.
//
// A few KB of work: what it costs is the launch and a chain of memory trips, so it
// is one launch without scratch memory.  Every workgroup scans the lengths itself
// (4096 at a time in LDS) and then fills its own rows; no workgroup waits for
// another.
#include <algorithm>

#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kPer = 8, kChunk = kThreads * kPer;   // requests per thread and per scan
constexpr int kRows = 4, kTile = kThreads * kRows;  // rows per thread and per step

struct Maps {
    const int32_t *lens, *past, *adapter_ids, *free_slots;
    int32_t *cu, *last_rows, *token_seq, *token_pos, *token_adapter, *ckpt_offsets, *ckpt_slots, *err;
    int32_t n_seq, n_adapters, ckpt_every, n_free, max_ckpt;
    uint32_t max_tok;
    int vec;   // the per-token arrays that are given are 16-byte aligned
};

// Exclusive sum over the workgroup, saturating at cap (below 2^31: sums of two fit).
// Adding and cutting off commute as nothing is negative.  total: the whole sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t cap, uint32_t* waves, uint32_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(s, d);
        if (lane >= d) s = min(s + o, cap);
    }
    if (lane == 63) waves[wave] = s;
    __syncthreads();
    uint32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) base = all;
        all = min(all + waves[w], cap);
    }
    __syncthreads();   // waves[] is free again
    *total = all;
    const uint32_t before = __shfl_up(s, 1);
    return lane ? min(base + before, cap) : base;
}

__device__ __forceinline__ void put4(int32_t* p, int64_t r, const int (&v)[kRows], uint32_t in, bool vec) {
    if (!p) return;
    if (vec && in == 15u) {
        *reinterpret_cast<int4*>(p + r) = make_int4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (in >> i & 1) p[r + i] = v[i];
}

__global__ __launch_bounds__(kThreads) void batch_maps_kernel(Maps a) {
    __shared__ uint32_t cu[kChunk + 1], waves[kWaves];
    const int tid = threadIdx.x;
    const uint32_t cap = a.max_tok + 1;
    const bool tokens = a.token_seq || a.token_pos || a.token_adapter;
    uint32_t carry = 0, ck_carry = 0;
    int bad = 0;
    for (int c0 = 0; c0 < a.n_seq; c0 += kChunk) {
        const int here = min(kChunk, a.n_seq - c0);
        const bool writer = (unsigned)(c0 / kChunk) % gridDim.x == blockIdx.x;
        uint32_t len[kPer], sum = 0, total;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int j = tid * kPer + k;
            const int l = j < here ? a.lens[c0 + j] : 0;
            if (l < 0) bad |= kErrSeqlens;
            len[k] = min((uint32_t)max(l, 0), cap);
            sum = min(sum + len[k], cap);
        }
        uint32_t at = min(carry + block_scan(sum, cap, waves, &total), cap);
        uint32_t end[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            cu[tid * kPer + k] = min(at, a.max_tok);
            at = min(at + len[k], cap);
            end[k] = min(at, a.max_tok);
        }
        carry = min(carry + total, cap);
        if (tid == 0) cu[kChunk] = min(carry, a.max_tok);
        if (a.ckpt_every > 0) {
            const uint32_t most = (uint32_t)a.max_ckpt, every = (uint32_t)a.ckpt_every;
            uint32_t n[kPer], rows = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                n[k] = (end[k] - cu[tid * kPer + k]) / every;
                rows = min(rows + n[k], most);
            }
            uint32_t off = min(ck_carry + block_scan(rows, most, waves, &total), most);
            ck_carry = min(ck_carry + total, most);
            if (writer)
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    if (tid * kPer + k < here) a.ckpt_offsets[c0 + tid * kPer + k] = (int32_t)off;
                    off = min(off + n[k], most);
                }
        }
        __syncthreads();
        if (writer)
            for (int j = tid; j < here; j += kThreads) {
                const uint32_t s = cu[j], e = cu[j + 1];
                a.cu[c0 + j] = (int32_t)s;
                if (a.last_rows) a.last_rows[c0 + j] = e > s ? (int32_t)e - 1 : -1;
                if (a.adapter_ids && a.adapter_ids[c0 + j] >= a.n_adapters) bad |= kErrAdapter;
            }
        if (tokens) {
            const uint32_t lo = cu[0], hi = cu[kChunk];
            for (uint64_t t0 = (uint64_t)blockIdx.x * kTile; t0 < hi; t0 += (uint64_t)gridDim.x * kTile) {
                if (t0 + kTile <= lo) continue;
                const uint64_t r = t0 + (uint64_t)tid * kRows;
                if (r >= hi || r + kRows <= lo) continue;
                const uint32_t first = (uint32_t)max(r, (uint64_t)lo);
                int j = 0;   // the last request that starts at or before the first row
#pragma unroll
                for (int step = kChunk / 2; step > 0; step /= 2)
                    if (cu[j + step] <= first) j += step;
                int seq[kRows], pos[kRows], ad[kRows];
                uint32_t in = 0;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const uint64_t t = r + i;
                    seq[i] = pos[i] = ad[i] = -1;
                    if (t < lo || t >= hi) continue;
                    in |= 1u << i;
                    while (cu[j + 1] <= (uint32_t)t) ++j;   // ends: t < cu[kChunk]
                    seq[i] = c0 + j;
                    if (a.token_pos) pos[i] = (a.past ? a.past[c0 + j] : 0) + (int)((uint32_t)t - cu[j]);
                    if (a.token_adapter) {
                        const int id = a.adapter_ids[c0 + j];
                        ad[i] = id < 0 || id >= a.n_adapters ? -1 : id;
                    }
                }
                put4(a.token_seq, (int64_t)r, seq, in, a.vec);
                put4(a.token_pos, (int64_t)r, pos, in, a.vec);
                put4(a.token_adapter, (int64_t)r, ad, in, a.vec);
            }
        }
        __syncthreads();   // cu[] is read out
    }
    if (carry > a.max_tok) bad |= kErrSeqlens;
    const uint32_t total = min(carry, a.max_tok);
    if (blockIdx.x == 0 && tid == 0) {
        a.cu[a.n_seq] = (int32_t)total;
        if (a.ckpt_every > 0) a.ckpt_offsets[a.n_seq] = (int32_t)ck_carry;
    }
    if (bad) atomicOr(a.err, bad);
    if (tokens)
        for (uint64_t t0 = (uint64_t)blockIdx.x * kTile; t0 < a.max_tok; t0 += (uint64_t)gridDim.x * kTile) {
            if (t0 + kTile <= total) continue;
            const uint64_t r = t0 + (uint64_t)tid * kRows;
            uint32_t in = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) in |= (uint32_t)(r + i >= total && r + i < a.max_tok) << i;
            const int none[kRows] = {-1, -1, -1, -1};
            put4(a.token_seq, (int64_t)r, none, in, a.vec);
            put4(a.token_pos, (int64_t)r, none, in, a.vec);
            put4(a.token_adapter, (int64_t)r, none, in, a.vec);
        }
    if (a.ckpt_every > 0) {
        const uint32_t have = min(ck_carry, (uint32_t)a.n_free);
        for (uint32_t i = blockIdx.x * kThreads + tid; i < (uint32_t)a.max_ckpt; i += gridDim.x * kThreads)
            a.ckpt_slots[i] = i < have ? a.free_slots[i] : -1;
    }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

hipError_t launch_batch_maps(const gdn_pool* pool, int32_t n_seq, const int32_t* lens, int64_t max_tok,
                             int32_t* cu_seqlens, int32_t* last_rows, int32_t* token_seq, const int32_t* past,
                             int32_t* token_pos, const int32_t* adapter_ids, int32_t n_adapters,
                             int32_t* token_adapter, int32_t ckpt_every, const int32_t* free_slots,
                             int32_t n_free, int32_t* ckpt_offsets, int32_t* ckpt_slots, int32_t max_ckpt,
                             hipStream_t stream) {
    Maps a{};
    a.lens = lens;
    a.past = past;
    a.adapter_ids = adapter_ids;
    a.free_slots = free_slots;
    a.cu = cu_seqlens;
    a.last_rows = last_rows;
    a.token_seq = token_seq;
    a.token_pos = token_pos;
    a.token_adapter = token_adapter;
    a.ckpt_offsets = ckpt_offsets;
    a.ckpt_slots = ckpt_slots;
    a.err = pool->view.err;
    a.n_seq = n_seq;
    a.n_adapters = n_adapters;
    a.ckpt_every = ckpt_every;
    a.n_free = n_free;
    a.max_ckpt = max_ckpt;
    a.max_tok = (uint32_t)max_tok;
    a.vec = aligned16(token_seq) && aligned16(token_pos) && aligned16(token_adapter);
    const bool tokens = token_seq || token_pos || token_adapter;
    const int64_t tiles = tokens ? (max_tok + kTile - 1) / kTile : 0;
    const int64_t ckpt = ckpt_every > 0 ? ((int64_t)max_ckpt + kThreads - 1) / kThreads : 0;
    const int64_t grid = std::min<int64_t>(1024, std::max<int64_t>(1, std::max(tiles, ckpt)));
    hipLaunchKernelGGL(batch_maps_kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
