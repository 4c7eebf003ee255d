// The maps of a batch from its requests' lengths: starts of the requests, maps
// from tokens to requests, positions and adapters, and the checkpoint table.
//
// A few KB of work: what it costs is the launch (1.9 us) and a chain of memory
// trips, so it is one launch without scratch memory.  Every workgroup loads what the
// requests bring, all loads in one trip, scans the lengths itself (512 to 4096 at a
// time, in LDS) and then fills its own rows; no workgroup waits for another.  All
// maps of 64 requests 4.2 us (5.3 with the loads one behind the other and scans
// through LDS), of 2000 requests with 300001 tokens and checkpoints 6.8 (3.7 MB).
#include <algorithm>

#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kRows = 4, kTile = kThreads * kRows;  // rows per thread and per step

struct Maps {
    const int32_t *lens, *past, *adapter_ids, *free_slots;
    int32_t *cu, *last_rows, *token_seq, *token_pos, *token_adapter, *ckpt_offsets, *ckpt_slots, *err;
    int32_t n_seq, n_adapters, ckpt_every, n_free, max_ckpt;
    uint32_t max_tok;
    int vec;   // the per-token arrays that are given are 16-byte aligned
};

// a + b, cut off at cap < 2^31.  Adding and cutting off commute as nothing is negative.
__device__ __forceinline__ uint32_t add_to(uint32_t a, uint32_t b, uint32_t cap) { return min(a + b, cap); }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {   // 0 where there is none
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}

// Inclusive sum over the wave: shifts inside rows of 16 lanes, then the last lanes of
// the rows before.
__device__ __forceinline__ uint32_t wave_scan(uint32_t s, uint32_t cap) {
    s = add_to(s, from_lane<0x111, 0xF>(s), cap);   // row_shr 1, 2, 4, 8
    s = add_to(s, from_lane<0x112, 0xF>(s), cap);
    s = add_to(s, from_lane<0x114, 0xF>(s), cap);
    s = add_to(s, from_lane<0x118, 0xF>(s), cap);
    s = add_to(s, from_lane<0x142, 0xA>(s), cap);   // lane 15 of the row before
    s = add_to(s, from_lane<0x143, 0xC>(s), cap);   // lane 31
    return s;
}

struct Scan {
    uint32_t before, total;   // of this thread's part, and in all
};

// After wave_scan and a barrier behind the waves' totals.
__device__ __forceinline__ Scan block_scan(uint32_t inclusive, uint32_t cap, const uint32_t (&waves)[kWaves]) {
    const int wave = threadIdx.x >> 6;
    Scan r{0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) r.before = r.total;
        r.total = add_to(r.total, waves[w], cap);
    }
    const uint32_t own = from_lane<0x138, 0xF>(inclusive);   // wave_shr 1
    r.before = add_to(r.before, own, cap);
    return r;
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

// PER requests to a thread: as few as hold them all, since what the threads scan and
// put into LDS grows with it (64 requests 4.2 us, eight to a thread 5.6; 2000 requests
// four to a thread 6.8, eight 8.1).
template <int PER>
__global__ __launch_bounds__(kThreads) void batch_maps_kernel(Maps a) {
    constexpr int kChunk = kThreads * PER;
    __shared__ uint32_t cu[kChunk + 1], waves[kWaves], ck_waves[kWaves];
    __shared__ int32_t past[kChunk], adapter[kChunk];
    const int tid = threadIdx.x;
    const uint32_t cap = a.max_tok + 1, most = (uint32_t)a.max_ckpt;
    const bool tokens = a.token_seq || a.token_pos || a.token_adapter;
    uint32_t carry = 0, ck_carry = 0;
    int bad = 0;
    // this thread's first checkpoint row, in case it is one
    const uint32_t row0 = blockIdx.x * kThreads + tid;
    const int32_t slot0 = a.ckpt_every > 0 && row0 < min((uint32_t)a.n_free, most) ? a.free_slots[row0] : -1;
    // the last chunk may end at 2^31: what is left is counted down beside its start
    uint32_t c0 = 0;
    for (int left = a.n_seq; left > 0; left -= kChunk, c0 += kChunk) {
        const int here = min(kChunk, left);
        const bool writer = c0 / kChunk % gridDim.x == blockIdx.x;
        int32_t raw[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {   // neighbouring requests in neighbouring lanes
            const int j = k * kThreads + tid;
            raw[k] = j < here ? a.lens[c0 + j] : 0;
            if (a.token_pos) past[j] = a.past && j < here ? a.past[c0 + j] : 0;
            if (a.adapter_ids) {
                const int id = j < here ? a.adapter_ids[c0 + j] : -1;
                if (id >= a.n_adapters) bad |= kErrAdapter;
                adapter[j] = id < 0 || id >= a.n_adapters ? -1 : id;
            }
        }
        if constexpr (PER > 1) {   // PER consecutive requests to a thread from here on
#pragma unroll
            for (int k = 0; k < PER; ++k) cu[k * kThreads + tid] = (uint32_t)raw[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < PER; ++k) raw[k] = (int32_t)cu[tid * PER + k];
        }
        uint32_t len[PER], n[PER], sum = 0, rows = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (raw[k] < 0) bad |= kErrSeqlens;
            len[k] = min((uint32_t)max(raw[k], 0), cap);
            sum = add_to(sum, len[k], cap);
            n[k] = a.ckpt_every > 0 ? len[k] / (uint32_t)a.ckpt_every : 0;
            rows = add_to(rows, n[k], most);
        }
        sum = wave_scan(sum, cap);
        rows = wave_scan(rows, most);
        if ((tid & 63) == 63) {
            waves[tid >> 6] = sum;
            ck_waves[tid >> 6] = rows;
        }
        __syncthreads();
        const Scan s = block_scan(sum, cap, waves);
        Scan ck = block_scan(rows, most, ck_waves);
        uint32_t at = add_to(carry, s.before, cap);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t begin = min(at, a.max_tok);
            cu[tid * PER + k] = begin;
            at = add_to(at, len[k], cap);
            len[k] = min(at, a.max_tok) - begin;   // what there is room for
        }
        carry = add_to(carry, s.total, cap);
        if (tid == 0) cu[kChunk] = min(carry, a.max_tok);
        if (a.ckpt_every > 0) {
            if (carry > a.max_tok) {   // the checkpoints of what there is room for
                rows = 0;
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    n[k] = len[k] / (uint32_t)a.ckpt_every;
                    rows = add_to(rows, n[k], most);
                }
                rows = wave_scan(rows, most);
                __syncthreads();
                if ((tid & 63) == 63) ck_waves[tid >> 6] = rows;
                __syncthreads();
                ck = block_scan(rows, most, ck_waves);
            }
            uint32_t off = add_to(ck_carry, ck.before, most);
            ck_carry = add_to(ck_carry, ck.total, most);
            if (writer)
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    if (tid * PER + k < here) a.ckpt_offsets[c0 + tid * PER + k] = (int32_t)off;
                    off = add_to(off, n[k], most);
                }
        }
        __syncthreads();
        if (writer)
            for (int j = tid; j < here; j += kThreads) {
                const uint32_t s0 = cu[j], e0 = cu[j + 1];
                a.cu[c0 + j] = (int32_t)s0;
                if (a.last_rows) a.last_rows[c0 + j] = e0 > s0 ? (int32_t)e0 - 1 : -1;
            }
        if (tokens) {
            const uint32_t lo = cu[0], hi = cu[kChunk];
            for (uint64_t t0 = (uint64_t)blockIdx.x * kTile; t0 < hi; t0 += (uint64_t)gridDim.x * kTile) {
                if (t0 + kTile <= lo) continue;
                const uint64_t r = t0 + (uint64_t)tid * kRows;
                if (r >= hi || r + kRows <= lo) continue;
                const uint32_t first = (uint32_t)max(r, (uint64_t)lo);
                int j = 0;   // the last request that starts at or before the first row
                for (int step = 1 << (31 - __builtin_clz(here)); step > 0; step /= 2)
                    if (j + step < here && cu[j + step] <= first) j += step;
                int seq[kRows], pos[kRows], ad[kRows];
                uint32_t in = 0;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const uint64_t t = r + i;
                    seq[i] = pos[i] = ad[i] = -1;
                    if (t < lo || t >= hi) continue;
                    in |= 1u << i;
                    while (cu[j + 1] <= (uint32_t)t) ++j;   // ends: t < cu[kChunk]
                    seq[i] = (int)c0 + j;
                    if (a.token_pos) pos[i] = past[j] + (int)((uint32_t)t - cu[j]);
                    if (a.token_adapter) ad[i] = adapter[j];
                }
                put4(a.token_seq, (int64_t)r, seq, in, a.vec);
                put4(a.token_pos, (int64_t)r, pos, in, a.vec);
                put4(a.token_adapter, (int64_t)r, ad, in, a.vec);
            }
        }
        if (left > kChunk) __syncthreads();   // cu[] is read out
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
        for (uint32_t i = row0; i < most; i += gridDim.x * kThreads)
            a.ckpt_slots[i] = i >= have ? -1 : i == row0 ? slot0 : a.free_slots[i];
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
    if (n_seq <= kThreads)
        hipLaunchKernelGGL(batch_maps_kernel<1>, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
    else if (n_seq <= 4 * kThreads)
        hipLaunchKernelGGL(batch_maps_kernel<4>, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(batch_maps_kernel<8>, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
