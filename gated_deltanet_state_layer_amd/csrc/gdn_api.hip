// libgdn host API: descriptor checks, the slot pool, argument validation and
// dispatch to the kernels.  Every check runs before anything is enqueued, so
// a negative status leaves device memory untouched.
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "gdn_common.h"
#include "mx_plan.h"

namespace gdn {
size_t decode_verify_lds_bytes(const gdn_pool* pool, int32_t n_tok);

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kMaxLds = 64 * 1024;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

gdn_status check_desc(const gdn_pool_desc* d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->n_slots < 1 || d->n_layers < 1 || d->h_k < 1 || d->h_v < 1 || d->d_k < 1 ||
        d->d_v < 1 || d->conv_k < 1)
        return GDN_ERR_INVALID_ARG;
    if (d->h_v % d->h_k != 0) return GDN_ERR_INVALID_ARG;
    if (d->io_dtype != GDN_F32 && d->io_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (!(d->q_scale >= 0.f) || !(d->norm_eps >= 0.f) || std::isinf(d->q_scale) ||
        std::isinf(d->norm_eps))
        return GDN_ERR_INVALID_ARG;
    if (d->flags & ~(GDN_VALIDATE | GDN_GROUP_KERNEL)) return GDN_ERR_INVALID_ARG;
    if (d->ring_len < 0) return GDN_ERR_INVALID_ARG;
    if (d->ring_len > kMaxRingSolve - kMaxVerifyTokens) return GDN_ERR_UNSUPPORTED;
    if (d->d_k != d->d_v) return GDN_ERR_UNSUPPORTED;
    if (d->d_k != 32 && d->d_k != 64 && d->d_k != 128) return GDN_ERR_UNSUPPORTED;
    if (d->conv_k < 2 || d->conv_k > kMaxConvK) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Byte offsets inside the aux buffer (the layout documented in gdn.h).
struct AuxLayout {
    size_t window_bytes, meta, ctr, ring_cnt, ring_arr, ring, total;
    int64_t ring_stride;   // floats per (slot, layer) ring block
};

AuxLayout aux_layout(const gdn_pool_desc* d) {
    AuxLayout x{};
    const size_t io = d->io_dtype == GDN_BF16 ? 2 : 4;
    const size_t c_conv = 2 * (size_t)d->h_k * d->d_k + (size_t)d->h_v * d->d_v;
    const size_t sl = (size_t)d->n_slots * d->n_layers;
    x.window_bytes = sl * (d->conv_k - 1) * c_conv * io;
    // windows | meta block (error word) | row-split decode counters | ring
    x.meta = align_up(x.window_bytes, kAlign);
    x.ctr = x.meta + kAlign;
    x.total = x.ctr + align_up(sl * d->h_k * sizeof(int32_t), kAlign);
    if (d->ring_len > 0) {
        const size_t per_tok = (size_t)d->h_k * d->d_k + (size_t)d->h_v * d->d_v + 2 * (size_t)d->h_v;
        x.ring_stride = (int64_t)align_up(d->ring_len * per_tok, 64);
        x.ring_cnt = x.total;
        x.ring_arr = x.ring_cnt + align_up(sl * sizeof(int32_t), kAlign);
        x.ring = x.ring_arr + align_up(sl * sizeof(int32_t), kAlign);
        x.total = x.ring + sl * x.ring_stride * sizeof(float);
    }
    return x;
}

void layout(const gdn_pool_desc* d, size_t* state_bytes, size_t* window_bytes, size_t* aux_bytes) {
    *state_bytes = (size_t)d->n_slots * d->n_layers * d->h_v * d->d_v * d->d_k * sizeof(float);
    const AuxLayout x = aux_layout(d);
    *window_bytes = x.window_bytes;
    *aux_bytes = x.total;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Host-side C++ failures (a host array that cannot be allocated in
// GDN_VALIDATE mode) never cross the C ABI: they become GDN_ERR_HOST, and
// nothing has been enqueued by then.
template <typename F>
gdn_status guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return GDN_ERR_HOST;
    }
}

// GDN_VALIDATE: copy a device index array to the host and check it.
gdn_status host_check_ids(const int32_t* ids, int32_t n, int32_t n_slots, hipStream_t s) {
    std::vector<int32_t> h(n);
    if (n == 0) return GDN_OK;
    if (hipMemcpyAsync(h.data(), ids, n * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess)
        return GDN_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return GDN_ERR_HIP;
    std::vector<int32_t> seen;
    for (int32_t x : h) {
        if (x >= n_slots) return GDN_ERR_BAD_INDEX;
        if (x >= 0) seen.push_back(x);
    }
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return GDN_ERR_BAD_INDEX;
    return GDN_OK;
}

gdn_status host_check_seqlens(const int32_t* cu, int32_t n_seq, int64_t total, hipStream_t s) {
    std::vector<int32_t> h(n_seq + 1);
    if (hipMemcpyAsync(h.data(), cu, (n_seq + 1) * sizeof(int32_t), hipMemcpyDeviceToHost, s) !=
        hipSuccess)
        return GDN_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return GDN_ERR_HIP;
    if (h[0] != 0 || h[n_seq] != total) return GDN_ERR_BAD_INDEX;
    for (int j = 0; j < n_seq; ++j)
        if (h[j + 1] < h[j]) return GDN_ERR_BAD_INDEX;
    return GDN_OK;
}

// Host check of the checkpoint lists (GDN_VALIDATE): offsets from 0,
// non-decreasing; every sequence and checkpoint slot in range and distinct.
// The row count is bounded before anything is sized from it: no sequence can
// use more than len_j / ckpt_every rows, so more than
// total_tokens / ckpt_every + n_seq rows in all is rejected.
gdn_status host_check_ckpt(const int32_t* slot_ids, int32_t n_seq, const int32_t* off,
                           const int32_t* slots, int32_t n_slots, int64_t total_tokens,
                           int32_t ckpt_every, hipStream_t s) {
    std::vector<int32_t> ho(n_seq + 1), hs(n_seq);
    if (hipMemcpyAsync(ho.data(), off, (n_seq + 1) * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipMemcpyAsync(hs.data(), slot_ids, n_seq * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
        return GDN_ERR_HIP;
    if (ho[0] != 0) return GDN_ERR_BAD_INDEX;
    for (int j = 0; j < n_seq; ++j)
        if (ho[j + 1] < ho[j]) return GDN_ERR_BAD_INDEX;
    if ((int64_t)ho[n_seq] > total_tokens / ckpt_every + n_seq) return GDN_ERR_BAD_INDEX;
    std::vector<int32_t> hc(ho[n_seq]);
    if (!hc.empty() &&
        (hipMemcpyAsync(hc.data(), slots, hc.size() * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
         hipStreamSynchronize(s) != hipSuccess))
        return GDN_ERR_HIP;
    std::vector<int32_t> seen;
    for (int32_t x : hs) if (x >= 0) seen.push_back(x);
    for (int32_t x : hc) if (x >= 0) seen.push_back(x);
    for (int32_t x : seen) if (x >= n_slots) return GDN_ERR_BAD_INDEX;
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return GDN_ERR_BAD_INDEX;
    return GDN_OK;
}

// GDN_VALIDATE for the one-call path on a ring pool: every listed slot's ring
// for `layer` must be empty (the call reads and writes the state tile).
gdn_status host_check_rings_empty(const gdn_pool* pool, int32_t layer, const int32_t* ids,
                                  int32_t n, hipStream_t s) {
    if (pool->desc.ring_len == 0 || n == 0) return GDN_OK;
    const size_t sl = (size_t)pool->desc.n_slots * pool->desc.n_layers;
    std::vector<int32_t> h(n), cnt(sl);
    if (hipMemcpyAsync(h.data(), ids, n * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipMemcpyAsync(cnt.data(), pool->view.ring_cnt, sl * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
        return GDN_ERR_HIP;
    for (int32_t x : h)
        if (x >= 0 && x < pool->desc.n_slots && cnt[(size_t)x * pool->desc.n_layers + layer] != 0)
            return GDN_ERR_RING;
    return GDN_OK;
}

gdn_status prefill_common(gdn_pool* pool, int32_t layer, int32_t n_seq, const int32_t* cu_seqlens,
                          const int32_t* slot_ids, int64_t total_tokens, int32_t chunk,
                          const void* q, const void* k, const void* v, const float* a,
                          const float* b, const float* conv_w, void* out, int32_t ckpt_every,
                          const int32_t* ckpt_offsets, const int32_t* ckpt_slots, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (!pool || layer < 0 || layer >= pool->desc.n_layers || n_seq < 0 || total_tokens < 0)
        return GDN_ERR_INVALID_ARG;
    if (chunk != 16 && chunk != 32 && chunk != 64) return GDN_ERR_UNSUPPORTED;
    if (total_tokens > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if (ckpt_every < 0 || ckpt_every % chunk != 0) return GDN_ERR_INVALID_ARG;
    if (n_seq == 0) return GDN_OK;
    if (!cu_seqlens || !slot_ids || !conv_w) return GDN_ERR_INVALID_ARG;
    if (ckpt_every > 0 && (!ckpt_offsets || !ckpt_slots)) return GDN_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !a || !b || !out)) return GDN_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16)))
        return GDN_ERR_INVALID_ARG;
    const size_t need = prefill_workspace_bytes(pool, n_seq, total_tokens, chunk);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GDN_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    hipStream_t s = as_stream(stream);
    if (pool->desc.flags & GDN_VALIDATE) {
        gdn_status st = ckpt_every > 0
                            ? host_check_ckpt(slot_ids, n_seq, ckpt_offsets, ckpt_slots,
                                              pool->desc.n_slots, total_tokens, ckpt_every, s)
                            : host_check_ids(slot_ids, n_seq, pool->desc.n_slots, s);
        if (st != GDN_OK) return st;
        st = host_check_seqlens(cu_seqlens, n_seq, total_tokens, s);
        if (st != GDN_OK) return st;
        st = host_check_rings_empty(pool, layer, slot_ids, n_seq, s);
        if (st == GDN_OK && ckpt_every > 0) {
            int32_t n_ck = 0;
            if (hipMemcpyAsync(&n_ck, ckpt_offsets + n_seq, sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
                hipStreamSynchronize(s) != hipSuccess)
                return GDN_ERR_HIP;
            st = host_check_rings_empty(pool, layer, ckpt_slots, n_ck, s);
        }
        if (st != GDN_OK) return st;
    }
    const Ckpt ck{ckpt_every / chunk, ckpt_offsets, ckpt_slots};
    hipError_t e = launch_prefill(pool, layer, n_seq, cu_seqlens, slot_ids, total_tokens, chunk, q,
                                  k, v, a, b, conv_w, out, workspace, ck, s);
    if (e == hipErrorNotSupported) return GDN_ERR_UNSUPPORTED;
    return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_pool_bytes(const gdn_pool_desc* desc, size_t* state_bytes, size_t* aux_bytes) {
    gdn_status st = check_desc(desc);
    if (st != GDN_OK) return st;
    if (!state_bytes || !aux_bytes) return GDN_ERR_INVALID_ARG;
    size_t wb;
    layout(desc, state_bytes, &wb, aux_bytes);
    return GDN_OK;
}

gdn_status gdn_pool_create(const gdn_pool_desc* desc, void* state_buf, void* aux_buf, void* stream,
                           gdn_pool** out) {
    gdn_status st = check_desc(desc);
    if (st != GDN_OK) return st;
    if (!state_buf || !aux_buf || !out) return GDN_ERR_INVALID_ARG;
    if (!aligned(state_buf, kAlign) || !aligned(aux_buf, kAlign)) return GDN_ERR_INVALID_ARG;
    gdn_pool* p = new (std::nothrow) gdn_pool();
    if (!p) return GDN_ERR_INVALID_ARG;
    p->desc = *desc;
    if (p->desc.q_scale == 0.f) p->desc.q_scale = 1.0f / std::sqrt((float)desc->d_k);
    if (p->desc.norm_eps == 0.f) p->desc.norm_eps = 1e-6f;
    layout(desc, &p->state_bytes, &p->window_bytes, &p->aux_bytes);
    p->io_size = desc->io_dtype == GDN_BF16 ? 2 : 4;
    PoolView& v = p->view;
    v.state = static_cast<float*>(state_buf);
    v.window = aux_buf;
    const AuxLayout ax = aux_layout(desc);
    char* aux = static_cast<char*>(aux_buf);
    v.err = reinterpret_cast<int32_t*>(aux + ax.meta);
    v.ctr = reinterpret_cast<int32_t*>(aux + ax.ctr);
    v.ring_len = desc->ring_len;
    v.ring_cnt = desc->ring_len > 0 ? reinterpret_cast<int32_t*>(aux + ax.ring_cnt) : nullptr;
    v.ring_arr = desc->ring_len > 0 ? reinterpret_cast<int32_t*>(aux + ax.ring_arr) : nullptr;
    v.ring = desc->ring_len > 0 ? reinterpret_cast<float*>(aux + ax.ring) : nullptr;
    v.ring_stride = ax.ring_stride;
    v.n_slots = desc->n_slots;
    v.n_layers = desc->n_layers;
    v.h_k = desc->h_k;
    v.h_v = desc->h_v;
    v.d = desc->d_k;
    v.conv_k = desc->conv_k;
    v.c_conv = 2 * desc->h_k * desc->d_k + desc->h_v * desc->d_v;
    v.q_scale = p->desc.q_scale;
    v.eps = p->desc.norm_eps;
    hipStream_t s = as_stream(stream);
    if (launch_fill_zero(state_buf, p->state_bytes, s) != hipSuccess ||
        launch_fill_zero(aux_buf, p->aux_bytes, s) != hipSuccess) {
        delete p;
        return GDN_ERR_HIP;
    }
    *out = p;
    return GDN_OK;
}

gdn_status gdn_pool_destroy(gdn_pool* pool) {
    if (!pool) return GDN_ERR_INVALID_ARG;
    delete pool;
    return GDN_OK;
}

gdn_status gdn_slot_reset(gdn_pool* pool, int32_t n, const int32_t* slot_ids, void* stream) {
    return guarded([&]() -> gdn_status {
        if (!pool || n < 0 || (n > 0 && !slot_ids)) return GDN_ERR_INVALID_ARG;
        if (n == 0) return GDN_OK;
        if (n > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y limit
        hipStream_t s = as_stream(stream);
        if (pool->desc.flags & GDN_VALIDATE) {
            gdn_status st = host_check_ids(slot_ids, n, pool->desc.n_slots, s);
            if (st != GDN_OK) return st;
        }
        return launch_slot_reset(pool, n, slot_ids, s) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
}

static gdn_status check_step_args(gdn_pool* pool, int32_t layer, int32_t n, const int32_t* slot_ids,
                                  int32_t n_tok, const void* q, const void* k, const void* v,
                                  const float* a, const float* b, const float* conv_w,
                                  const void* out, bool out_optional = false) {
    if (!pool) return GDN_ERR_INVALID_ARG;
    if (layer < 0 || layer >= pool->desc.n_layers || n < 0) return GDN_ERR_INVALID_ARG;
    if (n_tok < 1 || n_tok > kMaxVerifyTokens) return GDN_ERR_INVALID_ARG;
    if (n > 0 && (!slot_ids || !q || !k || !v || !a || !b || !conv_w || (!out && !out_optional)))
        return GDN_ERR_INVALID_ARG;
    if (n > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y limit
    if (n > 0 && out && !aligned(out, 16)) return GDN_ERR_INVALID_ARG;  // 16-byte output vectors
    if (decode_verify_lds_bytes(pool, n_tok) > kMaxLds) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status gdn_decode_step(gdn_pool* pool, int32_t layer, int32_t n, const int32_t* slot_ids,
                           const void* q, const void* k, const void* v, const float* a,
                           const float* b, const float* conv_w, void* out, void* stream) {
    return guarded([&]() -> gdn_status {
        gdn_status st = check_step_args(pool, layer, n, slot_ids, 1, q, k, v, a, b, conv_w, out);
        if (st != GDN_OK || n == 0) return st;
        hipStream_t s = as_stream(stream);
        if (pool->desc.flags & GDN_VALIDATE) {
            st = host_check_ids(slot_ids, n, pool->desc.n_slots, s);
            if (st == GDN_OK) st = host_check_rings_empty(pool, layer, slot_ids, n, s);
            if (st != GDN_OK) return st;
        }
        // Few entries: split each head's rows over several workgroups so that
        // more CUs stream the state (same arithmetic, bitwise equal results).
        // Otherwise one value head per workgroup (d_k 64 or 128), else the
        // one-workgroup-per-group kernel.  All three are bitwise equal.
        const bool group = pool->desc.flags & GDN_GROUP_KERNEL;
        const int nrb = group ? 1 : decode_rows_split(pool, n);
        const hipError_t e =
            nrb > 1 ? launch_decode_rows(pool, nrb, layer, n, slot_ids, q, k, v, a, b, conv_w, out, s)
            : !group && decode_heads_ok(pool)
                ? launch_decode_heads(pool, layer, n, slot_ids, 1, q, k, v, a, b, conv_w, nullptr,
                                      out, s)
                : launch_decode_verify(pool, layer, n, slot_ids, 1, q, k, v, a, b, conv_w, nullptr,
                                       out, s);
        return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
}

gdn_status gdn_verify_step(gdn_pool* pool, int32_t layer, int32_t n, const int32_t* slot_ids,
                           int32_t n_tok, const void* q, const void* k, const void* v,
                           const float* a, const float* b, const float* conv_w,
                           const int32_t* accept_len, void* out, void* stream) {
    return guarded([&]() -> gdn_status {
        gdn_status st = check_step_args(pool, layer, n, slot_ids, n_tok, q, k, v, a, b, conv_w, out, true);
        if (st != GDN_OK) return st;
        if (n > 0 && !accept_len) return GDN_ERR_INVALID_ARG;
        if (n == 0) return GDN_OK;
        hipStream_t s = as_stream(stream);
        if (pool->desc.flags & GDN_VALIDATE) {
            st = host_check_ids(slot_ids, n, pool->desc.n_slots, s);
            if (st == GDN_OK) st = host_check_rings_empty(pool, layer, slot_ids, n, s);
            if (st != GDN_OK) return st;
        }
        // One value head per workgroup where it applies (d_k 64 or 128),
        // else one workgroup per q/k group; bitwise equal.
        const hipError_t e =
            !(pool->desc.flags & GDN_GROUP_KERNEL) && decode_heads_ok(pool)
                ? launch_decode_heads(pool, layer, n, slot_ids, n_tok, q, k, v, a, b, conv_w,
                                      accept_len, out, s)
                : launch_decode_verify(pool, layer, n, slot_ids, n_tok, q, k, v, a, b, conv_w,
                                       accept_len, out, s);
        return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
}

gdn_status gdn_prefill_workspace_bytes(const gdn_pool* pool, int32_t n_seq, int64_t total_tokens,
                                       int32_t chunk, size_t* bytes) {
    if (!pool || !bytes || n_seq < 0 || total_tokens < 0) return GDN_ERR_INVALID_ARG;
    if (chunk != 16 && chunk != 32 && chunk != 64) return GDN_ERR_UNSUPPORTED;
    *bytes = prefill_workspace_bytes(pool, n_seq, total_tokens, chunk);
    return GDN_OK;
}

gdn_status gdn_prefill_chunked(gdn_pool* pool, int32_t layer, int32_t n_seq,
                               const int32_t* cu_seqlens, const int32_t* slot_ids,
                               int64_t total_tokens, int32_t chunk, const void* q, const void* k,
                               const void* v, const float* a, const float* b, const float* conv_w,
                               void* out, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> gdn_status {
        return prefill_common(pool, layer, n_seq, cu_seqlens, slot_ids, total_tokens, chunk, q, k, v,
                              a, b, conv_w, out, 0, nullptr, nullptr, workspace, workspace_bytes,
                              stream);
    });
}

gdn_status gdn_prefill_chunked_static(gdn_pool* pool, int32_t layer, int32_t n_seq,
                                      const int32_t* cu_seqlens, const int32_t* slot_ids,
                                      int64_t total_tokens, int32_t chunk, const void* q,
                                      const void* k, const void* v, const float* a,
                                      const float* b, const float* conv_w, void* out,
                                      void* stream) {
    return guarded([&]() -> gdn_status {
        if (!pool || n_seq < 0 || total_tokens < 0) return GDN_ERR_INVALID_ARG;
        if (chunk != 16 && chunk != 32 && chunk != 64) return GDN_ERR_UNSUPPORTED;
        if (prefill_workspace_bytes(pool, n_seq, total_tokens, chunk) > kStaticScratchBytes)
            return GDN_ERR_WORKSPACE;
        void* ws = nullptr;
        if (prefill_static_scratch(&ws) != hipSuccess) return GDN_ERR_HIP;
        return prefill_common(pool, layer, n_seq, cu_seqlens, slot_ids, total_tokens, chunk, q, k,
                              v, a, b, conv_w, out, 0, nullptr, nullptr, ws, kStaticScratchBytes,
                              stream);
    });
}

gdn_status gdn_prefill_chunked_ckpt(gdn_pool* pool, int32_t layer, int32_t n_seq,
                                    const int32_t* cu_seqlens, const int32_t* slot_ids,
                                    int64_t total_tokens, int32_t chunk, const void* q,
                                    const void* k, const void* v, const float* a, const float* b,
                                    const float* conv_w, void* out, int32_t ckpt_every,
                                    const int32_t* ckpt_offsets, const int32_t* ckpt_slots,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> gdn_status {
        return prefill_common(pool, layer, n_seq, cu_seqlens, slot_ids, total_tokens, chunk, q, k, v,
                              a, b, conv_w, out, ckpt_every, ckpt_offsets, ckpt_slots, workspace,
                              workspace_bytes, stream);
    });
}

gdn_status gdn_slot_copy(gdn_pool* pool, int32_t n, const int32_t* src_ids,
                         const int32_t* dst_ids, void* stream) {
    return guarded([&]() -> gdn_status {
        if (!pool || n < 0 || (n > 0 && (!src_ids || !dst_ids))) return GDN_ERR_INVALID_ARG;
        if (n == 0) return GDN_OK;
        if (n > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y limit
        hipStream_t s = as_stream(stream);
        if (pool->desc.flags & GDN_VALIDATE) {
            // sources in range; destinations in range, distinct and not sources
            std::vector<int32_t> hs(n), hd(n);
            if (hipMemcpyAsync(hs.data(), src_ids, n * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
                hipMemcpyAsync(hd.data(), dst_ids, n * sizeof(int32_t), hipMemcpyDeviceToHost, s) != hipSuccess ||
                hipStreamSynchronize(s) != hipSuccess)
                return GDN_ERR_HIP;
            std::vector<int32_t> dst;
            for (int i = 0; i < n; ++i) {
                if (hs[i] >= pool->desc.n_slots || hd[i] >= pool->desc.n_slots) return GDN_ERR_BAD_INDEX;
                if (hs[i] >= 0 && hd[i] >= 0) dst.push_back(hd[i]);
            }
            std::sort(dst.begin(), dst.end());
            if (std::adjacent_find(dst.begin(), dst.end()) != dst.end()) return GDN_ERR_BAD_INDEX;
            for (int i = 0; i < n; ++i)
                if (hs[i] >= 0 && hd[i] >= 0 && std::binary_search(dst.begin(), dst.end(), hs[i]))
                    return GDN_ERR_BAD_INDEX;
        }
        return launch_slot_copy(pool, n, src_ids, dst_ids, s) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
}

gdn_status gdn_slot_reorder(gdn_pool* pool, int32_t n_req, int32_t width, const int32_t* slots,
                            const int32_t* parents, int32_t* slots_out, void* stream) {
    return guarded([&]() -> gdn_status {
        if (!pool || n_req < 0 || width < 1) return GDN_ERR_INVALID_ARG;
        if (n_req > 0 && (!slots || !parents || !slots_out)) return GDN_ERR_INVALID_ARG;
        if (width > GDN_BEAM_MAX || (int64_t)n_req * width > 65535) return GDN_ERR_UNSUPPORTED;  // grid.y limit
        if (n_req == 0) return GDN_OK;
        hipStream_t s = as_stream(stream);
        if (pool->desc.flags & GDN_VALIDATE) {
            const gdn_status st = host_check_ids(slots, n_req * width, pool->desc.n_slots, s);
            if (st != GDN_OK) return st;
        }
        return launch_slot_reorder(pool, n_req, width, slots, parents, slots_out, s) == hipSuccess ? GDN_OK
                                                                                                  : GDN_ERR_HIP;
    });
}

static gdn_status beam_args(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out) {
    if (n_req < 0 || width < 1 || vocab < 1 || n_out < 1) return GDN_ERR_INVALID_ARG;
    if (width > GDN_BEAM_MAX || n_out > GDN_BEAM_MAX || vocab > 1 << 30 || (int64_t)n_req * width > 1 << 20)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status gdn_beam_select_workspace_bytes(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out,
                                           size_t* bytes) {
    const gdn_status st = beam_args(n_req, width, vocab, n_out);
    if (st != GDN_OK) return st;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    *bytes = beam_select_workspace_bytes(n_req, width, vocab, n_out);
    return GDN_OK;
}

gdn_status gdn_beam_select(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out, gdn_dtype dtype,
                           const void* logits, int64_t ld, const float* scores, const uint8_t* finished,
                           int32_t eos, int32_t* parents, int32_t* tokens, float* scores_out,
                           uint8_t* finished_out, void* workspace, size_t workspace_bytes, void* stream) {
    const gdn_status st = beam_args(n_req, width, vocab, n_out);
    if (st != GDN_OK) return st;
    if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (finished && eos < 0) return GDN_ERR_INVALID_ARG;
    if (n_req == 0) return GDN_OK;
    if (!logits || !scores || !parents || !tokens || !scores_out) return GDN_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == GDN_BF16 ? 2 : 4) || !aligned(scores, 4) || !aligned(parents, 4) ||
        !aligned(tokens, 4) || !aligned(scores_out, 4))
        return GDN_ERR_INVALID_ARG;
    if (n_req * width > 1 && ld < vocab) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < beam_select_workspace_bytes(n_req, width, vocab, n_out) || !workspace)
        return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    return launch_beam_select(n_req, width, vocab, n_out, dtype, logits, ld, scores, finished, eos, parents,
                              tokens, scores_out, finished_out, workspace, as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

gdn_status gdn_batch_maps(gdn_pool* pool, int32_t n_seq, const int32_t* lens, int64_t max_tok,
                          int32_t* cu_seqlens, int32_t* last_rows, int32_t* token_seq, const int32_t* past,
                          int32_t* token_pos, const int32_t* adapter_ids, int32_t n_adapters,
                          int32_t* token_adapter, int32_t ckpt_every, const int32_t* free_slots,
                          int32_t n_free, int32_t* ckpt_offsets, int32_t* ckpt_slots, int32_t max_ckpt,
                          void* stream) {
    if (!pool || n_seq < 0 || max_tok < 0 || ckpt_every < 0 || !cu_seqlens) return GDN_ERR_INVALID_ARG;
    if (n_seq > 0 && !lens) return GDN_ERR_INVALID_ARG;
    if ((adapter_ids && n_adapters < 0) || (token_adapter && !adapter_ids && n_seq > 0)) return GDN_ERR_INVALID_ARG;
    if (ckpt_every > 0 && (n_free < 0 || max_ckpt < 0 || !ckpt_offsets || (n_free > 0 && !free_slots) ||
                           (max_ckpt > 0 && !ckpt_slots)))
        return GDN_ERR_INVALID_ARG;
    // sums of two counts that are cut off one past the limit stay in 32 bits
    if (max_tok > INT32_MAX - 1) return GDN_ERR_UNSUPPORTED;
    for (const void* p : {(const void*)lens, (const void*)cu_seqlens, (const void*)last_rows, (const void*)token_seq,
                          (const void*)past, (const void*)token_pos, (const void*)adapter_ids,
                          (const void*)token_adapter, (const void*)free_slots, (const void*)ckpt_offsets,
                          (const void*)ckpt_slots})
        if (!aligned(p, 4)) return GDN_ERR_INVALID_ARG;
    return launch_batch_maps(pool, n_seq, lens, max_tok, cu_seqlens, last_rows, token_seq, past, token_pos,
                             adapter_ids, n_adapters, token_adapter, ckpt_every, free_slots, n_free, ckpt_offsets,
                             ckpt_slots, max_ckpt, as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

static gdn_status ring_call(gdn_pool* pool, RingOp op, int32_t layer, int32_t n,
                            const int32_t* slot_ids, int32_t n_tok, const void* q, const void* k,
                            const void* v, const float* a, const float* b, const float* conv_w,
                            const int32_t* accept_len, void* out, void* stream) {
    return guarded([&]() -> gdn_status {
        if (!pool || layer < 0 || layer >= pool->desc.n_layers || n < 0) return GDN_ERR_INVALID_ARG;
        if (pool->desc.ring_len == 0) return GDN_ERR_UNSUPPORTED;
        if (op != RingOp::kFlush) {
            if (n_tok < 1 || n_tok > kMaxVerifyTokens) return GDN_ERR_INVALID_ARG;
            if (pool->desc.ring_len + n_tok > kMaxRingSolve) return GDN_ERR_UNSUPPORTED;
            if (n > 0 && (!q || !k || !v || !a || !b || !conv_w)) return GDN_ERR_INVALID_ARG;
            if (n > 0 && op == RingOp::kVerify && !out) return GDN_ERR_INVALID_ARG;
            if (n > 0 && op == RingOp::kCommit && !accept_len) return GDN_ERR_INVALID_ARG;
        }
        if (n > 0 && !slot_ids) return GDN_ERR_INVALID_ARG;
        if (n == 0) return GDN_OK;
        hipStream_t s = as_stream(stream);
        if (pool->desc.flags & GDN_VALIDATE) {
            const gdn_status st = host_check_ids(slot_ids, n, pool->desc.n_slots, s);
            if (st != GDN_OK) return st;
        }
        const hipError_t e = launch_ring(pool, op, layer, n, slot_ids, op == RingOp::kFlush ? 0 : n_tok,
                                         q, k, v, a, b, conv_w, accept_len, out, s);
        if (e == hipErrorNotSupported) return GDN_ERR_UNSUPPORTED;
        return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    });
}

gdn_status gdn_ring_verify(gdn_pool* pool, int32_t layer, int32_t n, const int32_t* slot_ids,
                           int32_t n_tok, const void* q, const void* k, const void* v,
                           const float* a, const float* b, const float* conv_w, void* out,
                           void* stream) {
    return ring_call(pool, RingOp::kVerify, layer, n, slot_ids, n_tok, q, k, v, a, b, conv_w,
                     nullptr, out, stream);
}

gdn_status gdn_ring_commit(gdn_pool* pool, int32_t layer, int32_t n, const int32_t* slot_ids,
                           int32_t n_tok, const void* q, const void* k, const void* v,
                           const float* a, const float* b, const float* conv_w,
                           const int32_t* accept_len, void* stream) {
    return ring_call(pool, RingOp::kCommit, layer, n, slot_ids, n_tok, q, k, v, a, b, conv_w,
                     accept_len, nullptr, stream);
}

gdn_status gdn_ring_flush(gdn_pool* pool, int32_t layer, int32_t n, const int32_t* slot_ids,
                          void* stream) {
    return ring_call(pool, RingOp::kFlush, layer, n, slot_ids, 0, nullptr, nullptr, nullptr,
                     nullptr, nullptr, nullptr, nullptr, nullptr, stream);
}

static gdn_status in_proj_args(const gdn_pool* pool, int64_t n_tok, int32_t hidden) {
    if (!pool || n_tok < 0 || hidden < 1) return GDN_ERR_INVALID_ARG;
    if (hidden % 32 != 0) return GDN_ERR_UNSUPPORTED;
    const int64_t n_out = pool->view.c_conv + 2 * pool->view.h_v;
    // 32-bit byte offsets inside x and W (128 rows of slack for ragged tiles)
    if ((n_tok + 128) * hidden * 2 >= INT32_MAX || (n_out + 128) * hidden * 2 >= INT32_MAX)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status gdn_in_proj_workspace_bytes(const gdn_pool* pool, int64_t n_tok, int32_t hidden,
                                       size_t* bytes) {
    const gdn_status st = in_proj_args(pool, n_tok, hidden);
    if (st != GDN_OK) return st;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    *bytes = in_proj_workspace_bytes(pool, n_tok, hidden);
    return GDN_OK;
}

gdn_status gdn_in_proj(gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x, const void* w,
                       void* q, void* k, void* v, float* a, float* b, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const gdn_status st = in_proj_args(pool, n_tok, hidden);
    if (st != GDN_OK) return st;
    if (n_tok == 0) return GDN_OK;
    if (!x || !w || !q || !k || !v || !a || !b) return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16)) return GDN_ERR_INVALID_ARG;
    const size_t need = in_proj_workspace_bytes(pool, n_tok, hidden);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GDN_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
    return launch_in_proj(pool, n_tok, hidden, x, w, q, k, v, a, b, workspace,
                          as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

static bool dtype_ok(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
static size_t elem_bytes(gdn_dtype t) { return t == GDN_BF16 ? 2 : 4; }

gdn_status gdn_block_norm(int64_t n_tok, int32_t hidden, gdn_dtype io_dtype, gdn_dtype res_dtype,
                          const void* y, int64_t ld_y, const float* w_post, float res_scale,
                          const void* res, int64_t ld_res, void* res_out, int64_t ld_res_out,
                          const float* w_pre, float w_offset, float eps, void* x, int64_t ld_x,
                          void* stream) {
    if (n_tok < 0 || hidden < 1 || !dtype_ok(io_dtype) || !dtype_ok(res_dtype)) return GDN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(res_scale) || !std::isfinite(w_offset))
        return GDN_ERR_INVALID_ARG;
    if (hidden > GDN_BLOCK_NORM_MAX_HIDDEN) return GDN_ERR_UNSUPPORTED;
    if (n_tok == 0) return GDN_OK;
    if (!res || !w_pre || !x) return GDN_ERR_INVALID_ARG;
    if (y ? !res_out : (res_out || w_post)) return GDN_ERR_INVALID_ARG;
    if (n_tok > 1 && (ld_res < hidden || ld_x < hidden || (y && (ld_y < hidden || ld_res_out < hidden))))
        return GDN_ERR_INVALID_ARG;
    const size_t io = elem_bytes(io_dtype), rs = elem_bytes(res_dtype);
    if (!aligned(y, io) || !aligned(x, io) || !aligned(res, rs) || !aligned(res_out, rs) ||
        !aligned(w_pre, 4) || !aligned(w_post, 4))
        return GDN_ERR_INVALID_ARG;
    return launch_block_norm(n_tok, hidden, io_dtype, res_dtype, y, ld_y, w_post, res_scale, res, ld_res,
                             res_out, ld_res_out, w_pre, w_offset, eps, x, ld_x,
                             as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

gdn_status gdn_gated_norm(const gdn_pool* pool, int64_t n_tok, const void* o, int64_t ld_o, const void* z,
                          int64_t ld_z, const float* w, float eps, gdn_dtype out_dtype, void* out,
                          int64_t ld_out, void* stream) {
    if (!pool || n_tok < 0 || !dtype_ok(out_dtype) || !(eps >= 0.f) || !std::isfinite(eps))
        return GDN_ERR_INVALID_ARG;
    if (n_tok == 0) return GDN_OK;
    if (!o || !z || !w || !out) return GDN_ERR_INVALID_ARG;
    if (!aligned(o, 16) || !aligned(z, 16) || !aligned(w, 16) || !aligned(out, 16)) return GDN_ERR_INVALID_ARG;
    const int64_t width = (int64_t)pool->view.h_v * pool->view.d;
    if (n_tok > 1)
        for (const int64_t ld : {ld_o, ld_z, ld_out})
            if (ld < width || ld % 8 != 0) return GDN_ERR_INVALID_ARG;
    return launch_gated_norm(pool, n_tok, o, ld_o, z, ld_z, w, eps, out_dtype, out, ld_out,
                             as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

static gdn_status mx_format_args(int64_t rows, int32_t cols, gdn_dtype dtype) {
    if (rows < 0 || cols < 1 || !dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
    if (cols % GDN_MX_GROUP != 0) return GDN_ERR_UNSUPPORTED;
    return rows > INT64_MAX / cols / 4 ? GDN_ERR_INVALID_ARG : GDN_OK;
}

gdn_status gdn_mx_quantize(int64_t rows, int32_t cols, gdn_dtype dtype, const void* src, void* codes,
                           uint8_t* scales, void* stream) {
    const gdn_status st = mx_format_args(rows, cols, dtype);
    if (st != GDN_OK) return st;
    if (rows == 0) return GDN_OK;
    if (!src || !codes || !scales || !aligned(src, 16) || !aligned(codes, 16)) return GDN_ERR_INVALID_ARG;
    return launch_mx_quantize(rows, cols, dtype, src, codes, scales, as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

gdn_status gdn_mx_dequantize(int64_t rows, int32_t cols, const void* codes, const uint8_t* scales,
                             gdn_dtype dtype, void* dst, void* stream) {
    const gdn_status st = mx_format_args(rows, cols, dtype);
    if (st != GDN_OK) return st;
    if (rows == 0) return GDN_OK;
    if (!dst || !codes || !scales || !aligned(dst, 16) || !aligned(codes, 16)) return GDN_ERR_INVALID_ARG;
    return launch_mx_dequantize(rows, cols, dtype, codes, scales, dst, as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

static gdn_status mx_proj_args(int64_t n_tok, int32_t n_in, int64_t n_out) {
    if (n_tok < 0 || n_in < 1 || n_out < 1) return GDN_ERR_INVALID_ARG;
    if (n_in % GDN_MX_GROUP != 0 || n_in > GDN_MX_MAX_IN || n_out > INT32_MAX - 256 ||
        !mx_proj_fits(n_tok, n_out))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Output channels of the in-projection of a pool's layer.
static int64_t mx_in_proj_channels(const gdn_pool* pool, bool with_z) {
    const PoolView& P = pool->view;
    return (int64_t)P.c_conv + (with_z ? (int64_t)P.h_v * P.d : 0) + 2 * (int64_t)P.h_v;
}

// No size needs scratch memory; one that is given has to be aligned all the same.
static gdn_status mx_workspace_ok(const void* workspace) {
    return workspace && !aligned(workspace, kAlign) ? GDN_ERR_INVALID_ARG : GDN_OK;
}

gdn_status gdn_mx_proj_workspace_bytes(int64_t n_tok, int32_t n_in, int32_t n_out, size_t* bytes) {
    const gdn_status st = mx_proj_args(n_tok, n_in, n_out);
    if (st != GDN_OK) return st;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    *bytes = 0;
    return GDN_OK;
}

// The checks that both forms of a projection make; a single row's strides are set.
static gdn_status mx_proj_operands(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t* ld_x,
                                   const void* codes, const uint8_t* scales, gdn_dtype y_dtype, const void* y,
                                   int64_t* ld_y) {
    if (!x || !codes || !scales || !y) return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(y, elem_bytes(y_dtype))) return GDN_ERR_INVALID_ARG;
    if (n_tok == 1) {   // a single row has no stride
        *ld_x = n_in;
        *ld_y = n_out;
    }
    if (*ld_x < n_in || *ld_x % 8 != 0 || *ld_y < n_out) return GDN_ERR_INVALID_ARG;
    return *ld_x > 2 * GDN_MX_MAX_IN ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn_status gdn_mx_proj(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t ld_x,
                       const void* codes, const uint8_t* scales, gdn_dtype y_dtype, void* y, int64_t ld_y,
                       void* workspace, size_t /*workspace_bytes*/, void* stream) {
    gdn_status st = mx_proj_args(n_tok, n_in, n_out);
    if (st != GDN_OK) return st;
    if (!dtype_ok(y_dtype)) return GDN_ERR_INVALID_ARG;
    if (n_tok == 0) return GDN_OK;
    st = mx_proj_operands(n_tok, n_in, n_out, x, &ld_x, codes, scales, y_dtype, y, &ld_y);
    if (st != GDN_OK) return st;
    st = mx_workspace_ok(workspace);
    if (st != GDN_OK) return st;
    return launch_mx_proj(n_tok, n_in, n_out, x, ld_x, codes, scales, y_dtype, y, ld_y, as_stream(stream)) ==
                   hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

gdn_status gdn_mx_in_proj_workspace_bytes(const gdn_pool* pool, int64_t n_tok, int32_t hidden,
                                          int32_t with_z, size_t* bytes) {
    if (!pool) return GDN_ERR_INVALID_ARG;
    const int64_t n_out = mx_in_proj_channels(pool, with_z != 0);
    const gdn_status st = mx_proj_args(n_tok, hidden, n_out);
    if (st != GDN_OK) return st;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    *bytes = 0;
    return GDN_OK;
}

static gdn_status mx_in_proj_operands(const gdn_pool* pool, const void* x, const void* codes, const uint8_t* scales,
                                      const void* q, const void* k, const void* v, const void* z, const float* a,
                                      const float* b) {
    if (!x || !codes || !scales || !q || !k || !v || !a || !b) return GDN_ERR_INVALID_ARG;
    const size_t io = (size_t)pool->io_size;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(q, io) || !aligned(k, io) || !aligned(v, io) ||
        !aligned(z, io) || !aligned(a, 4) || !aligned(b, 4))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn_status gdn_mx_in_proj(const gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x,
                          const void* codes, const uint8_t* scales, void* q, void* k, void* v, void* z,
                          float* a, float* b, void* workspace, size_t /*workspace_bytes*/, void* stream) {
    if (!pool) return GDN_ERR_INVALID_ARG;
    const int64_t n_out = mx_in_proj_channels(pool, z != nullptr);
    gdn_status st = mx_proj_args(n_tok, hidden, n_out);
    if (st != GDN_OK) return st;
    if (n_tok == 0) return GDN_OK;
    st = mx_in_proj_operands(pool, x, codes, scales, q, k, v, z, a, b);
    if (st != GDN_OK) return st;
    st = mx_workspace_ok(workspace);
    if (st != GDN_OK) return st;
    return launch_mx_in_proj(pool, n_tok, hidden, x, codes, scales, q, k, v, z, a, b, as_stream(stream)) ==
                   hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

static gdn_status lora_rank_ok(int32_t rank) {
    if (rank < 1) return GDN_ERR_INVALID_ARG;
    return rank % 8 != 0 || rank > GDN_LORA_MAX_RANK ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

static gdn_status lora_operands(int64_t n_tok, const LoraArgs& l, const void* workspace, size_t workspace_bytes) {
    if (!l.a || !l.b || !l.scale || !l.ids) return GDN_ERR_INVALID_ARG;
    if (!aligned(l.a, 16) || !aligned(l.b, 16) || !aligned(l.scale, 4) || !aligned(l.ids, 4)) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < lora_workspace_bytes(n_tok, l.rank) || !workspace) return GDN_ERR_WORKSPACE;
    return aligned(workspace, kAlign) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

gdn_status gdn_mx_proj_lora_workspace_bytes(int64_t n_tok, int32_t n_in, int32_t n_out, int32_t rank,
                                            size_t* bytes) {
    gdn_status st = mx_proj_args(n_tok, n_in, n_out);
    if (st == GDN_OK) st = lora_rank_ok(rank);
    if (st != GDN_OK) return st;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    *bytes = lora_workspace_bytes(n_tok, rank);
    return GDN_OK;
}

gdn_status gdn_mx_proj_lora(int64_t n_tok, int32_t n_in, int32_t n_out, const void* x, int64_t ld_x,
                            const void* codes, const uint8_t* scales, int32_t n_adapters, int32_t rank,
                            const void* lora_a, const void* lora_b, const float* lora_scale,
                            const int32_t* token_adapter, gdn_dtype y_dtype, void* y, int64_t ld_y,
                            void* workspace, size_t workspace_bytes, void* stream) {
    if (n_adapters < 0) return GDN_ERR_INVALID_ARG;
    if (n_adapters == 0)
        return gdn_mx_proj(n_tok, n_in, n_out, x, ld_x, codes, scales, y_dtype, y, ld_y, workspace,
                           workspace_bytes, stream);
    gdn_status st = mx_proj_args(n_tok, n_in, n_out);
    if (st == GDN_OK) st = lora_rank_ok(rank);
    if (st != GDN_OK) return st;
    if (!dtype_ok(y_dtype)) return GDN_ERR_INVALID_ARG;
    if (n_tok == 0) return GDN_OK;
    const LoraArgs l{n_adapters, rank, lora_a, lora_b, lora_scale, token_adapter, workspace};
    st = mx_proj_operands(n_tok, n_in, n_out, x, &ld_x, codes, scales, y_dtype, y, &ld_y);
    if (st == GDN_OK) st = lora_operands(n_tok, l, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    return launch_mx_proj_lora(n_tok, n_in, n_out, x, ld_x, codes, scales, l, y_dtype, y, ld_y,
                               as_stream(stream)) == hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

gdn_status gdn_mx_in_proj_lora_workspace_bytes(const gdn_pool* pool, int64_t n_tok, int32_t hidden,
                                               int32_t rank, int32_t with_z, size_t* bytes) {
    if (!pool) return GDN_ERR_INVALID_ARG;
    gdn_status st = mx_proj_args(n_tok, hidden, mx_in_proj_channels(pool, with_z != 0));
    if (st == GDN_OK) st = lora_rank_ok(rank);
    if (st != GDN_OK) return st;
    if (!bytes) return GDN_ERR_INVALID_ARG;
    *bytes = lora_workspace_bytes(n_tok, rank);
    return GDN_OK;
}

gdn_status gdn_mx_in_proj_lora(const gdn_pool* pool, int64_t n_tok, int32_t hidden, const void* x,
                               const void* codes, const uint8_t* scales, int32_t n_adapters, int32_t rank,
                               const void* lora_a, const void* lora_b, const float* lora_scale,
                               const int32_t* token_adapter, void* q, void* k, void* v, void* z, float* a,
                               float* b, void* workspace, size_t workspace_bytes, void* stream) {
    if (!pool || n_adapters < 0) return GDN_ERR_INVALID_ARG;
    if (n_adapters == 0)
        return gdn_mx_in_proj(pool, n_tok, hidden, x, codes, scales, q, k, v, z, a, b, workspace, workspace_bytes,
                              stream);
    gdn_status st = mx_proj_args(n_tok, hidden, mx_in_proj_channels(pool, z != nullptr));
    if (st == GDN_OK) st = lora_rank_ok(rank);
    if (st != GDN_OK) return st;
    if (n_tok == 0) return GDN_OK;
    const LoraArgs l{n_adapters, rank, lora_a, lora_b, lora_scale, token_adapter, workspace};
    st = mx_in_proj_operands(pool, x, codes, scales, q, k, v, z, a, b);
    if (st == GDN_OK) st = lora_operands(n_tok, l, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    return launch_mx_in_proj_lora(pool, n_tok, hidden, x, codes, scales, l, q, k, v, z, a, b, as_stream(stream)) ==
                   hipSuccess
               ? GDN_OK
               : GDN_ERR_HIP;
}

gdn_status gdn_pool_error(gdn_pool* pool, void* stream, int32_t* device_error) {
    if (!pool || !device_error) return GDN_ERR_INVALID_ARG;
    hipStream_t s = as_stream(stream);
    int32_t h = 0;
    if (hipStreamSynchronize(s) != hipSuccess) return GDN_ERR_HIP;
    if (hipMemcpy(&h, pool->view.err, sizeof(int32_t), hipMemcpyDeviceToHost) != hipSuccess)
        return GDN_ERR_HIP;
    if (h != 0) {
        if (launch_fill_zero(pool->view.err, kAlign, s) != hipSuccess) return GDN_ERR_HIP;
        if (hipStreamSynchronize(s) != hipSuccess) return GDN_ERR_HIP;
    }
    *device_error = h;
    return GDN_OK;
}

const char* gdn_status_string(gdn_status status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument";
        case GDN_ERR_UNSUPPORTED: return "unsupported shape or option";
        case GDN_ERR_BAD_INDEX: return "slot id out of range or repeated, or malformed cu_seqlens";
        case GDN_ERR_WORKSPACE: return "workspace too small";
        case GDN_ERR_HIP: return "HIP runtime error";
        case GDN_ERR_RING: return "a listed slot's verify ring is not empty (flush it first)";
        case GDN_ERR_HOST: return "host-side failure (host memory)";
        default: return "unknown status";
    }
}

}  // extern "C"
