// Beam selection: the best n_out continuations of each request's beams over the
// vocabulary, by score + logit - log(sum of exp(logits)).
//
// Within a beam the order is that of the logits alone, so one pass over them finds
// both a beam's best tokens and its sum; a second, small kernel puts the beams of a
// request together.  A wave takes a stretch of a row: it sums exp(x - c), c a
// logit near the largest so far, and holds the best 64 keys, sorted, one to a
// lane, a key being logit and token.  An element is compared with the last key that
// counts; the few that pass go through 64 places of LDS and are then sorted and
// merged into the list.
//
// Scores of different beams may lie closer than 32 bits resolve, and tokens are
// whole numbers, right or wrong.  So exponentials and sums are fp64 here: the vector
// units run them at fp32's rate, and a polynomial of degree 8 on |r| <= ln 2 / 2
// (Chebyshev interpolation, 1.1e-12) keeps sums to about 1e-12.
#include <algorithm>
#include <cfloat>

#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = 8, kStep = 64 * kPer;       // logits per lane and per wave of a step
constexpr int kMaxSplits = 64;                   // a lane per stretch when they are put together
constexpr int kMergeThreads = 512, kMergeWaves = kMergeThreads / 64;
constexpr float kNone = -__builtin_inff();

// exp(d) for -700 <= d <= 700 (below: exp(-700)).
__device__ __forceinline__ double exp64(double d) {
    constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: the sum's low bits are the integer
    d = fmax(d, -700.0);
    const double m = fma(d, 1.4426950408889634, kMagic), n = m - kMagic;
    const double r = fma(n, -0.6931471805599453, d);
    double p = 2.4876070919998397e-05;
    p = fma(p, r, 0.00019915868674658883);
    p = fma(p, r, 0.001388882190450549);
    p = fma(p, r, 0.008333266094398913);
    p = fma(p, r, 0.04166666688931224);
    p = fma(p, r, 0.16666666891065027);
    p = fma(p, r, 0.4999999999980122);
    p = fma(p, r, 0.9999999999797838);
    p = fma(p, r, 1.0000000000000004);
    const uint64_t bits = __builtin_bit_cast(uint64_t, p) + ((uint64_t)(uint32_t)__builtin_bit_cast(uint64_t, m) << 52);
    return __builtin_bit_cast(double, bits);
}

// Order-preserving images of floating-point numbers; never 0 for numbers.
__device__ __forceinline__ uint32_t image(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0 is 0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float image_value(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t image(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | (uint64_t)1 << 63);
}
__device__ __forceinline__ double image_value(uint64_t k) {
    return __builtin_bit_cast(double, k ^ (k >> 63 ? (uint64_t)1 << 63 : ~(uint64_t)0));
}

// A logit and its token: larger logits first, of equal ones the lower token.  0: none.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) {
    return x > kNone ? (uint64_t)image(x) << 32 | (uint32_t)~token : 0;
}

// A continuation: its score's image (0: none), beam * 64 + place in the beam's list.
struct Entry {
    uint64_t score;
    uint32_t tag;
};

__device__ __forceinline__ uint64_t across(uint64_t v, int mask) { return __shfl_xor(v, mask); }
__device__ __forceinline__ Entry across(Entry v, int mask) {
    return {__shfl_xor(v.score, mask), __shfl_xor(v.tag, mask)};
}
__device__ __forceinline__ bool better(uint64_t a, uint64_t b) { return a > b; }
__device__ __forceinline__ bool better(Entry a, Entry b) {
    return a.score > b.score || (a.score == b.score && a.tag < b.tag);
}

// One step of a sorting network: of lanes `mask` apart, the one with `first` keeps
// the better value.
template <typename V>
__device__ __forceinline__ V exchange(V v, int mask, bool first) {
    const V o = across(v, mask);
    return better(o, v) == first ? o : v;
}

// The wave's 64 values, best in lane 0.
template <typename V>
__device__ __forceinline__ V sort64(V v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 2; k <= 64; k *= 2) {
        v = exchange(v, k - 1, !(lane & (k / 2)));
#pragma unroll
        for (int j = k / 4; j > 0; j /= 2) v = exchange(v, j, !(lane & j));
    }
    return v;
}

// The best 64 of two sorted lists, sorted.
template <typename V>
__device__ __forceinline__ V merge64(V a, V b) {
    const int lane = threadIdx.x & 63;
    const V o = across(b, 63);
    V v = better(o, a) ? o : a;
#pragma unroll
    for (int j = 32; j > 0; j /= 2) v = exchange(v, j, !(lane & j));
    return v;
}

__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// A wave's own places of LDS: what its lanes wrote is there for all of them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The best keys of a stream: a sorted list in registers, and those that may join it
// in LDS until there are 64.
struct Best {
    uint64_t list;
    uint64_t* held;   // 128 places of the wave's own
    int n;

    __device__ __forceinline__ void join(int count) {
        const int lane = threadIdx.x & 63;
        wave_sync();
        const uint64_t v = lane < count ? held[lane] : 0;
        list = merge64(list, sort64(v));
        wave_sync();
    }
    // Every lane brings a key; those of `mask` join.
    __device__ __forceinline__ void add(uint64_t key, uint64_t mask) {
        const int lane = threadIdx.x & 63;
        if (mask >> lane & 1) held[n + __popcll(mask & (((uint64_t)1 << lane) - 1))] = key;
        n += __popcll(mask);
        if (n < 64) return;
        join(64);
        const uint64_t rest = lane < n - 64 ? held[64 + lane] : 0;
        wave_sync();
        held[lane] = rest;
        wave_sync();
        n -= 64;
    }
    __device__ __forceinline__ void finish() {
        if (n > 0) join(n);
        n = 0;
    }
};

// Logits i .. i+7 of a row, -infinity behind its end; NaN reads as -infinity and
// +infinity as the largest finite value.  Rows need not be aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int i, int vocab, float (&x)[kPer]) {
    T raw[kPer];
    if (i + kPer <= vocab) {
        __builtin_memcpy(raw, row + i, sizeof raw);
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[k] = Io<T>::load(raw, k);
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[k] = i + k < vocab ? Io<T>::load(row, i + k) : kNone;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[k] = x[k] != x[k] ? kNone : fminf(x[k], FLT_MAX);
}

// What a stretch of a row leaves: the logit c, the sum of exp(x - c), the keys.
struct Stretch {
    double sum;
    float c;
    int pad;
};

struct Shape {
    int rows, width, vocab, n_out, splits, steps;   // steps of 512 logits to a stretch
};

// One wave per stretch of a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void beam_rows_kernel(Shape sh, const T* logits, int64_t ld, const float* scores,
                                                            const uint8_t* finished, Stretch* stats, uint64_t* keys) {
    __shared__ uint64_t held[kWaves][128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t item = (int64_t)blockIdx.x * kWaves + wave;
    if (item >= (int64_t)sh.rows * sh.splits) return;
    const int row = __builtin_amdgcn_readfirstlane((int)(item / sh.splits));
    const int split = __builtin_amdgcn_readfirstlane((int)(item % sh.splits));
    // a beam without continuations, or with one that needs no logits
    if (!(fabsf(scores[row]) <= FLT_MAX) || (finished && finished[row])) return;
    const T* x_row = logits + row * ld;
    const int begin = split * sh.steps * kStep, end = (int)min((int64_t)sh.vocab, (int64_t)begin + sh.steps * kStep);
    float c = -FLT_MAX;
    double sum = 0.0;
    Best best{0, held[wave], 0};
    float least = kNone;   // of the list's last key that counts
    for (int i = begin; i < end; i += kStep) {
        float x[kPer];
        const int at = i + lane * kPer;
        load8(x_row, at, sh.vocab, x);
        float top = x[0];
#pragma unroll
        for (int k = 1; k < kPer; ++k) top = fmaxf(top, x[k]);
        if (__any(top > c + 600.0f)) {   // also the first time
            float t = top;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) t = fmaxf(t, __shfl_xor(t, d));
            sum *= exp64((double)c - (double)t);
            c = t;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) sum += exp64((double)x[k] - (double)c);
        if (i == begin) {
            // the n_out-th of the lanes' best keys: no fewer than n_out reach it
            uint64_t mine = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const uint64_t key = key_of(x[k], at + k);
                mine = key > mine ? key : mine;
            }
            const uint64_t bar = read_lane(sort64(mine), sh.n_out - 1);
#pragma unroll 1
            for (int k = 0; k < kPer; ++k) {
                const uint64_t key = key_of(x[k], at + k);
                best.add(key, __ballot(key && key >= bar));
            }
            best.finish();
        } else if (__any(top > least)) {
            // Later tokens lose against equal logits in the list; within the step
            // the keys decide, so all of it is compared with the list from before.
#pragma unroll 1
            for (int k = 0; k < kPer; ++k) {
                const uint64_t mask = __ballot(x[k] > least);
                if (mask) best.add(key_of(x[k], at + k), mask);
            }
        } else {
            continue;
        }
        const uint32_t last = (uint32_t)(read_lane(best.list, sh.n_out - 1) >> 32);
        least = last ? image_value(last) : kNone;
    }
    best.finish();
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (lane == 0) stats[item] = {sum, c, 0};
    if (lane < sh.n_out) keys[item * sh.n_out + lane] = best.list;
}

// One workgroup per request: each wave puts the stretches of its beams together,
// then one the waves' lists.
__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(Shape sh, const Stretch* stats, const uint64_t* keys,
                                                                  const float* scores, const uint8_t* finished, int eos,
                                                                  int32_t* parents, int32_t* tokens, float* scores_out,
                                                                  uint8_t* finished_out) {
    __shared__ uint64_t held[kMergeWaves][128], l_score[kMergeWaves][64];
    __shared__ uint32_t l_tag[kMergeWaves][64];
    __shared__ int32_t token[GDN_BEAM_MAX * GDN_BEAM_MAX];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t req = blockIdx.x;
    Entry mine{0, ~0u};
    for (int b = wave; b < sh.width; b += kMergeWaves) {
        const int64_t row = req * sh.width + b;
        const float base = scores[row];
        if (!(fabsf(base) <= FLT_MAX)) continue;
        Entry e{0, (uint32_t)(b * 64 + lane)};
        if (finished && finished[row]) {
            if (lane == 0) {
                e.score = image((double)base);
                token[b * 64] = eos;
            }
        } else {
            const Stretch st = lane < sh.splits ? stats[row * sh.splits + lane] : Stretch{0.0, -FLT_MAX, 0};
            float c = st.c;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) c = fmaxf(c, __shfl_xor(c, d));
            double sum = st.sum * exp64((double)st.c - (double)c);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
            // One lane's sum for all: products contracted into the additions leave the
            // lanes' a rounding apart, and equal logits need equal scores.  Apart from c,
            // beside which it would be lost where logits reach 1e38.
            const double norm = log(__builtin_bit_cast(double, read_lane(__builtin_bit_cast(uint64_t, sum), 0)));
            // The lists are sorted: their first keys come first, and few others pass.
            const uint64_t* from = keys + row * sh.splits * sh.n_out;
            Best best{0, held[wave], 0};
            uint64_t bar = 0;
            for (int i = 0; i < sh.splits * sh.n_out; i += 64) {
                const int f = i + lane;
                const uint64_t key =
                    f < sh.splits * sh.n_out ? from[f % sh.splits * sh.n_out + f / sh.splits] : 0;
                const uint64_t mask = __ballot(key > bar);
                if (!mask) break;   // every list has a key here, and none further down is larger
                best.add(key, mask);
                best.finish();
                bar = read_lane(best.list, sh.n_out - 1);
            }
            if (best.list && lane < sh.n_out) {
                e.score = image((double)base +
                                (((double)image_value((uint32_t)(best.list >> 32)) - (double)c) - norm));
                token[b * 64 + lane] = (int32_t)~(uint32_t)best.list;
            }
        }
        mine = merge64(mine, e);
    }
    l_score[wave][lane] = mine.score;
    l_tag[wave][lane] = mine.tag;
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < min(kMergeWaves, sh.width); ++w) mine = merge64(mine, Entry{l_score[w][lane], l_tag[w][lane]});
    if (lane >= sh.n_out) return;
    const int64_t at = req * sh.n_out + lane;
    const bool some = mine.score != 0;
    const int parent = some ? (int)(mine.tag / 64) : -1, tok = some ? token[mine.tag] : -1;
    parents[at] = parent;
    tokens[at] = tok;
    scores_out[at] = some ? (float)image_value(mine.score) : kNone;
    if (finished_out)
        finished_out[at] = some && ((finished && finished[req * sh.width + parent]) || tok == eos);
}

// Stretches: enough waves for the card, at most a lane's worth, none empty.
Shape beam_shape(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out) {
    const int rows = n_req * width, steps = (vocab + kStep - 1) / kStep;
    const int want = std::max(1, std::min({kMaxSplits, steps, 8192 / std::max(1, rows)}));
    const int per = (steps + want - 1) / want;
    return {rows, width, vocab, n_out, (steps + per - 1) / per, per};
}

size_t stats_bytes(const Shape& s) {
    return ((size_t)s.rows * s.splits * sizeof(Stretch) + 255) / 256 * 256;
}

}  // namespace

size_t beam_select_workspace_bytes(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out) {
    const Shape s = beam_shape(n_req, width, vocab, n_out);
    return stats_bytes(s) + (size_t)s.rows * s.splits * n_out * sizeof(uint64_t);
}

hipError_t launch_beam_select(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out, gdn_dtype dtype,
                              const void* logits, int64_t ld, const float* scores, const uint8_t* finished,
                              int32_t eos, int32_t* parents, int32_t* tokens, float* scores_out,
                              uint8_t* finished_out, void* workspace, hipStream_t stream) {
    const Shape s = beam_shape(n_req, width, vocab, n_out);
    Stretch* stats = static_cast<Stretch*>(workspace);
    uint64_t* keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + stats_bytes(s));
    const dim3 grid((unsigned)(((int64_t)s.rows * s.splits + kWaves - 1) / kWaves));
    if (dtype == GDN_BF16)
        hipLaunchKernelGGL(beam_rows_kernel<uint16_t>, grid, dim3(kThreads), 0, stream, s,
                           static_cast<const uint16_t*>(logits), ld, scores, finished, stats, keys);
    else
        hipLaunchKernelGGL(beam_rows_kernel<float>, grid, dim3(kThreads), 0, stream, s,
                           static_cast<const float*>(logits), ld, scores, finished, stats, keys);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(beam_merge_kernel, dim3(n_req), dim3(kMergeThreads), 0, stream, s, stats, keys, scores,
                       finished, eos, parents, tokens, scores_out, finished_out);
    return hipGetLastError();
}

}  // namespace gdn
