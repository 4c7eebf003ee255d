// Beam selection: the best n_out continuations of each request's beams over the
// vocabulary, by score + logit - log(sum of exp(logits)).
//
// Within a beam the order is that of the logits alone, so one pass over them finds
// both a beam's best tokens and its sum; a second, small kernel puts the beams of a
// request together.  A workgroup takes a stretch of a row.  Its waves sum
// exp(x - c), c a logit near the largest so far, and compare each element with the
// last key that counts, a key being logit and token.  The few that pass wait in
// LDS; once there are 64, one wave sorts them, one to a lane, and merges them into
// the sorted list of the best 64.  In the end each sum is divided by the term of the
// stretch's largest logit, made in the same way: a row that is all but certain of a
// token has a sum of 1 and little more, and of 1 exactly with one token left.
//
// Scores of different beams may lie closer than 32 bits resolve, and tokens are
// whole numbers, right or wrong.  So exponentials and sums are fp64 here: the vector
// units run them at fp32's rate.
//
// 64 x 8 x 131072 bf16 (134 MB) take 58 us (2.3 TB/s), 47 without exponentials, 43
// without the selection, about as much when the logits lie in the L2 caches.  No unit
// is busy all the time: the vector units issue in 40 % of the cycles, LDS works in 20 %,
// and waves wait for 61 % of theirs.  What bounds it is latency at four waves to a SIMD,
// as many as 76 KB of LDS a workgroup (half of it the table, half the keys that wait)
// leave room for, with a barrier in each step.  In fp32 (268 MB) 73 us, 3.7 TB/s.
// 1 x 4 x 32000: 9.5 us, of which two launches are 3.8.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "gdn_common.h"

namespace gdn {
namespace {

constexpr int kPer = 8;                          // logits per lane and step
constexpr int kHeld = 64 + 64 * kPer;            // keys of a wave that wait, 63 and a step's
constexpr int kSide = 4;                         // exponentials side by side (1 to 8: the same time)
constexpr int kMaxSplits = 64;                   // a lane per stretch when they are put together
constexpr int kMergeThreads = 1024, kMergeWaves = kMergeThreads / 64;
constexpr int kBatch = 4;                        // loads of 64 keys at a time
constexpr float kNone = -__builtin_inff();

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453;
constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: a sum's low bits are its integer

// exp(r) 2^n of N values side by side, |r| <= ln 2 / 2 or a little more, n in the low
// bits of m.  The polynomial is 1 + r + r^2 q(r), q the Chebyshev interpolation of
// degree 8 (1.2e-15, what fp64 rounds), so that exp(0) is 1.  Degrees 8 and 9 in all
// leave 2e-12 and 7e-14, where scores below 1 are told apart by 2^-41 of themselves.
// The barriers keep the N chains of dependent products interleaved.
template <int N>
__device__ __forceinline__ void exp_scaled(const double (&r)[N], const double (&m)[N], double (&p)[N]) {
    constexpr double kCoef[] = {2.761379764561564e-07, 2.7625104515531025e-06, 2.4801536405296596e-05,
                                0.0001984120875246986, 0.001388888890587323,   0.00833333335371942,
                                0.041666666666651364,  0.166666666666483,      0.5, 1.0, 1.0};
    constexpr int kTerms = sizeof(kCoef) / sizeof(double);
#pragma unroll
    for (int k = 0; k < N; ++k) p[k] = kCoef[0];
#pragma unroll
    for (int j = 1; j < kTerms; ++j) {
#pragma unroll
        for (int k = 0; k < N; ++k) p[k] = fma(p[k], r[k], kCoef[j]);
        if constexpr (N > 1) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        u32x2 bits = __builtin_bit_cast(u32x2, p[k]);
        bits[1] += __builtin_bit_cast(u32x2, m[k])[0] << 20;
        p[k] = __builtin_bit_cast(double, bits);
    }
}

// exp(d), d <= 0; below -700 as there.
__device__ __forceinline__ double exp64(double d) {
    d = fmax(d, -700.0);
    const double m[1] = {fma(d, kLog2e, kMagic)}, r[1] = {fma(m[0] - kMagic, -kLn2, d)};
    double p[1];
    exp_scaled(r, m, p);
    return p[0];
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

// A logit and its token: larger logits first, of equal ones the lower token.  0: none
// (-infinity and NaN); +infinity counts as the largest finite value.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) {
    return x > kNone ? (uint64_t)image(fminf(x, FLT_MAX)) << 32 | (uint32_t)~token : 0;
}

// A continuation: the image of its score, rounded to 41 bits, then beam * 64 + place in
// the beam's list, the lower the better: scores that are equal in 41 bits are equal.
// Rounded to nearest, since scores are often numbers of 24 bits (a beam's own, with
// one token left): they lie in the middle of what is rounded to them.  0: none.
__device__ __forceinline__ uint64_t entry_of(double score, uint32_t tag) {
    const uint64_t u = (__builtin_bit_cast(uint64_t, score) + 0x800) & ~(uint64_t)0xfff;
    return (image(__builtin_bit_cast(double, u)) & ~(uint64_t)0xfff) | (0xfff - tag);
}
__device__ __forceinline__ double entry_score(uint64_t e) {
    return __builtin_bit_cast(double, e >> 63 ? (e & ~(uint64_t)0xfff) ^ (uint64_t)1 << 63 : ~(e | 0xfff));
}

// The value of lane (this ^ MASK).  Inside rows of 16 lanes by DPP, across them by the
// row and half swaps: a sort of 64 keys makes no trip through LDS.
template <int MASK>
__device__ __forceinline__ uint32_t across(uint32_t v) {
    static_assert(MASK > 0 && MASK < 64, "lanes");
    if constexpr (MASK == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (threadIdx.x & 32) ? r[0] : r[1];
    } else if constexpr (MASK == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return (threadIdx.x & 16) ? r[0] : r[1];
    } else if constexpr (MASK > 32) {
        return across<32>(across<MASK - 32>(v));
    } else if constexpr (MASK > 16) {
        return across<16>(across<MASK - 16>(v));
    } else if constexpr (MASK == 4) {
        return across<7>(across<3>(v));
    } else {
        // quad permutes, mirror of half a row, turn by half a row, mirror of a row
        constexpr int kCtrl = MASK == 1 ? 0xB1 : MASK == 2 ? 0x4E : MASK == 3 ? 0x1B : MASK == 7 ? 0x141
                              : MASK == 8 ? 0x128 : 0x140;
        static_assert(MASK == 1 || MASK == 2 || MASK == 3 || MASK == 7 || MASK == 8 || MASK == 15, "one step");
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xF, 0xF, false);
    }
}
template <int MASK>
__device__ __forceinline__ uint64_t across(uint64_t v) {
    return (uint64_t)across<MASK>((uint32_t)(v >> 32)) << 32 | across<MASK>((uint32_t)v);
}
// One step of a sorting network: of lanes MASK apart, the one whose bit BIT is clear
// keeps the better value.
template <int MASK, int BIT>
__device__ __forceinline__ uint64_t exchange(uint64_t v) {
    const uint64_t o = across<MASK>(v);
    return (o > v) == !(threadIdx.x & BIT) ? o : v;
}

// Sorts groups of 2 W lanes whose values rise and then fall, or the like.
template <int W>
__device__ __forceinline__ uint64_t settle(uint64_t v) {
    if constexpr (W > 0) return settle<W / 2>(exchange<W, W>(v));
    else return v;
}

// The wave's 64 values, best in lane 0.
template <int W = 2>
__device__ __forceinline__ uint64_t sort64(uint64_t v) {
    v = settle<W / 4>(exchange<W - 1, W / 2>(v));
    if constexpr (W < 64) return sort64<2 * W>(v);
    else return v;
}

// The best 64 of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge64(uint64_t a, uint64_t b) {
    const uint64_t o = across<63>(b);
    return settle<32>(o > a ? o : a);
}

// The best 64 of the lists of waves 0 to `waves` - 1 (sorted), in wave 0: half of them
// go into the other half at a time.  By all waves of the workgroup.
template <int W>
__device__ __forceinline__ uint64_t merge_waves(uint64_t v, uint64_t (*lists)[64], int waves) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int w = W / 2; w > 0; w /= 2) {
        if (w >= waves) continue;
        if (wave >= w && wave < 2 * w) lists[wave - w][lane] = v;
        __syncthreads();
        if (wave < w) v = merge64(v, lists[wave][lane]);
        __syncthreads();
    }
    return v;
}

// Sum and maximum over the wave, in every lane (the lanes' sums a rounding apart
// where the compiler contracts a product into the first addition).
template <int MASK = 1>
__device__ __forceinline__ double all_sum(double v) {
    v += __builtin_bit_cast(double, across<MASK>(__builtin_bit_cast(uint64_t, v)));
    if constexpr (MASK < 32) return all_sum<2 * MASK>(v);
    else return v;
}
template <int MASK = 1>
__device__ __forceinline__ double all_max(double v) {
    v = fmax(v, __builtin_bit_cast(double, across<MASK>(__builtin_bit_cast(uint64_t, v))));
    if constexpr (MASK < 32) return all_max<2 * MASK>(v);
    else return v;
}
template <int MASK = 1>
__device__ __forceinline__ float all_max(float v) {
    v = fmaxf(v, __uint_as_float(across<MASK>(__float_as_uint(v))));
    if constexpr (MASK < 32) return all_max<2 * MASK>(v);
    else return v;
}

__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// Logits i .. i+7 of a row as they are, -infinity behind its end.  Rows need not be
// aligned.
template <typename T> struct None;
template <> struct None<float> { static constexpr float value = kNone; };
template <> struct None<uint16_t> { static constexpr uint16_t value = 0xff80; };

template <typename T>
struct Eight {
    T v[kPer];
    __device__ __forceinline__ void load(const T* row, int i, int vocab) {
        if (i + kPer <= vocab) {
            __builtin_memcpy(v, row + i, sizeof v);
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k) v[k] = i + k < vocab ? row[i + k] : None<T>::value;
        }
    }
};

// A wave's own places of LDS: what its lanes wrote is there for all of them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// What a stretch of a row leaves: its largest logit c and the sum of exp(x - c), beside
// its best keys.
struct Stretch {
    double c, sum;
};

struct Shape {
    int rows, width, vocab, n_out, splits, steps, waves;   // steps of 512 logits per wave to a stretch
};

// Of equal groups of lanes the least of the groups' largest.
template <int MASK = 1>
__device__ __forceinline__ float reached(float top, int group) {
    const float o = __uint_as_float(across<MASK>(__float_as_uint(top)));
    top = MASK < group ? fmaxf(top, o) : fminf(top, o);
    if constexpr (MASK < 32) return reached<2 * MASK>(top, group);
    else return top;
}

// The larger of two numbers.  fmaxf takes a second instruction for NaN that signal.
__device__ __forceinline__ float max_number(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// exp of bf16 values by table: those of magnitudes 2^-13 up to 64, both signs, an
// entry of 1 for what is smaller (with a correction where it is not 0), and of 0 for
// what is larger (negative, and far below the row's largest: see where it is used).
// Looking one up takes a quarter of the vector instructions of computing one (26.0
// to 16.0 million in all at 64 x 8 x 131072), and an LDS read whose lanes' places
// collide (4.5 of 8.2 million LDS cycles are conflicts).
struct ExpTable {
    static constexpr int kFirst = 0x3900, kPast = 0x4280, kSize = kPast - kFirst + 2;   // bits of 2^-13 and 64
    static constexpr int kBytes = 2 * kSize * 8;
    static_assert(kBytes < 65536, "byte offsets in 16 bits");
    static __device__ __forceinline__ void fill(double* t, int thread, int threads) {
        for (int j = thread; j < kSize; j += threads) {
            const double x = (double)bf16_to_f32((uint16_t)(kFirst - 1 + j));
            const double up = fma(x, kLog2e, kMagic), down = kMagic - (up - kMagic), rest = fma(up - kMagic, -kLn2, x);
            const double m[2] = {up, down}, r[2] = {rest, -rest};   // exp(x) and exp(-x)
            double e[2];
            exp_scaled(r, m, e);
#pragma unroll
            for (int i = 0; i < 2; ++i) t[i * kSize + j] = j == 0 ? 1.0 : j == kSize - 1 ? 0.0 : e[i];
        }
    }
    // exp(d) - 1 of magnitudes below 2^-13, beside the entry of 1.
    static __device__ __forceinline__ double rest(double d) { return fma(d * d, fma(d, 1.0 / 6.0, 0.5), d); }
    // Byte offsets of two values; their places (0: below 2^-13).
    static __device__ __forceinline__ u16x2 offsets(uint32_t two, u16x2& place) {
        const u16x2 b = __builtin_bit_cast(u16x2, two), size = {kSize * 8, kSize * 8}, lo = {kFirst - 1, kFirst - 1};
        const u16x2 m = __builtin_elementwise_max(__builtin_bit_cast(u16x2, two & 0x7fff7fffu), lo) - lo;
        place = __builtin_elementwise_min(m, u16x2{kSize - 1, kSize - 1});
        return place * (uint16_t)8 + (b >> (uint16_t)15) * size;
    }
};

// One workgroup of W waves per stretch of a row.  TABLE (bf16): exponentials by table
// where a wave's values allow it.
template <typename T, int W, bool TABLE>
__global__ __launch_bounds__(64 * W) void beam_rows_kernel(Shape sh, const T* logits, int64_t ld, const float* scores,
                                                          const uint8_t* finished, Stretch* stats, uint64_t* keys) {
    constexpr int kWaves = W, kThreads = 64 * W, kStep = kThreads * kPer;
    extern __shared__ __align__(16) uint8_t lds[];
    auto* held = reinterpret_cast<u32x2(*)[kHeld]>(lds);   // [wave]: logit and token
    [[maybe_unused]] auto* table = reinterpret_cast<double*>(lds + sizeof(u32x2) * kHeld * kWaves);
    __shared__ uint64_t list[64], lists[kWaves / 2][64];
    __shared__ int kept[2][kWaves];   // of even and odd steps: the last step's may still be read
    __shared__ double sums[kWaves];
    __shared__ float2 bounds[kWaves];
    __shared__ float last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = blockIdx.x / sh.splits, split = blockIdx.x % sh.splits;
    const T* x_row = logits + row * ld;
    const int begin = split * sh.steps * kStep, end = (int)min((int64_t)sh.vocab, (int64_t)begin + sh.steps * kStep);
    Eight<T> next;
    next.load(x_row, begin + (int)threadIdx.x * kPer, sh.vocab);
    // a beam without continuations, or with one that needs no logits
    if (!(fabsf(scores[row]) <= FLT_MAX) || (finished && finished[row])) return;
    if constexpr (TABLE) ExpTable::fill(table, threadIdx.x, kThreads);   // a barrier follows in the first step
    // lanes to a part, for the first bound: parts of one wave, of all waves
    const int alone = 64 >> (sh.n_out > 1 ? 32 - __builtin_clz(sh.n_out - 1) : 0);
    const int group = min(64, alone * kWaves);
    // Sums are of exp(x - c) with c = n ln 2, so that the exponent's integer takes c in;
    // where |c| is large, x is first made x - base in fp32, exact where it counts.  That
    // c is no logit, so the largest one's term is 1 within its rounding only.
    float c = -FLT_MAX, base = c, least = kNone;   // least: the list's last key that counts
    double shift = kMagic, sum = 0.0;
    [[maybe_unused]] bool by_table = false;   // the wave's largest is -20 to 64 so far, and c is 0
    int n = 0, joins = 0, odd = 0;
    for (int i = begin; i < end; i += kStep) {
        float x[kPer];
        const int at = i + (int)threadIdx.x * kPer;
        const Eight<T> now = next;
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[k] = Io<T>::load(now.v, k);
        if (i + kStep < end) next.load(x_row, at + kStep, sh.vocab);
        // infinities and NaN are always above and always far
        const float reach = TABLE && by_table ? 63.75f : c + 600.0f, bar = fminf(least, reach);
        uint64_t above[kPer], some = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) some |= above[k] = __ballot(!(x[k] <= bar));
        if (some || i == begin) {
            uint64_t far = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (above[k]) far |= __ballot(!(x[k] <= reach));
            if (far || i == begin) {
#pragma unroll
                for (int k = 0; k < kPer; ++k) x[k] = x[k] != x[k] ? kNone : fminf(x[k], FLT_MAX);
                float top = x[0];
#pragma unroll
                for (int k = 1; k < kPer; ++k) top = fmaxf(top, x[k]);
                if (__any(top > reach)) {   // also the first time, unless nothing is above the lowest value
                    const double old = (double)base + (kMagic - shift) * kLn2;
                    c = all_max(top);
                    by_table = TABLE && c >= -20.0f && c < 64.0f;
                    if (by_table) c = 0.0f;
                    const double ints = rint((double)c * kLog2e);
                    base = fabsf(c) > 1e5f ? c : 0.0f;
                    shift = fabsf(c) > 1e5f ? kMagic : kMagic - ints;
                    sum *= exp64(old - ((double)base + (kMagic - shift) * kLn2));
                }
                if (i == begin) {
                    // A bound that n_out logits of the step reach: of equal parts of the lanes,
                    // no fewer than n_out, the least of the parts' largest; parts of all waves,
                    // or of one where another has little.  Those equal to it may count, so
                    // it is the number below it.
                    const float own = reached(top, alone);
                    top = reached(top, group);
                    if (lane == 0) bounds[wave] = {top, own};
                    __syncthreads();
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) top = fminf(top, bounds[w].x);
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, bounds[w].y);
                    least = top > kNone ? image_value(image(top) - (top == 0.0f ? 2 : 1)) : kNone;
                }
            }
            // Equal to the list's last is not enough: tokens are higher here.
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (!above[k] && i != begin) continue;
                const uint64_t mask = __ballot(x[k] > least);
                const uint32_t to = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                              __builtin_amdgcn_mbcnt_lo((uint32_t)mask, n));
                if (x[k] > least) held[wave][to] = u32x2{__float_as_uint(x[k]), (uint32_t)(at + k)};
                n += __popcll(mask);
            }
        }
        odd ^= 1;
        if (lane == 0) kept[odd][wave] = n;
        if (TABLE && by_table) {
            if constexpr (TABLE) {
                uint32_t two[kPer / 2];
                __builtin_memcpy(two, now.v, sizeof two);
                u16x2 least_place = {0xffff, 0xffff};
                double e[kPer];
#pragma unroll
                for (int k = 0; k < kPer; k += 2) {
                    u16x2 place;
                    const u16x2 at2 = ExpTable::offsets(two[k / 2], place);
                    least_place = __builtin_elementwise_min(least_place, place);
                    e[k] = *reinterpret_cast<const double*>(reinterpret_cast<const char*>(table) + at2[0]);
                    e[k + 1] = *reinterpret_cast<const double*>(reinterpret_cast<const char*>(table) + at2[1]);
                }
#pragma unroll
                for (int k = 0; k < kPer; ++k) sum += e[k];
                if (__any(least_place[0] == 0 || least_place[1] == 0)) {
#pragma unroll
                    for (int k = 0; k < kPer; ++k) sum += ExpTable::rest(fabsf(x[k]) < 0x1p-13f ? (double)x[k] : 0.0);
                }
            }
        } else {
            if (base != 0.0f) {
#pragma unroll
                for (int k = 0; k < kPer; ++k) x[k] = x[k] - base;
            }
            const float low = c - base - 700.0f;
#pragma unroll
            for (int k0 = 0; k0 < kPer; k0 += kSide) {
                double m[kSide], r[kSide], e[kSide];
#pragma unroll
                for (int k = 0; k < kSide; ++k) {
                    const double d = (double)max_number(x[k0 + k], low);
                    m[k] = fma(d, kLog2e, shift);
                    r[k] = fma(m[k] - shift, -kLn2, d);
                }
                exp_scaled(r, m, e);
#pragma unroll
                for (int k = 0; k < kSide; ++k) sum += e[k];
            }
        }
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) total += kept[odd][w];
        if (total < 64 && i != begin && i + kStep < end) continue;
        // A few keys one wave sorts, the waves in turn; more every wave its own.
        const bool many = total > 64;
        uint64_t best = 0;
        if (many) {
            for (int from = 0; from < n; from += 64) {
                const u32x2 e = from + lane < n ? held[wave][from + lane] : u32x2{__float_as_uint(kNone), 0};
                const uint64_t v = sort64(key_of(__uint_as_float(e[0]), e[1]));
                best = from ? merge64(best, v) : v;
            }
            best = merge_waves<kWaves>(best, lists, kWaves);
        }
        if (wave == (many ? 0 : joins % kWaves)) {
            if (!many) {
                // place lane of the waves' keys, one behind the other
                int w = 0, to = lane;
                while (w < kWaves && to >= kept[odd][w]) to -= kept[odd][w++];
                const u32x2 e = w < kWaves ? held[w][to] : u32x2{__float_as_uint(kNone), 0};
                best = sort64(key_of(__uint_as_float(e[0]), e[1]));
            }
            if (joins) best = merge64(best, list[lane]);
            list[lane] = best;
            const uint32_t high = (uint32_t)(read_lane(best, sh.n_out - 1) >> 32);
            if (lane == 0) last = high ? image_value(high) : kNone;
        }
        __syncthreads();
        least = last;
        n = 0;
        ++joins;
    }
    // The sum beside the largest logit, of the whole stretch: over its term as this wave
    // makes terms, so that what the one logit leaves of the sum is 1.  Another wave may
    // hold one that this wave's terms cannot express.
    sum = all_sum(sum);
    const uint64_t first = list[0];
    const float most = first ? image_value((uint32_t)(first >> 32)) : -FLT_MAX;
    if (!first) {
        sum = 0.0;
    } else if (!(most <= (TABLE && by_table ? 63.75f : c + 600.0f))) {
        sum *= exp64((double)base + (kMagic - shift) * kLn2 - (double)most);
    } else if (TABLE && by_table) {
        if constexpr (TABLE) {
            u16x2 place;
            const u16x2 at2 = ExpTable::offsets(__float_as_uint(most) >> 16, place);
            double e = *reinterpret_cast<const double*>(reinterpret_cast<const char*>(table) + at2[0]);
            if (place[0] == 0) e += ExpTable::rest((double)most);
            sum /= e;
        }
    } else {
        const double d = (double)max_number(most - base, c - base - 700.0f);
        const double m[1] = {fma(d, kLog2e, shift)}, r[1] = {fma(m[0] - shift, -kLn2, d)};
        double e[1];
        exp_scaled(r, m, e);
        sum /= e[0];
    }
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) all += sums[w];
        stats[blockIdx.x] = {(double)most, all};
    }
    if (wave == 0 && lane < sh.n_out) keys[(int64_t)blockIdx.x * sh.n_out + lane] = list[lane];
}

// One workgroup per request: each wave puts the stretches of its beams together, then
// half of the waves' lists go into the other half's at a time.  4.9 us for 64 x 8
// beams, a launch and three trips to memory.
__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(Shape sh, const Stretch* stats, const uint64_t* keys,
                                                                  const float* scores, const uint8_t* finished, int eos,
                                                                  int32_t* parents, int32_t* tokens, float* scores_out,
                                                                  uint8_t* finished_out) {
    __shared__ uint64_t held[kMergeWaves][128];
    __shared__ int32_t token[GDN_BEAM_MAX * GDN_BEAM_MAX];
    auto* lists = reinterpret_cast<uint64_t(*)[64]>(held);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t req = blockIdx.x;
    uint64_t mine = 0;
    for (int b = wave; b < sh.width; b += kMergeWaves) {
        const int64_t row = req * sh.width + b;
        // all loads at once; what a beam without logits has there is not looked at
        const int count = sh.splits * sh.n_out;
        const uint64_t* from = keys + row * count;
        // the lists' first keys come first
        const auto key_at = [&](int i) { return i < count ? from[i % sh.splits * sh.n_out + i / sh.splits] : 0; };
        uint64_t key[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) key[j] = key_at(j * 64 + lane);
        const Stretch st = lane < sh.splits ? stats[row * sh.splits + lane] : Stretch{-HUGE_VAL, 0.0};
        const float base = scores[row];
        const bool done = finished && finished[row];
        if (!(fabsf(base) <= FLT_MAX)) continue;
        const uint32_t tag = b * 64 + lane;
        uint64_t e = 0;
        if (done) {
            if (lane == 0) {
                e = entry_of((double)base, tag);
                token[tag] = eos;
            }
        } else {
            const double c = all_max(st.c);
            const double sum = all_sum(st.sum * exp64(st.c - c));
            // One lane's sum for all: equal logits need equal scores.  Apart from c, beside
            // which the logarithm would be lost where logits reach 1e38.
            const double norm = log(__builtin_bit_cast(double, read_lane(__builtin_bit_cast(uint64_t, sum), 0)));
            // The lists are sorted, so few keys but the first pass; they wait in LDS for
            // a sort of 64.  Where none of 64 passes, every list has one, and none further
            // down is larger.
            uint64_t best = sh.splits > 1 ? sort64(key[0]) : key[0], bar = read_lane(best, sh.n_out - 1);
            int n = 0;
            const auto join = [&]() {
                wave_sync();
                best = merge64(best, sort64(lane < n ? held[wave][lane] : 0));
                bar = read_lane(best, sh.n_out - 1);
                const uint64_t rest = 64 + lane < n ? held[wave][64 + lane] : 0;
                wave_sync();
                held[wave][lane] = rest;
                n = max(n - 64, 0);
            };
            bool more = true;
            for (int i = 64; i < count && more; i += 64 * kBatch) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) key[j] = j + 1 < kBatch && i == 64 ? key[j + 1] : key_at(i + j * 64 + lane);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const uint64_t mask = __ballot(key[j] > bar);
                    more = more && mask;
                    if (!more) continue;
                    const uint32_t to = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                                  __builtin_amdgcn_mbcnt_lo((uint32_t)mask, n));
                    if (key[j] > bar) held[wave][to] = key[j];
                    n += __popcll(mask);
                    if (n >= 64) join();
                }
            }
            if (n > 0) join();
            if (best && lane < sh.n_out) {
                token[tag] = (int32_t)~(uint32_t)best;
                e = entry_of((double)base + (((double)image_value((uint32_t)(best >> 32)) - c) - norm), tag);
            }
        }
        mine = b < kMergeWaves ? e : merge64(mine, e);
    }
    __syncthreads();   // held is free
    mine = merge_waves<kMergeWaves>(mine, lists, sh.width);
    if (wave != 0 || lane >= sh.n_out) return;
    const int64_t at = req * sh.n_out + lane;
    const bool some = mine != 0;
    const int tag = some ? 0xfff - (int)(mine & 0xfff) : 0;
    const int parent = some ? tag / 64 : -1, tok = some ? token[tag] : -1;
    parents[at] = parent;
    tokens[at] = tok;
    scores_out[at] = some ? (float)entry_score(mine) : kNone;   // of the rounded score: it never rises
    if (finished_out)
        finished_out[at] = some && ((finished && finished[req * sh.width + parent]) || tok == eos);
}

// Stretches: enough workgroups for the card, at most a lane's worth, none empty.
Shape beam_shape(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out, int waves, int wanted) {
    const int rows = n_req * width, step = waves * 64 * kPer, steps = (vocab + step - 1) / step;
    const int want = std::max(1, std::min({kMaxSplits, steps, wanted / std::max(1, rows)}));
    const int per = (steps + want - 1) / want;
    return {rows, width, vocab, n_out, (steps + per - 1) / per, per, waves};
}

// Workgroups of eight waves with the table, two to a CU, where each has eight steps or
// more to fill it for; of four waves otherwise, four to a CU.  With the table and
// without it: 64 x 8 x 131072 58 and 77 us, 32 x 8 x 131072 38 and 46, 64 x 8 x 32000
// (eight steps) 28.0 and 31.0, 64 x 4 x 32000 (four) 20.7 and 20.0, 1 x 4 x 32000 11.7
// and 9.5.  Twice the workgroups with the table: 68 us for 64 x 8 x 131072.
Shape beam_plan(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out, gdn_dtype dtype) {
    const Shape s = beam_shape(n_req, width, vocab, n_out, 8, 512);
    return dtype == GDN_BF16 && s.steps >= 8 ? s : beam_shape(n_req, width, vocab, n_out, 4, 1024);
}

size_t stats_bytes(const Shape& s) {
    return ((size_t)s.rows * s.splits * sizeof(Stretch) + 255) / 256 * 256;
}

template <typename T, int W, bool TABLE>
hipError_t launch_rows(const Shape& s, const void* logits, int64_t ld, const float* scores, const uint8_t* finished,
                       Stretch* stats, uint64_t* keys, hipStream_t stream) {
    constexpr int lds = sizeof(u32x2) * kHeld * W + (TABLE ? ExpTable::kBytes : 0);
    if (lds > 60000) {
        static std::atomic<uint64_t> done{0};
        const hipError_t e = allow_dynamic_lds(&beam_rows_kernel<T, W, TABLE>, lds, &done);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((beam_rows_kernel<T, W, TABLE>), dim3((unsigned)(s.rows * s.splits)), dim3(64 * W), lds, stream, s,
                       static_cast<const T*>(logits), ld, scores, finished, stats, keys);
    return hipGetLastError();
}

}  // namespace

// Enough for either type.
size_t beam_select_workspace_bytes(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out) {
    size_t most = 0;
    for (const gdn_dtype t : {GDN_F32, GDN_BF16}) {
        const Shape s = beam_plan(n_req, width, vocab, n_out, t);
        most = std::max(most, stats_bytes(s) + (size_t)s.rows * s.splits * n_out * sizeof(uint64_t));
    }
    return most;
}

hipError_t launch_beam_select(int32_t n_req, int32_t width, int32_t vocab, int32_t n_out, gdn_dtype dtype,
                              const void* logits, int64_t ld, const float* scores, const uint8_t* finished,
                              int32_t eos, int32_t* parents, int32_t* tokens, float* scores_out,
                              uint8_t* finished_out, void* workspace, hipStream_t stream) {
    const Shape s = beam_plan(n_req, width, vocab, n_out, dtype);
    Stretch* stats = static_cast<Stretch*>(workspace);
    uint64_t* keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + stats_bytes(s));
    const hipError_t e =
        dtype == GDN_F32 ? launch_rows<float, 4, false>(s, logits, ld, scores, finished, stats, keys, stream)
        : s.waves == 4   ? launch_rows<uint16_t, 4, false>(s, logits, ld, scores, finished, stats, keys, stream)
                         : launch_rows<uint16_t, 8, true>(s, logits, ld, scores, finished, stats, keys, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(beam_merge_kernel, dim3(n_req), dim3(kMergeThreads), 0, stream, s, stats, keys, scores,
                       finished, eos, parents, tokens, scores_out, finished_out);
    return hipGetLastError();
}

}  // namespace gdn
