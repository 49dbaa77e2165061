// route_scored_kernels.cuh -- routing on given logits: scores, selection bias, groups,
// top-k, renormalised gates; and the gradient of the gates to the logits.
//
// For a row of logits l (E experts):
//     s_i = exp(l_i) / sum_j exp(l_j)   or   s_i = 1 / (1 + exp(-l_i))
//     c_i = s_i + bias_i                          (the choice; bias optional)
//     groups of E / n_group experts, valued by the sum of their group_top
//     largest choices; the topk_group best groups stay
//     S = the k largest choices left (ties: the lower index)
//     gate_i = scale * s_i / sum_{j in S} s_j     (or scale * s_i)
//
// Forward: LPR lanes (8, 16 or 32) work on a row, so 4, 2 or 1 rows share a warp's
// instructions; a lane holds V experts, and a group is P whole lanes (rows whose groups
// do not fill their lanes are padded with -inf).  A choice becomes a 32-bit key, its
// value in the upper 23 bits and the expert's number in the lower 9, so that minimum
// and maximum move both at once and a lower number wins a tie.  The value is the distance
// from the row's largest choice in fixed point, 2^-23 of a range of 4 (biased choices)
// or 32 (logits); bf16 logits without a bias keep their 16 bits instead.  Each lane
// sorts its best KL >= k keys; a group's value comes from the first two of its lanes'
// lists; then the lanes' lists are merged in pairs, KL against KL, which leaves the
// row's best in every lane and the best of all that fell out in `out`.
//
// Further attempts, each taken only where the one before could not tell two experts
// (or the last kept and first dropped group) apart:
//  1. the keys: rows whose neighbours in the selected order have the same value, or
//     differ by less than the error of a float32 score, go on; groups whose values lie
//     that close are valued by their two best keys' choices in float64.
//  2. the KL best in float64, one a lane: their ranking decides, unless `out` may lie
//     as high as the k-th.
//  3. all keys that may lie as high as the k-th, one a lane, in float64.
//  4. all choices in float64 by the whole warp: where a biased softmax needs its sum in
//     float64, or a selected choice lies beyond the keys' range.  Groups without a live
//     expert, and slots that no live expert is left for, are known without it.
// So the selection is that of float64 scores.  A launch waits for its last warp, and
// 16384 rows nearly always hold some of the second and third kind: with the fourth
// attempt in place of the third, and for close groups, it took 3 to 8 us longer.
//
// What bounds it: instructions.  16384 rows of 256 experts, sigmoid, bias, 4 of 8
// groups, top-8 (18 MB, 3 us at the memory's rate) take 16 to 20 us, 12 of them the keys
// and lists of about 400 instructions a row and the rest scores, groups and the last warps'
// further attempts; a row a warp with rounds of warp-wide maxima took 1000 instructions and 31 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "route_scored.cuh"

namespace moe {
namespace scored {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;         // backward: rows in work per block
constexpr int kForwardWarps = 4;  // forward: warps per block
// Blocks an SM holds: as many as V values a lane leave registers for.
constexpr int blocks_per_sm(int V) { return V <= 2 ? 6 : V == 4 ? 5 : V == 8 ? 4 : 2; }

struct Args {
    int T, E, k;
    int sigmoid, renorm;
    int n_group, group_size, topk_group;
    int group_lanes;  // forward: P, lanes of one group
    int lane_size;    // forward: V, the experts that a lane takes of its group
    int aligned;      // forward: expert i is value i of the row's lanes (no padding inside)
    int biased;       // choices are scores plus a bias; otherwise logits order them
    int sums;         // groups are valued by a sum of two choices
    int whole_keys;   // without a bias, keys leave their low bits zero (bf16 logits)
    float steps;      // key values per unit of choice (2^23 / range)
    int slots;        // k, rounded up to a power of two
    int unit;         // bytes a row can be read in at a time (16, 8, 4 or 2)
    int vec;          // backward: rows can be read in vectors
    float scale;
};

// ------------------------------------------------------------------ row access
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <int BYTES>
struct Vec {
    typedef uint4 type;
};
template <>
struct Vec<8> {
    typedef uint2 type;
};
template <>
struct Vec<4> {
    typedef uint32_t type;
};
template <>
struct Vec<2> {
    typedef uint16_t type;
};

template <typename L, int V>
struct RowVec {
    static constexpr int kBytes = V * (int)sizeof(L);
    static constexpr int kUnit = kBytes < 16 ? kBytes : 16;
    static constexpr int kUnits = kBytes / kUnit;
    typedef typename Vec<kUnit>::type type;
    union {
        type u[kUnits];
        L v[V];
    };
};

// This lane's V logits as they are stored; past E, -inf.
template <typename L, int V>
__device__ __forceinline__ void load_row(const L* row, const Args& a, int i0, RowVec<L, V>& r) {
    typedef RowVec<L, V> R;
    if (a.vec && i0 + V <= a.E) {
        const typename R::type* src = reinterpret_cast<const typename R::type*>(row + i0);
#pragma unroll
        for (int j = 0; j < R::kUnits; ++j) r.u[j] = __ldg(src + j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) r.v[j] = i0 + j < a.E ? row[i0 + j] : (L)(-INFINITY);
    }
}

// ... as floats, NaN as -inf.
template <typename L, int V>
__device__ __forceinline__ void to_floats(const RowVec<L, V>& r, float (&l)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = fmaxf(to_float(r.v[j]), -INFINITY);
}

// ------------------------------------------------------------------ ordered keys
// key(a) > key(b) exactly when a > b; 0 is below every number and stands for
// "not selectable".  Adding +0 makes the two zeros one.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ unsigned long long ordered(double f) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(f + 0.0);
    return b ^ ((unsigned long long)((long long)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_key(unsigned long long k) {
    return __longlong_as_double(
        (long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : 0xffffffffffffffffull)));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((unsigned long long)hi << 32) | lo;
}

template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}

__device__ __forceinline__ float warp_max_float(float v) { return from_key(warp_max(ordered(v))); }

// exp(l - m) with l <= m; 1 where they are equal (both infinite among it).
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }
// Relative to e^-|l|, so that values below float32's smallest normal number (l < -87.3) do not read 0.
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return __fdiv_rn(l >= 0.0f ? 1.0f : e, 1.0f + e);
}
__device__ __forceinline__ double sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }

// The row's largest logit and the sum of exp(l - m) over its live experts.
template <typename R, int V>
__device__ __forceinline__ void softmax_stats(const float (&l)[V], R& m, R& sum) {
    float mine = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j) mine = fmaxf(mine, l[j]);
    m = (R)warp_max_float(mine);
    R part = (R)0;
#pragma unroll
    for (int j = 0; j < V; ++j) part += l[j] > -INFINITY ? exp_below((R)l[j], m) : (R)0;
    sum = warp_sum(part);
}

// Two largest of two pairs of two (b1 >= b2).
template <typename K>
__device__ __forceinline__ void merge_top2(K& b1, K& b2, K o1, K o2) {
    const K lo = b1 < o1 ? b1 : o1;
    b1 = b1 < o1 ? o1 : b1;
    b2 = b2 < o2 ? o2 : b2;
    b2 = b2 < lo ? lo : b2;
}

// ------------------------------------------------------------------ fourth attempt
static __device__ __noinline__ double score_double(double x, bool is_sigmoid, double m, double inv) {
    // one exponential for both kinds: it is the bulk of this path's instructions, which
    // nearly always have to be fetched when a row needs them
    const double e = exp(is_sigmoid ? -x : (x == m ? 0.0 : x - m));
    return is_sigmoid ? 1.0 / (1.0 + e) : e * inv;
}

// Selects the row's k experts by the whole warp: lane r < k returns the expert of slot
// r, or -1.  All choices in float64, in `c` (E values of shared memory); without a
// bias the logits order the experts.  Rolled loops: few rows come here, and a kernel's
// last warp waits for them (8 us a row with the loops unrolled, 2 without).
template <typename L>
__device__ __noinline__ int select_double(const L* __restrict__ row, const Args& a,
                                          const float* __restrict__ bias, int lane, double* c) {
    typedef unsigned long long K;
    double m = 0.0, inv = 1.0;
    if (!a.sigmoid && (a.biased || a.sums)) {
        float top = -INFINITY;
#pragma unroll 1
        for (int i = lane; i < a.E; i += 32) top = fmaxf(top, to_float(row[i]));
        m = (double)from_key(__reduce_max_sync(kAll, ordered(top)));
        double sum = 0.0;
#pragma unroll 1
        for (int i = lane; i < a.E; i += 32) {
            const float f = to_float(row[i]);
            if (f > -INFINITY) sum += score_double((double)f, false, m, 1.0);
        }
        inv = 1.0 / warp_sum(sum);
    }
#pragma unroll 1
    for (int i0 = lane; i0 < a.E; i0 += 128) {
        double v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (an expert past E has score 1 or inv, and no place)
            const int i = i0 + 32 * j;
            v[j] = i < a.E ? (double)to_float(row[i]) : m;
        }
        if (a.biased) {
            double b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double x = v[j];
                b[j] = exp(a.sigmoid ? -x : (x == m ? 0.0 : x - m));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 32 * j;
                if (v[j] > -INFINITY)
                    v[j] = (a.sigmoid ? 1.0 / (1.0 + b[j]) : b[j] * inv) +
                           (i < a.E ? (double)__ldg(bias + i) : 0.0);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + 32 * j < a.E) c[i0 + 32 * j] = v[j] > -INFINITY ? v[j] : -INFINITY;
    }
    __syncwarp();
    if (a.n_group > 1) {
        K value = 0;
#pragma unroll 1
        for (int g = 0; g < a.n_group; ++g) {
            K t1 = 0, t2 = 0;
#pragma unroll 1
            for (int i = g * a.group_size + lane; i < (g + 1) * a.group_size; i += 32)
                merge_top2(t1, t2, c[i] > -INFINITY ? ordered(c[i]) : (K)0, (K)0);
            const K m1 = warp_max(t1);
            const bool many = __popc(__ballot_sync(kAll, t1 == m1)) > 1;
            const K m2 = warp_max(t1 == m1 && !many ? t2 : t1);
            if (lane == g && m1 != 0) {
                value = m1;
                if (a.sums) {
                    double v1 = from_key(m1), v2 = m2 != 0 ? from_key(m2) : 0.0;
                    if (!a.biased) {
                        v1 = score_double(v1, a.sigmoid, m, inv);
                        if (m2 != 0) v2 = score_double(v2, a.sigmoid, m, inv);
                    }
                    value = ordered(v1 + v2);
                }
            }
        }
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < a.n_group; ++g) {
            const K o = __shfl_sync(kAll, value, g);
            rank += o > value || (o == value && g < lane);
        }
        const unsigned keep = __ballot_sync(kAll, lane < a.n_group && rank < a.topk_group);
#pragma unroll 1
        for (int i = lane; i < a.E; i += 32)
            if (!((keep >> (i / a.group_size)) & 1u)) c[i] = -INFINITY;
        __syncwarp();
    }
    int mine = -1;
#pragma unroll 1
    for (int r = 0; r < a.k; ++r) {
        double head = -INFINITY;
        int at = 0x7fffffff;
#pragma unroll 4
        for (int i = lane; i < a.E; i += 32)
            if (c[i] > head) {
                head = c[i];
                at = i;
            }
        const K key = head > -INFINITY ? ordered(head) : (K)0;
        const K best = warp_max(key);
        if (best == 0) break;
        const int chosen = (int)__reduce_min_sync(kAll, key == best ? (unsigned)at : 0xffffffffu);
        if (lane == r) mine = chosen;
        if (lane == (chosen & 31)) c[chosen] = -INFINITY;
        __syncwarp();
    }
    __syncwarp();
    return mine;
}

// ------------------------------------------------------------------ packed keys
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A float32 score, off by less than score_error().
__device__ __forceinline__ float fast_score(float l, const Args& a, float m, float inv) {
    constexpr float kLog2e = 1.4426950408889634f;
    if (a.sigmoid) return rcp_fast(1.0f + exp2_fast(-l * kLog2e));
    return l == m ? inv : exp2_fast((l - m) * kLog2e) * inv;
}

// Sigmoid: the exponent's rounding and ex2's two ulps move s by s (1 - s) (|l| 2^-24 +
// 2^-22) < 0.9 2^-24, the sum and the reciprocal by 1.5 2^-24; bound 6 2^-24.  Softmax: the same
// and the rounding of its sum, a tree of at most 5 + 5 additions, relative to the row's
// largest score inv; bound 64 2^-24.
__device__ __forceinline__ float score_error(const Args& a, float inv) {
    return a.sigmoid ? 3.5762787e-7f : 3.8146973e-6f * inv;
}
constexpr float kRound = 6.0e-8f;  // 2^-24, rounded up

// Keys.  Value part: the low 23 bits of a float in [2^23, 2^24), whose
// integers they count; everything further than the range below `top`, -inf among it,
// has value 0.
constexpr int kNumberBits = 9;
constexpr uint32_t kNumber = (1u << kNumberBits) - 1u;
constexpr float kFull = 16777215.0f;   // 2^24 - 1: the value of the largest choice
constexpr float kNone = 8388608.0f;    // 2^23

// A key's number part.  A lane's places that no expert fills count on past the last expert, so
// their numbers may need more than 9 bits (510 experts in 15 groups of two lanes: up to 524); such
// a key holds -inf and is never selected, but its number must not reach the value part.
__host__ __device__ constexpr uint32_t number_part(int number) {
    return (kNumber - (uint32_t)number) & kNumber;
}
static_assert(number_part(0) == kNumber && number_part(kScoredMaxE - 1) == kNumber + 1 - kScoredMaxE,
              "lower numbers make higher keys");
static_assert(number_part(kScoredMaxE) <= kNumber && number_part(4 * kScoredMaxE) <= kNumber,
              "numbers past the last expert stay within the number part");

__device__ __forceinline__ uint32_t make_key(float c, float top, const Args& a, int number) {
    if (a.whole_keys) return (ordered(c) & 0xffff0000u) | number_part(number);
    const float v = fmaxf(fmaf(c - top, a.steps, kFull), kNone);
    return (__float_as_uint(v) << kNumberBits) | number_part(number);
}
// bf16 keys: -inf is below every number's key
__device__ __forceinline__ bool selectable(uint32_t key, const Args& a) {
    return key >= (a.whole_keys ? 0x00800000u : 1u << kNumberBits);
}
__device__ __forceinline__ int number_of(uint32_t key) { return (int)(kNumber - (key & kNumber)); }
// The choice, within half a step (exactly for bf16 logits: the bits that a negative
// one's complement would have set read as zero, so they are set here).
__device__ __forceinline__ float decode(uint32_t key, float top, const Args& a) {
    if (a.whole_keys) return from_key((key >> 31) ? key & 0xffff0000u : key | 0x0000ffffu);
    return top - (kFull - kNone - (float)(key >> kNumberBits)) * (1.0f / a.steps);
}

// Descending, by Batcher's odd-even merge network.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t* k) {
#pragma unroll
    for (int p = 1; p < N; p *= 2) {
#pragma unroll
        for (int q = p; q >= 1; q /= 2) {
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q) {
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(k[i + j], k[i + j + q]);
                        k[i + j + q] = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                    }
                }
            }
        }
    }
}

// a, b descending: a becomes the KL best of both, descending, `out` the largest of
// itself and the others.
template <int KL>
__device__ __forceinline__ void merge_best(uint32_t (&a)[KL], const uint32_t* b, uint32_t& out) {
#pragma unroll
    for (int i = 0; i < KL; ++i) {  // leaves a bitonic sequence
        out = max(out, min(a[i], b[KL - 1 - i]));
        a[i] = max(a[i], b[KL - 1 - i]);
    }
#pragma unroll
    for (int q = KL / 2; q >= 1; q /= 2) {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            if ((i & q) == 0) {
                const uint32_t hi = max(a[i], a[i + q]);
                a[i + q] = min(a[i], a[i + q]);
                a[i] = hi;
            }
        }
    }
}

// Weight of a selected expert before any division by the sum.  With
// renormalisation only ratios count: the sigmoid is then taken relative to
// exp(min(M, 0)), M the largest selected logit, so that it cannot underflow
// however negative all of them are.
__device__ __forceinline__ float sigmoid_ratio(float l, float M) {
    const float e = expf(-fabsf(l));
    const float top = l >= 0.0f ? 1.0f : (M < 0.0f ? exp_below(l, M) : e);
    return __fdiv_rn(top, 1.0f + e);
}

// ------------------------------------------------------------------ forward
// Place of expert i among the row's LPR * V values.
template <int V>
__device__ __forceinline__ int place_of(int i, const Args& a) {
    if (a.aligned) return i;
    const int g = i / a.group_size;
    const int in = i - g * a.group_size;
    const int part = in / a.lane_size;
    return (g * a.group_lanes + part) * V + in - part * a.lane_size;
}

// One asynchronous copy to shared memory.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "n"(kBytes)
                 : "memory");
}
template <int kBytes>
__device__ __forceinline__ void stage_bytes(const void* row, int bytes, int lane, void* to) {
    for (int b = lane * kBytes; b < bytes; b += 32 * kBytes)
        copy_async<kBytes>(static_cast<char*>(to) + b, static_cast<const char*>(row) + b);
}

// Copies one row to shared memory in the lanes' order, by the warp.  Asynchronously where
// the copy unit has the size for it, so that a warp's rows are all on their way at once
// (one after the other they cost 0.3 us each).
template <typename L, int V>
__device__ __forceinline__ void stage_row(const L* __restrict__ row, const Args& a, int lane,
                                          L* to) {
    const int bytes = a.E * (int)sizeof(L);
    if (a.aligned && a.unit == 16) {
        stage_bytes<16>(row, bytes, lane, to);
    } else if (a.aligned && a.unit == 8) {
        stage_bytes<8>(row, bytes, lane, to);
    } else if (a.aligned && a.unit == 4) {
        stage_bytes<4>(row, bytes, lane, to);
    } else if constexpr (sizeof(L) == 4) {
        for (int i = lane; i < a.E; i += 32) copy_async<4>(to + place_of<V>(i, a), row + i);
    } else {
#pragma unroll 4
        for (int i = lane; i < a.E; i += 32) to[place_of<V>(i, a)] = __ldg(row + i);
    }
}

template <int LPR, typename R>
__device__ __forceinline__ R row_sum(R v) {
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
// term(0) + ... + term(N - 1), neighbours first: ((0 + 1) + (2 + 3)) + ...  With row_sum
// behind it, the sum over a row's places is the same balanced tree however many lanes share the row
// (empty places add 0, and a turned piece stays beside its neighbour), so a row's bits do
// not depend on how many rows there are.
template <int N, typename F>
__device__ __forceinline__ float tree_sum(F term, int first = 0) {
    if constexpr (N == 1)
        return term(first);
    else
        return tree_sum<N / 2>(term, first) + tree_sum<N / 2>(term, first + N / 2);
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
    return v;
}

// Whether this lane's group stays.  b1, b2: its two best keys; `live`: it has an expert that can be
// chosen.  Each group's value is known to lie in [lo, hi]; `open`: these do not
// decide whether the group stays.
template <int LPR>
__device__ __forceinline__ bool keep_group(uint32_t b1, uint32_t b2, bool live, const Args& a,
                                           float top, float m, float inv, float error, int base,
                                           int group, bool& open) {
    // a group without a choice: below every other, a lower number first
    uint32_t lo = (uint32_t)(31 - (group & 31)), hi = lo;
    if (selectable(b1, a)) {
        float value, err;
        const float c1 = decode(b1, top, a);
        const bool two = selectable(b2, a);
        const float c2 = two ? decode(b2, top, a) : 0.0f;
        if (!a.sums) {
            value = c1;
            err = error;
        } else if (a.biased) {
            value = c1 + c2;
            err = 2.0f * error + kRound * fabsf(value);
        } else {  // scores: their own error, and what their logits' error moves them
            const float s1 = fast_score(c1, a, m, inv), s2 = two ? fast_score(c2, a, m, inv) : 0.0f;
            value = s1 + s2;
            err = 2.0f * score_error(a, inv) + 1.01f * error * value;
        }
        // a second best beyond the range could be anything below it
        if (a.sums && !two && !a.whole_keys) err = INFINITY;
        lo = ordered(value - err);
        hi = ordered(value + err);
        if (!(err < INFINITY)) {
            lo = 32u;
            hi = 0xffffffffu;
        }
    } else if (live && group < a.n_group) {
        // beyond the range: no choice above `far` (values up to 2^23 + 1/2 round to 0, and
        // another 1/2 for the float that it is formed from), and one or two of them in the value
        const float far = __fadd_ru(__fadd_ru(top, -8388606.0f * (1.0f / a.steps)), error);
        lo = 32u;
        hi = ordered(!a.sums    ? far
                     : a.biased ? fmaxf(far, 2.0f * far)
                                : 2.0f * (fast_score(far, a, m, inv) + score_error(a, inv)));
    }
    int above = 0, maybe = 0;  // groups surely, and possibly, above this one
    for (int g = 0; g < a.n_group; ++g) {
        const uint32_t ol = __shfl_sync(kAll, lo, base + g * a.group_lanes);
        const uint32_t oh = __shfl_sync(kAll, hi, base + g * a.group_lanes);
        const bool sure = ol > hi || (lo == hi && ol == oh && ol == lo && g < group);
        const bool not_below = oh >= lo && !(lo == hi && ol == oh && (ol != lo || g > group));
        above += sure;
        maybe += sure || (not_below && g != group);
    }
    const bool in = group < a.n_group;
    open = in && above < a.topk_group && maybe >= a.topk_group;
    return in && maybe < a.topk_group;
}

// The choice of a biased expert; a NaN (an unset place's bias, a NaN bias) reads -inf.
__device__ __forceinline__ float biased_choice(float l, float b, const Args& a, float m,
                                               float inv) {
    const float c = fmaxf(fast_score(l, a, m, inv) + b, -INFINITY);
    return l > -INFINITY ? c : -INFINITY;
}

// Three largest of two times three (b3 may be any bound of the others).
__device__ __forceinline__ void merge_top3(uint32_t& b1, uint32_t& b2, uint32_t& b3, uint32_t o1,
                                           uint32_t o2, uint32_t o3) {
    const uint32_t lo = min(b1, o1), second = max(b2, o2);
    b1 = max(b1, o1);
    b2 = max(lo, second);
    b3 = max(min(lo, second), max(b3, o3));
}

// Whether this lane's group stays (bit 0): `kept` says it unless the group is `open`; the open
// groups share the places that the kept ones leave, by the float64 values of their two best
// keys.  Bit 1: the group is not open, or these are surely its two best, because nothing
// else lies as high as the second and none is beyond the range.  `apart`: key
// values that may be the other way round.
template <typename L, int V>
__device__ __noinline__ int keep_group_double(const L* row, const Args& a,
                                              const float* bias, double m, uint32_t b1,
                                              uint32_t b2, uint32_t b3, uint32_t apart, int base,
                                              int group, bool kept, bool open) {
    double v = -INFINITY;
#pragma unroll 1
    for (int r = 0; r < 2; ++r) {
        const uint32_t key = r == 0 ? b1 : b2;
        if (!selectable(key, a)) break;
        const int i = number_of(key);
        const int at = place_of<V>(i, a);
        double c = (double)to_float(row[at]);
        if (a.biased || a.sums) c = score_double(c, a.sigmoid, m, 1.0);
        if (a.biased) c += (double)bias[at];
        v = r == 0 ? c : a.sums ? v + c : fmax(v, c);
    }
    const unsigned opens = __ballot_sync(kAll, open) >> base;
    const unsigned keeps = __ballot_sync(kAll, kept) >> base;
    int rank = 0;  // kept groups, and open ones above this one
#pragma unroll 1
    for (int g = 0; g < a.n_group; ++g) {
        const double o = __shfl_sync(kAll, v, base + g * a.group_lanes);
        const unsigned bit = 1u << (g * a.group_lanes);
        rank += (keeps & bit) != 0 || ((opens & bit) != 0 && (o > v || (o == v && g < group)));
    }
    const bool sure = (a.sigmoid || !a.biased) &&
                      (a.whole_keys || (a.group_size == 1 ? selectable(b1, a)
                                                          : selectable(b2, a) &&
                                            (b2 >> kNumberBits) - (b3 >> kNumberBits) > apart));
    return (kept || (open && rank < a.topk_group) ? 1 : 0) | (!open || sure ? 2 : 0);
}

// Selects a row's k experts from those whose keys do not lie below the k-th by more
// than `band` key values: their float64 choices, one a lane, by the whole warp.
// `row` and `bias` lie in shared memory in the lanes' order; `kept`: bit i / group_size * group_lanes is set if the group of expert i stays.
// Lane r < k gets the expert of slot r; false if there are more than 32, or fewer than k (the k
// slots' own keys are among them, so this says that the keys are not what they were).
template <typename L, int V>
__device__ __noinline__ bool select_close(const L* row, const Args& a,
                                          const float* bias, int lane, float top,
                                          uint32_t kth, uint32_t band, unsigned kept, int* list,
                                          int& mine) {
    if (kth <= band) return false;  // they reach beyond the range
    int count = 0;
#pragma unroll 2
    for (int i0 = 0; i0 < a.E; i0 += 32) {
        const int i = i0 + lane;
        bool in = false;
        if (i < a.E) {
            const int at = place_of<V>(i, a);
            float c = fmaxf(to_float(row[at]), -INFINITY);
            if (a.biased) c = biased_choice(c, bias[at], a, 0.0f, 1.0f);
            in = (make_key(c, top, a, i) >> kNumberBits) >= kth - band &&
                 ((kept >> (i / a.group_size * a.group_lanes)) & 1u);
        }
        const unsigned all = __ballot_sync(kAll, in);
        const int at = count + __popc(all & ((1u << lane) - 1u));
        if (in && at < 32) list[at] = i;
        count += __popc(all);
    }
    if (count > 32 || count < a.k) return false;
    __syncwarp();
    const int i = lane < count ? list[lane] : 0x7fffffff;
    double v = -INFINITY;
    if (lane < count) {
        const int at = place_of<V>(i, a);
        v = (double)to_float(row[at]);
        if (a.biased) v = score_double(v, true, 0.0, 1.0) + (double)bias[at];
    }
    int rank = 0;
#pragma unroll 1
    for (int r = 0; r < count; ++r) {
        const double o = __shfl_sync(kAll, v, r);
        const int oi = __shfl_sync(kAll, i, r);
        rank += o > v || (o == v && oi < i);
    }
    __syncwarp();
    if (lane < count) list[rank] = i;
    __syncwarp();
    mine = lane < a.k ? list[lane] : -1;
    __syncwarp();
    return true;
}

// Rows in work per warp: 32 / LPR, next to each other.
template <typename L, int LPR, int V, int KL, bool kGroups>
__global__ void __launch_bounds__(kForwardWarps * 32)
    route_kernel(const L* __restrict__ logits, const float* __restrict__ bias,
                 const uint8_t* __restrict__ mask, const __grid_constant__ Args a,
                 int32_t* __restrict__ idx, float* __restrict__ gate) {
    constexpr int kRows = 32 / LPR;
    constexpr int kPitch = LPR * V + 16 / (int)sizeof(L);  // rows start 4 banks apart
    __shared__ __align__(16) L s_rows[kForwardWarps][kRows * kPitch];
    __shared__ double s_choice[kForwardWarps][LPR * V < kScoredMaxE ? LPR * V : kScoredMaxE];
    __shared__ __align__(16) float s_bias[LPR * V];  // in the lanes' order
    grid_dependency_wait();
    if (a.biased) {
        for (int i = threadIdx.x; i < a.E; i += kForwardWarps * 32)
            s_bias[place_of<V>(i, a)] = __ldg(bias + i);
        __syncthreads();
    }
    const int lane = threadIdx.x & 31;
    const int sub = lane & (LPR - 1), base = lane - sub;  // lane of the row, its first lane
    L* rows = s_rows[threadIdx.x >> 5];
    const int t0 = ((int)blockIdx.x * kForwardWarps + (threadIdx.x >> 5)) * kRows;
    if (t0 >= a.T) return;
    const int t = t0 + lane / LPR;
    const bool routed = t < a.T && (!mask || __ldg(mask + t) != 0);

    // the lanes' values that no expert fills read -inf
    const int group = sub / a.group_lanes, part = sub - group * a.group_lanes;
    const int first = group * a.group_size + part * a.lane_size;
    const int count = group < a.n_group
                          ? max(0, min(a.lane_size, a.group_size - part * a.lane_size))
                          : 0;
    L* mine = rows + (lane / LPR) * kPitch + sub * V;
    if (count < V) {
        for (int j = count; j < V; ++j) mine[j] = (L)(-INFINITY);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (t0 + r < a.T)
            stage_row<L, V>(logits + (int64_t)(t0 + r) * a.E, a, lane, rows + r * kPitch);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();

    // this lane's logits, 16 bytes at a time in an order that differs from lane to lane, so
    // that the lanes' reads lie in different banks; value j is expert at(j)
    constexpr int kPer = 16 / (int)sizeof(L);  // values of a piece
    constexpr int kPieces = V / kPer > 0 ? V / kPer : 1;
    float l[V];
    const int turn = (sub * V / (kPer * 8)) & (kPieces - 1);
    auto at = [&](int j) {
        return V <= kPer ? first + j : first + ((j / kPer) ^ turn) * kPer + j % kPer;
    };
    if constexpr (V >= kPer) {
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            union {
                uint4 u;
                L v[kPer];
            } q;
            q.u = *reinterpret_cast<const uint4*>(mine + (c ^ turn) * kPer);
#pragma unroll
            for (int j = 0; j < kPer; ++j) l[c * kPer + j] = fmaxf(to_float(q.v[j]), -INFINITY);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = fmaxf(to_float(mine[j]), -INFINITY);
    }

    float m = 0.0f, sum = 1.0f;
    if (!a.sigmoid && (a.biased || a.sums || !a.renorm)) {
        m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
        m = row_max<LPR>(m);
        sum = row_sum<LPR>(tree_sum<V>([&](int j) {
            return l[j] > -INFINITY ? fast_score(l[j], a, m, 1.0f) : 0.0f;
        }));
    }
    const float inv = a.sigmoid ? 1.0f : __fdividef(1.0f, sum);

    if (a.biased) {
        const float* b = s_bias + sub * V - first;
        if constexpr (V >= 4) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 q = *reinterpret_cast<const float4*>(b + at(j));
                l[j] = biased_choice(l[j], q.x, a, m, inv);
                l[j + 1] = biased_choice(l[j + 1], q.y, a, m, inv);
                l[j + 2] = biased_choice(l[j + 2], q.z, a, m, inv);
                l[j + 3] = biased_choice(l[j + 3], q.w, a, m, inv);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) l[j] = biased_choice(l[j], b[at(j)], a, m, inv);
        }
    }
    float top = 0.0f;   // the row's largest choice
    bool live = false;  // this lane has one
    if (!a.whole_keys) {
        top = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) top = fmaxf(top, l[j]);
        live = top > -INFINITY;
        top = row_max<LPR>(top);
    }
    uint32_t key[V > KL ? V : KL];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = make_key(l[j], top, a, at(j));
    // error of a choice as a key of distance `d` from the top tells it: half a step, the
    // roundings of the distance and of score + bias, and the score's error
    const float step = 1.0f / a.steps;
    auto key_error = [&](float d) {
        if (a.whole_keys) return 0.0f;
        return 0.5f * step + kRound * d +
               (a.biased ? score_error(a, inv) + kRound * (fabsf(top) + d) : 0.0f);
    };
    uint32_t best[KL], out = 0u;
    constexpr int kFirst = V < KL ? V : KL;
    sort_descending<kFirst>(key);
#pragma unroll
    for (int j = 0; j < KL; ++j) best[j] = j < kFirst ? key[j] : 0u;
#pragma unroll
    for (int b = KL; b < V; b += KL) {
        sort_descending<KL>(key + b);
        merge_best<KL>(best, key + b, out);
    }
    // values that may be the other way round, `below` the lower of two keys: logits' keys keep
    // the order, biased ones are off
    auto apart = [&](uint32_t below) {
        const float far = (float)(0x7fffffu - (below >> kNumberBits)) * step;
        return a.biased ? (uint32_t)(2.0f * key_error(far) * a.steps) + 1u : 0u;
    };
    const L* row = rows + (lane / LPR) * kPitch;
    bool full = false, kept = true;
    if constexpr (kGroups) {
        uint32_t b1 = best[0], b2 = best[1];
        for (int off = 1; off < a.group_lanes; off <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kAll, b1, off);
            const uint32_t o2 = __shfl_xor_sync(kAll, b2, off);
            merge_top2(b1, b2, o1, o2);
        }
        const unsigned lives = __ballot_sync(kAll, live) >> (lane - part);  // of this group on
        const bool group_live = (lives & (0xffffffffu >> (32 - a.group_lanes))) != 0;
        kept = keep_group<LPR>(b1, b2, group_live, a, top, m, inv, key_error(8388608.0f * step),
                               base, group, full);
        if (__builtin_expect(__any_sync(kAll, full && routed), 0)) {
            uint32_t b3 = best[2];
            b1 = best[0];
            b2 = best[1];
#pragma unroll 1
            for (int off = 1; off < a.group_lanes; off <<= 1) {
                const uint32_t o1 = __shfl_xor_sync(kAll, b1, off);
                const uint32_t o2 = __shfl_xor_sync(kAll, b2, off);
                const uint32_t o3 = __shfl_xor_sync(kAll, b3, off);
                merge_top3(b1, b2, b3, o1, o2, o3);
            }
            const int bits = keep_group_double<L, V>(row, a, s_bias, (double)m, b1, b2, b3, apart(b3),
                                                     base, group, kept, full);
            const unsigned of_row = LPR == 32 ? kAll : ((1u << (LPR & 31)) - 1u) << base;
            const unsigned unsure = __ballot_sync(kAll, full) & of_row;  // by all lanes
            const unsigned exact = __ballot_sync(kAll, (bits & 2) != 0) & of_row;
            if (unsure != 0) {
                full = exact != of_row;
                kept = (bits & 1) != 0;
            }
        }
        if (!kept) {
#pragma unroll
            for (int j = 0; j < KL; ++j) best[j] = 0u;
            out = 0u;
        }
    }
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) {
        uint32_t other[KL];
#pragma unroll
        for (int j = 0; j < KL; ++j) other[j] = __shfl_xor_sync(kAll, best[j], off);
        out = max(out, __shfl_xor_sync(kAll, out, off));
        merge_best<KL>(best, other, out);
    }
    // slot `sub` of the row and the key behind it
    uint32_t slot = 0u, next = 0u;
#pragma unroll
    for (int j = 0; j < KL; ++j)
        if (sub == j) {
            slot = best[j];
            next = j + 1 < KL ? best[j + 1 < KL ? j + 1 : j] : out;
        }
    bool again = false, empty = false;
    if (sub < a.k) {
        if (a.whole_keys) {
            // exact: equal logits go by number
        } else if (!selectable(slot, a)) {
            empty = top > -INFINITY;  // no live expert is left for it, or one beyond the range
        } else {
            again = (slot >> kNumberBits) - (next >> kNumberBits) <= apart(next);
        }
    }
    int chosen = sub < a.k && selectable(slot, a) ? number_of(slot) : -1;

    if (__builtin_expect(__any_sync(kAll, (full || again || empty) && routed), 0)) {
        if (__any_sync(kAll, empty && routed)) {
            bool beyond = false;  // this lane has a live expert whose key says nothing
#pragma unroll 1
            for (int j = 0; j < V; ++j) {
                float c = fmaxf(to_float(mine[j]), -INFINITY);
                if (a.biased) c = biased_choice(c, s_bias[sub * V + j], a, m, inv);
                beyond |= kept && c > -INFINITY && !selectable(make_key(c, top, a, 0), a);
            }
            const unsigned of_row = LPR == 32 ? kAll : ((1u << (LPR & 31)) - 1u) << base;
            const unsigned beyonds = __ballot_sync(kAll, beyond) & of_row;
            full |= empty && beyonds != 0;
        }
        unsigned fulls = __ballot_sync(kAll, full && routed), close = 0u;
        if (a.sigmoid || !a.biased) {
            // second attempt, for all rows of the warp alike
            const bool live = selectable(slot, a);
            const int i = live ? number_of(slot) : 0x7fffffff;
            double v = -INFINITY;
            if (live) {
                const int at = place_of<V>(i, a);
                v = (double)to_float(row[at]);
                if (a.biased) v = score_double(v, true, 0.0, 1.0) + (double)s_bias[at];
            }
            int rank = 0;
#pragma unroll
            for (int r = 0; r < KL; ++r) {
                const double o = __shfl_sync(kAll, v, base + r);
                const int oi = __shfl_sync(kAll, i, base + r);
                rank += o > v || (o == v && oi < i);
            }
            if (!live) rank = 64;
            int ranked = -1;
#pragma unroll
            for (int r = 0; r < KL; ++r) {
                const int of = __shfl_sync(kAll, rank, base + r);
                const int oi = __shfl_sync(kAll, i, base + r);
                if (of == sub && sub < a.k) ranked = oi;
            }
            chosen = ranked;
            // `out` may be as high as the k-th, and more with it
            close = __ballot_sync(kAll, routed && !a.whole_keys && rank == a.k - 1 &&
                                            (slot >> kNumberBits) - (out >> kNumberBits) <= apart(out));
        } else {
            fulls |= __ballot_sync(kAll, again && routed);
        }
        const unsigned keeps = __ballot_sync(kAll, kept);
        const uint32_t wide = apart(slot);
        double* choices = s_choice[threadIdx.x >> 5];
#pragma unroll 1
        for (int r = 0; r < kRows; ++r) {  // row by row
            const unsigned of_row = LPR == 32 ? kAll : ((1u << (LPR & 31)) - 1u) << (r * LPR);
            if (!((fulls | close) & of_row)) continue;
            int got = -1;
            bool done = false;
            if (!(fulls & of_row)) {
                // the lower of two keys raises the values that may be swapped by a 2^-22th of
                // their distance, 2 at most
                const uint32_t kth = __shfl_sync(kAll, slot, r * LPR + a.k - 1) >> kNumberBits;
                const uint32_t band = __shfl_sync(kAll, wide, r * LPR + a.k - 1);
                const float row_top = __shfl_sync(kAll, top, r * LPR);
                done = select_close<L, V>(rows + r * kPitch, a, s_bias, lane, row_top, kth,
                                          a.biased ? band + 2u : 0u, keeps >> (r * LPR),
                                          reinterpret_cast<int*>(choices), got);
            }
            if (!done)
                got = select_double<L>(logits + (int64_t)(t0 + r) * a.E, a, bias, lane, choices);
            const int to = __shfl_sync(kAll, got, sub);
            if (lane / LPR == r) chosen = sub < a.k ? to : -1;
        }
    }

    float w = 0.0f;
    if (!routed) chosen = -1;
    const bool taken = chosen >= 0;
    const float lv =
        taken ? to_float(row[place_of<V>(chosen, a)]) : -INFINITY;
    if (a.renorm) {
        // the largest selected logit: slot 0's, unless a bias moved it
        const float M = a.biased ? row_max<LPR>(lv) : __shfl_sync(kAll, lv, base);
        if (taken) w = a.sigmoid ? sigmoid_ratio(lv, M) : exp_below(lv, M);
        float total = w;  // over the slots, in pairs
        for (int off = a.slots >> 1; off > 0; off >>= 1)
            total += __shfl_xor_sync(kAll, total, off);
        w = taken ? __fdiv_rn(w, total) : 0.0f;
    } else if (taken) {
        w = a.sigmoid ? sigmoid(lv) : __fdiv_rn(exp_below(lv, m), sum);
    }
    if (t < a.T && sub < a.k) {
        idx[(int64_t)t * a.k + sub] = chosen;
        gate[(int64_t)t * a.k + sub] = w * a.scale;
    }
}

// ------------------------------------------------------------------ gradient
// With u_r = scale * dgate_r over the filled slots r, i(r) their experts:
//   softmax, not renormalised   dl_i = s_i (sum_{r: i(r) = i} u_r - sum_r u_r s_{i(r)})
//   otherwise, w the gates before the scale (v_r = u_r - sum u w if renormalised,
//   else u_r)                   dl_i = sum_{r: i(r) = i} v_r w_r           softmax
//                               dl_i = sum_{r: i(r) = i} v_r w_r (1 - s_i)  sigmoid
// and 0 for every other expert.  The bias only steers the selection: it has no
// gradient.  A row is put together in shared memory and leaves as whole vectors.
template <typename L, int V>
__device__ __forceinline__ void store_row(L* row, const Args& a, int i0, const float (&g)[V]) {
    typedef RowVec<L, V> R;
    R out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (sizeof(L) == 2)
            out.v[j] = __float2bfloat16_rn(g[j]);
        else
            out.v[j] = g[j];
    }
    if (a.vec && i0 + V <= a.E) {
        typename R::type* dst = reinterpret_cast<typename R::type*>(row + i0);
#pragma unroll
        for (int j = 0; j < R::kUnits; ++j) dst[j] = out.u[j];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (i0 + j < a.E) row[i0 + j] = out.v[j];
    }
}

template <typename L, int V>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(V))
    backward_kernel(const L* __restrict__ logits, const int32_t* __restrict__ idx,
                    const float* __restrict__ dgate, const Args a, L* __restrict__ dlogits) {
    __shared__ float s_row[kWarps][32 * V];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int i0 = lane * V;
    const int step = (int)gridDim.x * kWarps;
    int t = (int)blockIdx.x * kWarps + (threadIdx.x >> 5);
    float* buf = s_row[threadIdx.x >> 5];
    const bool dense = !a.sigmoid && !a.renorm;
    // the next row's experts, their gradients and (dense) its logits load a row ahead
    int ahead_i = -1;
    float ahead_u = 0.0f;
    RowVec<L, V> ahead = {};
    const L* row = logits + (int64_t)t * a.E;
    const int64_t row_step = (int64_t)step * a.E;
    const int32_t* ip = idx + (int64_t)t * a.k + lane;
    const float* gp = dgate + (int64_t)t * a.k + lane;
    L* out = dlogits + (int64_t)t * a.E;
    auto fetch = [&](const L* from) {
        if (lane < a.k) {
            ahead_i = __ldg(ip);
            ahead_u = __ldg(gp);
        }
        if (dense) load_row(from, a, i0, ahead);
        ip += (int64_t)step * a.k;
        gp += (int64_t)step * a.k;
    };
    if (t < a.T) fetch(row);
    for (; t < a.T; t += step, row += row_step, out += row_step) {
        const int i = ahead_i >= 0 && ahead_i < a.E ? ahead_i : -1;
        float u = i >= 0 ? ahead_u * a.scale : 0.0f;
        const float lv = i >= 0 ? to_float(__ldg(row + i)) : -INFINITY;
        float l[V];
        if (dense) to_floats(ahead, l);
        if (t + step < a.T) fetch(row + row_step);
        const bool live = i >= 0 && lv > -INFINITY;
        float g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = 0.0f;
        if (__any_sync(kAll, live)) {
            float v = 0.0f;  // this slot's part of the gradient of its expert's logit
            if (dense) {
                float m, sum;
                softmax_stats<float, V>(l, m, sum);
                const float inv = __fdiv_rn(1.0f, sum);
                const float s = live ? exp_below(lv, m) * inv : 0.0f;
                v = live ? u * s : 0.0f;
                const float total = warp_sum(v);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    g[j] = l[j] > -INFINITY ? -(exp_below(l[j], m) * inv) * total : 0.0f;
            } else {
                float w = 0.0f;
                if (a.renorm) {
                    const float M = warp_max_float(live ? lv : -INFINITY);
                    if (live) w = a.sigmoid ? sigmoid_ratio(lv, M) : exp_below(lv, M);
                    w = __fdiv_rn(w, warp_sum(w));
                    u -= warp_sum(live ? u * w : 0.0f);
                } else if (live) {
                    w = sigmoid(lv);
                }
                // 1 - sigmoid(l) = sigmoid(-l), without cancellation
                if (live) v = u * w * (a.sigmoid ? sigmoid(-lv) : 1.0f);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) buf[i0 + j] = g[j];
            __syncwarp();
            // an expert named by several slots gets their sum, in slot order, from the first
            const unsigned same = __match_any_sync(kAll, live ? i : -1 - lane);
            const bool first = live && (same & ((1u << lane) - 1u)) == 0;
            if (__any_sync(kAll, live && same != (1u << lane))) {
                float add = 0.0f;
                for (int r = 0; r < a.k; ++r) {
                    const float o = __shfl_sync(kAll, v, r);
                    if ((same >> r) & 1u) add += o;
                }
                v = add;
            }
            if (first) buf[i] += v;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = buf[i0 + j];
            __syncwarp();
        }
        store_row<L, V>(out, a, i0, g);
    }
}

// ------------------------------------------------------------------ host side
inline int pow2_ceil(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

inline int unit_of(int bytes) { return bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : bytes % 4 == 0 ? 4 : 2; }

inline Args make_args(const moe_shape& s, const moe_scoring& r, bool has_bias, int esize) {
    Args a{};
    a.T = s.T;
    a.E = s.E;
    a.k = s.k;
    a.sigmoid = r.score == MOE_SCORE_SIGMOID;
    a.renorm = r.renorm != 0;
    a.n_group = r.n_group;
    a.group_size = s.E / r.n_group;
    a.topk_group = r.topk_group;
    a.biased = has_bias;
    a.sums = r.n_group > 1 && r.group_top > 1;
    a.whole_keys = esize == 2 && !has_bias;
    a.steps = 8388608.0f / (has_bias ? 4.0f : 32.0f);
    a.slots = pow2_ceil(s.k);
    a.unit = unit_of(s.E * esize);
    a.scale = r.scale;
    return a;
}

// Lanes to a row and values to a lane: as few lanes as hold the slots, a power of two of
// them for each group and no more than 32 values.
struct Fit {
    int lanes, values;
};
inline Fit fit(const moe_shape& s, Args& a) {
    const int groups = pow2_ceil(a.n_group);
    // a batch that leaves schedulers idle: a warp a row, which is the shortest chain
    const int64_t warps = (int64_t)device_sm_count() * 4;
    int lanes = std::max(s.T <= warps && s.E > 32 ? 32 : s.k <= 8 ? 8 : 16, groups);
    int per = 0, values = 0;
    for (;; lanes *= 2) {
        a.group_lanes = lanes / groups;
        per = (a.group_size + a.group_lanes - 1) / a.group_lanes;
        values = per <= 1 && lanes == 8 ? 1 : per <= 4 ? 4 : per <= 8 && lanes == 8 ? 8
                 : per <= 16 ? 16 : 32;
        if (per <= 32 || lanes == 32) break;
    }
    // lanes filled to the last: the experts' places then keep their order in the softmax's sum
    a.lane_size = values;
    a.aligned = a.n_group == 1 || a.group_size == values * a.group_lanes;
    return Fit{lanes, values};
}

template <typename L, int LPR, int V, int KL>
int launch_route(const moe_shape& s, const Args& a, const void* logits, const float* bias,
                 const uint8_t* mask, int32_t* idx, float* gate, cudaStream_t st) {
    constexpr int kRows = kForwardWarps * 32 / LPR;
    auto kern = route_kernel<L, LPR, V, KL, false>;
    if constexpr (KL > 2) {
        if (a.n_group > 1) kern = route_kernel<L, LPR, V, KL, true>;
    }
    return launch_pdl(kern, dim3((s.T + kRows - 1) / kRows), dim3(kForwardWarps * 32), 0, st,
                      static_cast<const L*>(logits), bias, mask, a, idx, gate) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <typename L, int KL, typename... Rest>
int route_lanes(const Fit& f, Rest... rest) {
    if constexpr (KL <= 8) {
        if (f.lanes == 8) {
            if (f.values == 1) return launch_route<L, 8, 1, KL>(rest...);
            if (f.values == 4) return launch_route<L, 8, 4, KL>(rest...);
            if (f.values == 8) return launch_route<L, 8, 8, KL>(rest...);
            if (f.values == 16) return launch_route<L, 8, 16, KL>(rest...);
            return launch_route<L, 8, 32, KL>(rest...);
        }
    }
    if (f.lanes == 16) {
        if (f.values == 4) return launch_route<L, 16, 4, KL>(rest...);
        if (f.values == 16) return launch_route<L, 16, 16, KL>(rest...);
        return launch_route<L, 16, 32, KL>(rest...);
    }
    if (f.values == 4) return launch_route<L, 32, 4, KL>(rest...);
    if (f.values == 16) return launch_route<L, 32, 16, KL>(rest...);
    return launch_route<L, 32, 32, KL>(rest...);
}

// Blocks of kWarps rows each, no more than fit at once (the warps then loop).
inline unsigned blocks_for(int T, int V) {
    return (unsigned)std::min<int64_t>(((int64_t)T + kWarps - 1) / kWarps,
                                       (int64_t)device_sm_count() * blocks_per_sm(V));
}

template <typename L, int V>
int launch_backward(const moe_shape& s, const moe_scoring& r, const void* logits,
                    const int32_t* idx, const float* dgate, void* dlogits, cudaStream_t st) {
    Args a = make_args(s, r, false, sizeof(L));
    a.vec = a.unit >= std::min(16, V * (int)sizeof(L));
    return launch_pdl(backward_kernel<L, V>, dim3(blocks_for(s.T, V)), dim3(kWarps * 32),
                      0, st, static_cast<const L*>(logits), idx, dgate, a,
                      static_cast<L*>(dlogits)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <typename L>
int route_for(const moe_shape& s, const moe_scoring& r, const void* logits, const float* bias,
              const uint8_t* mask, int32_t* idx, float* gate, cudaStream_t st) {
    Args a = make_args(s, r, bias != nullptr, sizeof(L));
    const Fit f = fit(s, a);
    if (s.k <= 2 && r.n_group == 1)
        return route_lanes<L, 2>(f, s, a, logits, bias, mask, idx, gate, st);
    if (s.k <= 8) return route_lanes<L, 8>(f, s, a, logits, bias, mask, idx, gate, st);
    return route_lanes<L, 16>(f, s, a, logits, bias, mask, idx, gate, st);
}

template <typename L>
int backward_for(const moe_shape& s, const moe_scoring& r, const void* logits, const int32_t* idx,
                 const float* dgate, void* dlogits, cudaStream_t st) {
    if (s.E <= 32) return launch_backward<L, 1>(s, r, logits, idx, dgate, dlogits, st);
    if (s.E <= 64) return launch_backward<L, 2>(s, r, logits, idx, dgate, dlogits, st);
    if (s.E <= 128) return launch_backward<L, 4>(s, r, logits, idx, dgate, dlogits, st);
    if (s.E <= 256) return launch_backward<L, 8>(s, r, logits, idx, dgate, dlogits, st);
    return launch_backward<L, 16>(s, r, logits, idx, dgate, dlogits, st);
}

}  // namespace scored
}  // namespace moe
