// route_scored.cu -- routing on given logits: scores, selection bias, groups,
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
// One warp works on one row.  Lane L holds the V consecutive experts from
// L * V, and choices are compared as unsigned integers in the floats' order, which
// makes the largest of 32 lanes one redux instruction.
//
// Three attempts, each taken only where the one before could not tell two experts
// (or the last kept and first dropped group) apart:
//  1. packed: the low bits of a choice's key give way to the expert's number, so that
//     one redux yields both and no lane has to be asked who won; each lane sorts its V
//     keys once, and a selected one is shifted out.  Rows whose neighbours in the selected
//     order lie within the lost bits and the error of a float32 score go on (under 1 in
//     100 of 256 biased sigmoids; bf16 logits without a bias lose no bits).
//  2. candidates: four more of them are taken, and each lane forms one candidate's
//     choice in float64; ranking them decides, unless the last may lie as high as
//     the k-th.
//  3. all choices in float64: where the groups are too close, or the second
//     attempt does not decide, or a biased softmax needs its sum in float64.
// So the selection is that of float64 scores.
//
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "route_scored.cuh"

namespace moe {
namespace scored {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;  // rows in work per block
// Blocks an SM holds: as many as V values a lane leave registers for.
constexpr int blocks_per_sm(int V) { return V <= 2 ? 6 : V == 4 ? 5 : V == 8 ? 4 : 2; }
constexpr int kExtra = 4;  // candidates beyond the first one left out (second attempt)

struct Args {
    int T, E, k;
    int sigmoid, renorm;
    int n_group, group_size, topk_group, group_top;
    int group_lanes;  // lanes of one group when groups are whole lanes, a power of two; else 0
    int biased;       // choices are scores plus a bias; otherwise logits order them
    int sums;         // groups are valued by a sum of two choices
    int whole_keys;   // without a bias, keys leave their low bits zero (bf16 logits)
    float lost;       // what a packed key may lose, relative to its value
    int slots;        // k, rounded up to a power of two
    int vec;          // rows can be read in vectors
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
__device__ __forceinline__ double exp_below(double l, double m) {
    return l == m ? 1.0 : exp(l - m);
}
__device__ __forceinline__ float sigmoid(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }
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

// ------------------------------------------------------------------ third attempt
// Selects the row's k experts: lane r < k returns the expert of slot r, or -1.  All
// choices in float64, whole keys; without a bias the logits order the experts.
template <int V>
__device__ __noinline__ int select_double(const float (&l)[V], const Args& a, const float* bias,
                                          int lane) {
    typedef unsigned long long K;
    const int i0 = lane * V;
    double m = 0.0, inv = 1.0;
    if (!a.sigmoid && (a.biased || a.sums)) {
        double sum;
        softmax_stats<double, V>(l, m, sum);
        inv = 1.0 / sum;
    }
    auto score = [&](double x) { return a.sigmoid ? sigmoid(x) : exp_below(x, m) * inv; };
    K key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        key[j] = 0;
        if (l[j] > -INFINITY) {
            double c = (double)l[j];
            if (a.biased) c = score(c) + (double)__ldg(bias + i0 + j);
            if (c > -INFINITY) key[j] = ordered(c);
        }
    }
    if (a.n_group > 1) {
        K value = 0;
        for (int g = 0; g < a.n_group; ++g) {
            K t1 = 0, t2 = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const unsigned in = (unsigned)(i0 + j - g * a.group_size);
                merge_top2(t1, t2, in < (unsigned)a.group_size ? key[j] : (K)0, (K)0);
            }
            const K m1 = warp_max(t1);
            const bool many = __popc(__ballot_sync(kAll, t1 == m1)) > 1;
            const K m2 = warp_max(t1 == m1 && !many ? t2 : t1);
            if (lane == g && m1 != 0) {
                value = m1;
                if (a.sums) {
                    const double v1 = from_key(m1), v2 = m2 != 0 ? from_key(m2) : 0.0;
                    value = ordered(a.biased ? v1 + v2
                                             : score(v1) + (m2 != 0 ? score(v2) : 0.0));
                }
            }
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const K o = __shfl_sync(kAll, value, g);
            rank += o > value || (o == value && g < lane);
        }
        const unsigned keep = __ballot_sync(kAll, lane < a.n_group && rank < a.topk_group);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (i0 + j < a.E && !((keep >> ((i0 + j) / a.group_size)) & 1u)) key[j] = 0;
    }
    int mine = -1;
    for (int r = 0; r < a.k; ++r) {
        K head = 0;
        int at = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (key[j] > head) {
                head = key[j];
                at = j;
            }
        const K best = warp_max(head);
        if (best == 0) break;
        const int owner = __ffs(__ballot_sync(kAll, head == best)) - 1;
        const int chosen = __shfl_sync(kAll, i0 + at, owner);
        if (lane == r) mine = chosen;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (i0 + j == chosen) key[j] = 0;
    }
    return mine;
}

// ------------------------------------------------------------------ packed attempt
template <int V>
struct Packed {
    static constexpr int kBits = V == 1 ? 5 : V == 2 ? 6 : V == 4 ? 7 : V == 8 ? 8 : 9;
    static constexpr uint32_t kLow = (1u << kBits) - 1u;
};

// Descending, by Batcher's odd-even merge network.
template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2) {
#pragma unroll
        for (int q = p; q >= 1; q /= 2) {
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q) {
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(k[i + j], k[i + j + q]);
                        k[i + j + q] = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                    }
                }
            }
        }
    }
}

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

// A float32 score, off by less than score_error(): the exponent's rounding moves exp by
// |l| 2^-24 (and s (1 - s) |l| by less than 0.3 2^-24), the others are a few ulps.
__device__ __forceinline__ float fast_score(float l, const Args& a, float m, float inv) {
    constexpr float kLog2e = 1.4426950408889634f;
    if (a.sigmoid) return rcp_fast(1.0f + exp2_fast(-l * kLog2e));
    return l == m ? inv : exp2_fast((l - m) * kLog2e) * inv;
}

// Error bound of a score and of the addition of a bias to it (relative to the choice
// it gives, where that is larger): 16 ulps of 1, or of the row's largest softmax score inv
// and 48 more for the rounding of its sum of V + 5 terms.
__device__ __forceinline__ float score_error(const Args& a, float inv) {
    return a.sigmoid ? 1.9073486e-6f : 7.6293945e-6f * inv;
}
constexpr float kAddError = 2.3841858e-7f;

// Which groups stay (bit g).  b1, b2: the two best keys of group `lane`.  `full`: the
// last group kept and the first dropped cannot be told apart.
template <int V>
__device__ __forceinline__ unsigned keep_groups(uint32_t b1, uint32_t b2, const Args& a, float m,
                                                float inv, int lane, bool& full) {
    constexpr uint32_t kLow = Packed<V>::kLow;
    const float lost = a.lost;
    const bool in = lane < a.n_group;
    float value = 0.0f, err = 0.0f;
    if (in && b1 != 0u) {
        const float c1 = from_key(b1 & ~kLow), c2 = b2 != 0u ? from_key(b2 & ~kLow) : 0.0f;
        value = c1;
        err = lost * fabsf(c1);
        if (a.sums) {
            if (a.biased) {
                value = c1 + c2;
                err += lost * fabsf(c2);
            } else {  // a score moves by less than its slope times what a logit lost
                const float s1 = fast_score(c1, a, m, inv);
                const float s2 = b2 != 0u ? fast_score(c2, a, m, inv) : 0.0f;
                value = s1 + s2;
                err = 1.01f * lost * (fabsf(c1) * (a.sigmoid ? s1 * (1.0f - s1) : s1) +
                                      fabsf(c2) * (a.sigmoid ? s2 * (1.0f - s2) : s2));
            }
        }
        if (a.biased || a.sums)
            err += 2.0f * score_error(a, inv) + kAddError * (fabsf(c1) + fabsf(c2));
    }
    const uint32_t vkey = in && b1 != 0u ? ordered(value) : 0u;
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
        const uint32_t o = __shfl_sync(kAll, vkey, g);
        rank += o > vkey || (o == vkey && g < lane);
    }
    const bool kept = in && rank < a.topk_group;
    const uint32_t out = __reduce_max_sync(kAll, in && !kept ? vkey : 0u);
    const uint32_t last = __reduce_min_sync(kAll, kept && vkey != 0u ? vkey : 0xffffffffu);
    const float worst = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(err)));
    // bf16 logits without a bias: errors of zero, and equal values go by number
    if (out != 0u && !(from_key(last) - from_key(out) > 2.0f * worst))
        full |= a.biased || a.sums || !a.whole_keys;
    return __ballot_sync(kAll, kept);
}

// The second attempt.  `mine`: the packed key of candidate `lane` (0: none), k + 1 +
// kExtra of them in descending order.  False if it does not decide.
template <int V, typename L>
__device__ __forceinline__ bool select_candidates(uint32_t mine, const Args& a, const L* row,
                                                  const float* __restrict__ bias, int lane,
                                                  int& chosen) {
    constexpr uint32_t kLow = Packed<V>::kLow;
    const int n = a.k + 1 + kExtra;
    const bool live = lane < n && mine != 0u;
    const int i = live ? (int)(kLow - (mine & kLow)) : 0x7fffffff;
    double v = -INFINITY;
    if (live) {
        v = (double)to_float(__ldg(row + i));
        if (a.biased) v = sigmoid(v) + (double)__ldg(bias + i);
    }
    int rank = 0;
    for (int r = 0; r < n; ++r) {
        const double o = __shfl_sync(kAll, v, r);
        const int oi = __shfl_sync(kAll, i, r);
        rank += o > v || (o == v && oi < i);
    }
    if (!live) rank = 32;
    chosen = -1;
    for (int r = 0; r < n; ++r) {
        const int of = __shfl_sync(kAll, rank, r);
        const int oi = __shfl_sync(kAll, i, r);
        if (of == lane && lane < a.k) chosen = oi;
    }
    // every expert that is no candidate lies below the last candidate's key
    const uint32_t last = __shfl_sync(kAll, mine, n - 1);
    const unsigned kth = __ballot_sync(kAll, rank == a.k - 1);
    if (last == 0u || kth == 0u) return true;
    const float c = from_key(last & ~kLow);
    const double top = (double)c + (double)(a.lost * fabsf(c)) +
                       (a.biased ? (double)score_error(a, 1.0f) : 0.0);
    return __shfl_sync(kAll, v, __ffs(kth) - 1) > top;
}

// Selects the row's k experts: lane r < k returns the expert of slot r, or -1.  The
// keys' low bits are the expert's number counted from the top (a lower expert has
// the larger key).
template <int V, typename L>
__device__ __forceinline__ int select(const float (&l)[V], const Args& a, const L* row,
                                      const float* __restrict__ bias, const float (&bv)[V],
                                      float m, float sum, int lane) {
    constexpr int kBits = Packed<V>::kBits;
    constexpr uint32_t kLow = Packed<V>::kLow;
    const int i0 = lane * V;
    const float inv = a.sigmoid ? 1.0f : __fdiv_rn(1.0f, sum);
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float c = l[j];
        if (a.biased && c > -INFINITY) c = fast_score(c, a, m, inv) + bv[j];
        key[j] = c > -INFINITY ? (ordered(c) & ~kLow) | (kLow - (uint32_t)(i0 + j)) : 0u;
    }
    bool full = false;
    if (a.n_group > 1 && !a.group_lanes) {
        uint32_t b1 = 0u, b2 = 0u;
        for (int g = 0; g < a.n_group; ++g) {
            uint32_t t1 = 0u, t2 = 0u;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const unsigned in = (unsigned)(i0 + j - g * a.group_size);
                merge_top2(t1, t2, in < (unsigned)a.group_size ? key[j] : 0u, 0u);
            }
            const uint32_t m1 = __reduce_max_sync(kAll, t1);
            const uint32_t m2 = __reduce_max_sync(kAll, t1 == m1 ? t2 : t1);
            if (lane == g) {
                b1 = m1;
                b2 = m2;
            }
        }
        const unsigned keep = keep_groups<V>(b1, b2, a, m, inv, lane, full);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (i0 + j < a.E && !((keep >> ((i0 + j) / a.group_size)) & 1u)) key[j] = 0u;
    }
    sort_descending(key);
    if (a.n_group > 1 && a.group_lanes) {
        uint32_t b1 = key[0], b2 = V > 1 ? key[V > 1 ? 1 : 0] : 0u;
        for (int off = 1; off < a.group_lanes; off <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kAll, b1, off);
            const uint32_t o2 = __shfl_xor_sync(kAll, b2, off);
            merge_top2(b1, b2, o1, o2);
        }
        const int src = (lane < a.n_group ? lane : 0) * a.group_lanes;
        b1 = __shfl_sync(kAll, b1, src);
        b2 = __shfl_sync(kAll, b2, src);
        const unsigned keep = keep_groups<V>(b1, b2, a, m, inv, lane, full);
        if (!((keep >> (lane / a.group_lanes)) & 1u)) key[0] = 0u;  // nothing of this lane
    }
    uint32_t mine = 0u;
    auto take = [&](int r) {
        const uint32_t best = __reduce_max_sync(kAll, key[0]);
        if (lane == r) mine = best;
        if (key[0] == best) {
#pragma unroll
            for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1];
            key[V - 1] = 0u;
        }
    };
    for (int r = 0; r <= a.k; ++r) take(r);
    bool again = false;
    const uint32_t next = __shfl_down_sync(kAll, mine, 1);
    if (lane < a.k && next != 0u) {
        if (a.biased) {
            const float hi = from_key(mine & ~kLow), lo = from_key(next & ~kLow);
            again = !(hi - lo > a.lost * fabsf(lo) + 2.0f * score_error(a, inv) +
                                    kAddError * (fabsf(hi) + fabsf(lo)));
        } else {
            again = !a.whole_keys && (mine >> kBits) == (next >> kBits);
        }
    }
    full = __any_sync(kAll, full);
    int chosen = lane < a.k && mine != 0u ? (int)(kLow - (mine & kLow)) : -1;
    if (!full && __any_sync(kAll, again)) {
        full = true;
        if (a.sigmoid || !a.biased) {
            for (int r = a.k + 1; r <= a.k + kExtra; ++r) take(r);
            full = !select_candidates<V>(mine, a, row, bias, lane, chosen);
        }
    }
    if (full) chosen = select_double<V>(l, a, bias, lane);
    return chosen;
}

// Weight of a selected expert before any division by the sum.  With
// renormalisation only ratios count: the sigmoid is then taken relative to
// exp(min(M, 0)), M the largest selected logit, so that it cannot underflow
// however negative all of them are.
__device__ __forceinline__ float sigmoid_ratio(float l, float M) {
    const float e = expf(-fabsf(l));
    const float top = l >= 0.0f ? 1.0f : (M < 0.0f ? exp_below(l, M) : e);
    return __fdividef(top, 1.0f + e);
}

// A warp takes rows t, t + warps, ...; the next row's logits load while it works on one.
template <typename L, int V>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(V))
    route_kernel(const L* __restrict__ logits, const float* __restrict__ bias,
                 const uint8_t* __restrict__ mask, const Args a, int32_t* __restrict__ idx,
                 float* __restrict__ gate) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int i0 = lane * V;
    const int step = (int)gridDim.x * kWarps;
    int t = (int)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    float bv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) bv[j] = a.biased && i0 + j < a.E ? __ldg(bias + i0 + j) : 0.0f;
    const L* row = logits + (int64_t)t * a.E;
    const int64_t row_step = (int64_t)step * a.E;
    int64_t at = (int64_t)t * a.k + lane;
    RowVec<L, V> ahead;
    load_row(row, a, i0, ahead);
    int ahead_mask = mask ? __ldg(mask + t) : 1;
    while (true) {
        float l[V];
        to_floats(ahead, l);
        const bool routed = ahead_mask != 0, more = t + step < a.T;
        if (more) {
            load_row(row + row_step, a, i0, ahead);
            if (mask) ahead_mask = __ldg(mask + t + step);
        }
        int chosen = -1;
        float w = 0.0f;
        if (routed) {
            float m = 0.0f, sum = 1.0f;
            if (!a.sigmoid && (a.biased || a.sums || !a.renorm)) softmax_stats<float, V>(l, m, sum);
            chosen = select<V>(l, a, row, bias, bv, m, sum, lane);
            const bool taken = chosen >= 0;
            const float lv = taken ? to_float(__ldg(row + chosen)) : -INFINITY;
            if (a.renorm) {
                // the largest selected logit: slot 0's, unless a bias moved it
                const float M = a.biased ? warp_max_float(lv) : __shfl_sync(kAll, lv, 0);
                if (taken) w = a.sigmoid ? sigmoid_ratio(lv, M) : exp_below(lv, M);
                float total = w;  // over the slots, in pairs
                for (int off = a.slots >> 1; off > 0; off >>= 1)
                    total += __shfl_xor_sync(kAll, total, off);
                w = taken ? __fdividef(w, total) : 0.0f;
            } else if (taken) {
                w = a.sigmoid ? sigmoid(lv) : __fdividef(exp_below(lv, m), sum);
            }
            w *= a.scale;
        }
        if (lane < a.k) {
            idx[at] = chosen;
            gate[at] = w;
        }
        if (!more) return;
        t += step;
        row += row_step;
        at += (int64_t)step * a.k;
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
Args make_args(const moe_shape& s, const moe_scoring& r, bool has_bias, int V, int esize) {
    Args a{};
    a.T = s.T;
    a.E = s.E;
    a.k = s.k;
    a.sigmoid = r.score == MOE_SCORE_SIGMOID;
    a.renorm = r.renorm != 0;
    a.n_group = r.n_group;
    a.group_size = s.E / r.n_group;
    a.topk_group = r.topk_group;
    a.group_top = r.group_top;
    const int lanes = a.group_size % V == 0 ? a.group_size / V : 0;
    a.group_lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
    a.biased = has_bias;
    a.sums = r.n_group > 1 && r.group_top > 1;
    a.whole_keys = esize == 2 && !has_bias;
    // V experts a lane: 2^B >= 32 V numbers in the low bits of 23
    a.lost = a.whole_keys ? 0.0f : std::ldexp(1.01f, (V == 1 ? 5 : V == 2 ? 6 : V == 4 ? 7 : V == 8 ? 8 : 9) - 23);
    const int unit = V * esize < 16 ? V * esize : 16;
    a.vec = (s.E * esize) % unit == 0;
    a.scale = r.scale;
    a.slots = 1;
    while (a.slots < s.k) a.slots *= 2;
    return a;
}

// Blocks of kWarps rows each, no more than fit at once (the warps then loop).
unsigned blocks_for(int T, int V) {
    return (unsigned)std::min<int64_t>(((int64_t)T + kWarps - 1) / kWarps,
                                       (int64_t)device_sm_count() * blocks_per_sm(V));
}

template <typename L, int V>
int launch_route(const moe_shape& s, const moe_scoring& r, const void* logits, const float* bias,
                 const uint8_t* mask, int32_t* idx, float* gate, cudaStream_t st) {
    const Args a = make_args(s, r, bias != nullptr, V, sizeof(L));
    return launch_pdl(route_kernel<L, V>, dim3(blocks_for(s.T, V)), dim3(kWarps * 32), 0,
                      st, static_cast<const L*>(logits), bias, mask, a, idx, gate) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <typename L, int V>
int launch_backward(const moe_shape& s, const moe_scoring& r, const void* logits,
                    const int32_t* idx, const float* dgate, void* dlogits, cudaStream_t st) {
    const Args a = make_args(s, r, false, V, sizeof(L));
    return launch_pdl(backward_kernel<L, V>, dim3(blocks_for(s.T, V)), dim3(kWarps * 32),
                      0, st, static_cast<const L*>(logits), idx, dgate, a,
                      static_cast<L*>(dlogits)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <typename L, typename... Rest>
int route_for(const moe_shape& s, Rest... rest) {
    if (s.E <= 32) return launch_route<L, 1>(s, rest...);
    if (s.E <= 64) return launch_route<L, 2>(s, rest...);
    if (s.E <= 128) return launch_route<L, 4>(s, rest...);
    if (s.E <= 256) return launch_route<L, 8>(s, rest...);
    return launch_route<L, 16>(s, rest...);
}

template <typename L, typename... Rest>
int backward_for(const moe_shape& s, Rest... rest) {
    if (s.E <= 32) return launch_backward<L, 1>(s, rest...);
    if (s.E <= 64) return launch_backward<L, 2>(s, rest...);
    if (s.E <= 128) return launch_backward<L, 4>(s, rest...);
    if (s.E <= 256) return launch_backward<L, 8>(s, rest...);
    return launch_backward<L, 16>(s, rest...);
}

}  // namespace scored

int launch_route_scored(const moe_shape& s, const moe_scoring& r, const void* logits,
                        bool logits_bf16, const float* bias, const uint8_t* mask, int32_t* idx,
                        float* gate, cudaStream_t stream) {
    return logits_bf16
               ? scored::route_for<__nv_bfloat16>(s, r, logits, bias, mask, idx, gate, stream)
               : scored::route_for<float>(s, r, logits, bias, mask, idx, gate, stream);
}

int launch_route_scored_backward(const moe_shape& s, const moe_scoring& r, const void* logits,
                                 bool logits_bf16, const int32_t* idx, const float* dgate,
                                 void* dlogits, cudaStream_t stream) {
    return logits_bf16
               ? scored::backward_for<__nv_bfloat16>(s, r, logits, idx, dgate, dlogits, stream)
               : scored::backward_for<float>(s, r, logits, idx, dgate, dlogits, stream);
}

}  // namespace moe
