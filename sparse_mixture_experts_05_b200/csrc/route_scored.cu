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
// L * V, so a lower lane is a lower index and a tie goes to the first lane of a
// ballot.  Choices are compared as unsigned integers in the floats' order, which
// makes the largest of 32 lanes one redux instruction; every selected expert
// costs one such round, and only its own lane looks for its next best.
//
// Exactness of the selection.  Without a bias the order of the choices is the
// order of the logits, and the logits themselves are compared.  Biased choices
// and sums of choices are formed in float32, whose error bound is known: a row in
// which two neighbours of the selected order, or the last kept and first dropped
// group, lie closer than that bound is selected again in float64 by the same
// code.  So the result is that of float64 at the price of float32 (a few rows in
// a thousand repeat).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "route_scored.cuh"

namespace moe {
namespace scored {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;  // rows per block

struct Args {
    int T, E, k;
    int sigmoid, renorm;
    int n_group, group_size, topk_group, group_top;
    int group_lanes;  // lanes of one group when groups are whole lanes, a power of two; else 0
    int biased;       // choices are scores plus a bias; otherwise logits order them
    int sums;         // groups are valued by a sum of two choices
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
};

// This lane's V logits; an expert past E, and one whose logit is NaN, reads -inf.
template <typename L, int V>
__device__ __forceinline__ void load_row(const L* row, const Args& a, int i0, float (&l)[V]) {
    typedef RowVec<L, V> R;
    if (a.vec && i0 + V <= a.E) {
        union {
            typename R::type u[R::kUnits];
            L v[V];
        } in;
        const typename R::type* src = reinterpret_cast<const typename R::type*>(row + i0);
#pragma unroll
        for (int j = 0; j < R::kUnits; ++j) in.u[j] = __ldg(src + j);
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = to_float(in.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = i0 + j < a.E ? to_float(row[i0 + j]) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = l[j] > -INFINITY ? l[j] : -INFINITY;
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

template <typename R>
struct KeyOf;
template <>
struct KeyOf<float> {
    typedef uint32_t type;
};
template <>
struct KeyOf<double> {
    typedef unsigned long long type;
};

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

__device__ __forceinline__ float magnitude(float v) { return fabsf(v); }
__device__ __forceinline__ double magnitude(double v) { return fabs(v); }

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

// Selects the row's k experts: lane r < k returns the expert of slot r, or -1.
// `near` reports that float32 cannot tell two of them, or two groups, apart.
template <typename R, int V>
__device__ __forceinline__ int select(const float (&l)[V], const Args& a,
                                      const float* __restrict__ bias, R m, R sum, int lane,
                                      bool& near) {
    typedef typename KeyOf<R>::type K;
    constexpr bool kFloat = sizeof(R) == 4;
    const int i0 = lane * V;
    K key[V];
    const R inv = a.sigmoid ? (R)1 : (R)1 / sum;
    // Error bound of a float32 score, with room: sigmoid, 8 ulps of its value (at
    // most 1); softmax, the same and the rounding of a sum of V + 5 additions,
    // relative to the row's largest score 1 / sum.
    const R tol = a.sigmoid ? (R)9.5367432e-7 : (R)3.8146973e-6 * inv;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool live = l[j] > -INFINITY;
        if (a.biased) {
            R c = (R)0;
            if (live) {
                c = a.sigmoid ? sigmoid((R)l[j]) : exp_below((R)l[j], m) * inv;
                c += (R)__ldg(bias + i0 + j);
            }
            key[j] = live && c > -(R)INFINITY ? ordered(c) : (K)0;
        } else {
            key[j] = live ? ordered((R)l[j]) : (K)0;
        }
    }
    bool close = false;
    if (a.n_group > 1) {
        // b1, b2: the two largest choices of group `lane`
        K b1 = (K)0, b2 = (K)0;
        if (a.group_lanes) {
#pragma unroll
            for (int j = 0; j < V; ++j) merge_top2(b1, b2, key[j], (K)0);
            for (int off = 1; off < a.group_lanes; off <<= 1) {
                const K o1 = __shfl_xor_sync(kAll, b1, off);
                const K o2 = __shfl_xor_sync(kAll, b2, off);
                merge_top2(b1, b2, o1, o2);
            }
            const int src = (lane < a.n_group ? lane : 0) * a.group_lanes;
            b1 = __shfl_sync(kAll, b1, src);
            b2 = __shfl_sync(kAll, b2, src);
        } else {
            for (int g = 0; g < a.n_group; ++g) {
                K t1 = (K)0, t2 = (K)0;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const unsigned in = (unsigned)(i0 + j - g * a.group_size);
                    merge_top2(t1, t2, in < (unsigned)a.group_size ? key[j] : (K)0, (K)0);
                }
                const K m1 = warp_max(t1);
                const bool many = __popc(__ballot_sync(kAll, t1 == m1)) > 1;
                const K m2 = warp_max(t1 == m1 && !many ? t2 : t1);
                if (lane == g) {
                    b1 = m1;
                    b2 = m2;
                }
            }
        }
        K value = (K)0;
        if (lane < a.n_group && b1 != (K)0) {
            value = b1;
            if (a.sums) {
                R v1 = from_key(b1), v2 = b2 != (K)0 ? from_key(b2) : (R)0;
                if (!a.biased) {
                    v1 = a.sigmoid ? sigmoid(v1) : exp_below(v1, m) * inv;
                    if (b2 != (K)0) v2 = a.sigmoid ? sigmoid(v2) : exp_below(v2, m) * inv;
                }
                value = ordered(v1 + v2);
            }
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const K o = __shfl_sync(kAll, value, g);
            rank += o > value || (o == value && g < lane);
        }
        const bool kept = lane < a.n_group && rank < a.topk_group;
        const unsigned keep = __ballot_sync(kAll, kept);
        if (kFloat && (a.biased || a.sums)) {
            const K first_out = warp_max(lane < a.n_group && !kept ? value : (K)0);
            const K last_in = ~warp_max(kept && value != (K)0 ? ~value : (K)0);
            if (first_out != (K)0) {
                const R lo = from_key(first_out), hi = from_key(last_in);
                close = !(hi - lo > 4 * tol + (R)4.7683716e-7 * (magnitude(hi) + magnitude(lo)));
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int g = a.group_lanes ? lane / a.group_lanes : (i0 + j) / a.group_size;
            if (g >= a.n_group || !((keep >> g) & 1u)) key[j] = (K)0;
        }
    }
    // k rounds, and one more for the first expert left out
    K head = (K)0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (key[j] > head) {
            head = key[j];
            at = j;
        }
    int mine = -1;
    K mine_key = (K)0;
    const int rounds = a.k + (kFloat && a.biased ? 1 : 0);
    for (int r = 0; r < rounds; ++r) {
        const K best = warp_max(head);
        if (best == (K)0) break;
        const int owner = __ffs(__ballot_sync(kAll, head == best)) - 1;
        const int chosen = __shfl_sync(kAll, i0 + at, owner);
        if (lane == r) {
            mine = chosen;
            mine_key = best;
        }
        if (lane == owner) {
            head = (K)0;
            int next = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (j == at) key[j] = (K)0;
                if (key[j] > head) {
                    head = key[j];
                    next = j;
                }
            }
            at = next;
        }
    }
    if (kFloat && a.biased) {
        const K next = __shfl_down_sync(kAll, mine_key, 1);
        if (lane < a.k && mine_key != (K)0 && next != (K)0) {
            const R hi = from_key(mine_key), lo = from_key(next);
            close |= !(hi - lo > 2 * tol + (R)2.3841858e-7 * (magnitude(hi) + magnitude(lo)));
        }
    }
    if (kFloat && (a.biased || a.sums)) near = __any_sync(kAll, close);
    return lane < a.k ? mine : -1;
}

// The float64 repetition of a row whose float32 choices lie too close.
template <int V>
__device__ __noinline__ int select_again(const float (&l)[V], const Args& a, const float* bias,
                                         int lane) {
    double m = 0.0, sum = 1.0;
    if (!a.sigmoid) softmax_stats<double, V>(l, m, sum);
    bool near = false;
    return select<double, V>(l, a, bias, m, sum, lane, near);
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

template <typename L, int V>
__global__ void __launch_bounds__(kWarps * 32)
    route_kernel(const L* __restrict__ logits, const float* __restrict__ bias,
                 const uint8_t* __restrict__ mask, const Args a, int32_t* __restrict__ idx,
                 float* __restrict__ gate) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    int chosen = -1;
    float w = 0.0f;
    if (!mask || __ldg(mask + t)) {
        const L* row = logits + t * a.E;
        float l[V];
        load_row<L, V>(row, a, lane * V, l);
        float m = 0.0f, sum = 1.0f;
        if (!a.sigmoid && (a.biased || a.sums || !a.renorm)) softmax_stats<float, V>(l, m, sum);
        bool near = false;
        chosen = select<float, V>(l, a, bias, m, sum, lane, near);
        if (near) chosen = select_again<V>(l, a, bias, lane);
        const bool taken = chosen >= 0;
        const float lv = taken ? to_float(row[chosen]) : -INFINITY;
        if (a.renorm) {
            const float M = warp_max_float(lv);
            if (taken) w = a.sigmoid ? sigmoid_ratio(lv, M) : exp_below(lv, M);
            const float total = warp_sum(w);
            if (taken) w = __fdiv_rn(w, total);
        } else if (taken) {
            w = a.sigmoid ? sigmoid(lv) : __fdiv_rn(exp_below(lv, m), sum);
        }
        w *= a.scale;
    }
    if (lane < a.k) {
        idx[t * a.k + lane] = chosen;
        gate[t * a.k + lane] = w;
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
    union {
        typename R::type u[R::kUnits];
        L v[V];
    } out;
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
__global__ void __launch_bounds__(kWarps * 32)
    backward_kernel(const L* __restrict__ logits, const int32_t* __restrict__ idx,
                    const float* __restrict__ dgate, const Args a, L* __restrict__ dlogits) {
    __shared__ float s_row[kWarps][32 * V];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    float* buf = s_row[threadIdx.x >> 5];
    const L* row = logits + t * a.E;
    const int i0 = lane * V;
    int i = -1;
    float u = 0.0f, lv = -INFINITY;
    if (lane < a.k) {
        i = __ldg(idx + t * a.k + lane);
        if (i < 0 || i >= a.E) i = -1;
        if (i >= 0) {
            u = __ldg(dgate + t * a.k + lane) * a.scale;
            lv = to_float(__ldg(row + i));
        }
    }
    const bool live = i >= 0 && lv > -INFINITY;
    float g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = 0.0f;
    if (__any_sync(kAll, live)) {
        float v = 0.0f;  // this slot's part of the gradient of its expert's logit
        if (!a.sigmoid && !a.renorm) {
            float l[V], m, sum;
            load_row<L, V>(row, a, i0, l);
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
    }
    store_row<L, V>(dlogits + t * a.E, a, i0, g);
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
    const int unit = V * esize < 16 ? V * esize : 16;
    a.vec = (s.E * esize) % unit == 0;
    a.scale = r.scale;
    return a;
}

template <typename L, int V>
int launch_route(const moe_shape& s, const moe_scoring& r, const void* logits, const float* bias,
                 const uint8_t* mask, int32_t* idx, float* gate, cudaStream_t st) {
    const Args a = make_args(s, r, bias != nullptr, V, sizeof(L));
    return launch_pdl(route_kernel<L, V>, dim3((s.T + kWarps - 1) / kWarps), dim3(kWarps * 32), 0,
                      st, static_cast<const L*>(logits), bias, mask, a, idx, gate) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <typename L, int V>
int launch_backward(const moe_shape& s, const moe_scoring& r, const void* logits,
                    const int32_t* idx, const float* dgate, void* dlogits, cudaStream_t st) {
    const Args a = make_args(s, r, false, V, sizeof(L));
    return launch_pdl(backward_kernel<L, V>, dim3((s.T + kWarps - 1) / kWarps), dim3(kWarps * 32),
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
