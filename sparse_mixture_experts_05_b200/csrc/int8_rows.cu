// int8_rows.cu -- row kernels of the int8 layer: token lists for up to 512 experts,
// rows and weight channels quantised to 8 bits, combine of bf16 expert outputs.
//
// Quantisation of a vector v of bf16 values (a token row, or an output channel):
//     amax = max |v_i|,   q_i = rint(v_i * 127 / amax),   scale = amax / 127
// q_i is the exact quotient rounded to nearest, ties to even.  One multiplication
// by r = 127 / amax rounded up gives it: v_i and amax have 8-bit significands, so
// a quotient that is no tie is at least 1 / (254 * 255) of its size away from one
// (127 v_i 2 and (2n + 1) amax are integers of at most 16 bits, scaled alike),
// against the 2^-23 by which r exceeds 127 / amax.  A tie is 127 * 2 |v_i| = (2n + 1) amax
// with 2n + 1 <= 253, and 127 is prime.  Either it divides 2n + 1, which is then 127: |v_i| =
// amax / 2, and the quotient 63.5, exact or rounded up, goes to the even 64 either way.  Or it
// divides amax's significand, which is then 254: many v_i tie, but 127 / amax is a power of two,
// r is that very number, and the product is exact.  The product and the rounding
// are one fused multiply-add onto 1.5 * 2^23, whose low byte is q_i.
// Where 127 / amax would leave the float range (amax below 1e-30) both sides are
// scaled by 2^100 first.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "dispatch.cuh"
#include "int8_rows.cuh"
#include "sm100.cuh"

namespace moe {
namespace int8rows {

constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ quantisation
// Multiplier of a vector whose largest |value| has the bf16 bits `amax`, and its scale.
struct Quant {
    float pre, r, scale;
};

__device__ __forceinline__ Quant make_quant(uint32_t amax) {
    Quant q;
    q.pre = 1.0f;
    if (amax >= 0x7f80u) {  // an infinity or a NaN: zeros, and a scale that shows it
        q.r = 0.0f;
        q.scale = __uint_as_float(0x7fc00000u);
        return q;
    }
    const float a = __uint_as_float(amax << 16);
    q.scale = __fdiv_rn(a, 127.0f);
    if (a < 1e-30f) q.pre = 0x1p100f;
    q.r = a > 0.0f ? __fdiv_ru(127.0f, a * q.pre) : 0.0f;
    return q;
}

// Two bf16 values: the low 16 bits hold q of the low one, the high 16 q of the high
// one, each in its low byte.
__device__ __forceinline__ uint32_t quantize2(uint32_t v, const Quant& q) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
    const float lo = __fmaf_rn(bf16_lo(v) * q.pre, q.r, kMagic);
    const float hi = __fmaf_rn(bf16_hi(v) * q.pre, q.r, kMagic);
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

// Four bf16 values in two words to four bytes.  (An infinity times 0 is NaN: the
// caller zeroes rows that hold one.)
__device__ __forceinline__ uint32_t quantize4(uint32_t v0, uint32_t v1, const Quant& q) {
    return __byte_perm(quantize2(v0, q), quantize2(v1, q), 0x6420);
}

__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t v) {
    return __vmaxu2(m, v & 0x7fff7fffu);
}

// 16 bf16 values (two uint4) to 16 bytes.
__device__ __forceinline__ uint4 quantize16(const uint4& a, const uint4& b, const Quant& q) {
    if (q.r == 0.0f) return make_uint4(0u, 0u, 0u, 0u);
    return make_uint4(quantize4(a.x, a.y, q), quantize4(a.z, a.w, q), quantize4(b.x, b.y, q),
                      quantize4(b.z, b.w, q));
}

__device__ __forceinline__ uint32_t max_abs16(const uint4& a, const uint4& b, uint32_t m) {
    m = max_abs2(max_abs2(max_abs2(max_abs2(m, a.x), a.y), a.z), a.w);
    return max_abs2(max_abs2(max_abs2(max_abs2(m, b.x), b.y), b.z), b.w);
}

// Largest of both halves over the row's threads, a warp or the block (every thread
// returns it).
template <bool kWarpRow>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* s_max) {
    uint32_t one = max(m & 0xffffu, m >> 16);
    one = __reduce_max_sync(kAll, one);
    if (kWarpRow) return one;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = one;
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < warps; ++w) all = max(all, s_max[w]);
    return all;
}

// Reads the row at `src` (`units` x 16 values, `threads` of them a row's) and returns
// its multiplier.  NU > 0: the row stays in v (NU units a thread); 0: it is read again
// when it is written.
template <int NU, bool kWarpRow>
__device__ __forceinline__ Quant read_row(const uint4* __restrict__ src, int units, int tid,
                                          int threads, uint4 (&v)[NU > 0 ? NU : 1][2],
                                          uint32_t* s_max) {
    uint32_t m = 0;
    if constexpr (NU > 0) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = tid + n * threads;
            v[n][0] = v[n][1] = make_uint4(0u, 0u, 0u, 0u);
            if (u < units) {
                v[n][0] = __ldg(src + 2 * u);
                v[n][1] = __ldg(src + 2 * u + 1);
            }
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) m = max_abs16(v[n][0], v[n][1], m);
    } else {
        for (int u = tid; u < units; u += threads)
            m = max_abs16(__ldg(src + 2 * u), __ldg(src + 2 * u + 1), m);
    }
    return make_quant(row_max<kWarpRow>(m, s_max));
}

// Writes the row read by read_row to row dst.
template <int NU>
__device__ __forceinline__ void write_row(const uint4* __restrict__ src, int units, int tid,
                                          int threads, const uint4 (&v)[NU > 0 ? NU : 1][2],
                                          const Quant& q, int64_t dst, uint4* __restrict__ xq,
                                          float* __restrict__ xs) {
    if (tid == 0) xs[dst] = q.scale;
    if constexpr (NU > 0) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = tid + n * threads;
            if (u < units) xq[dst * units + u] = quantize16(v[n][0], v[n][1], q);
        }
    } else {
        for (int u = tid; u < units; u += threads)
            xq[dst * units + u] = quantize16(__ldg(src + 2 * u), __ldg(src + 2 * u + 1), q);
    }
}

// A block, or (kWarpRow) a warp, quantises one row.  kScatter: row t goes to its k
// sorted rows; otherwise row r to row r itself, if r < *map.  Both directions are whole
// vectors of consecutive bytes, so the memory bounds them: rows of 14336 values, 8192 of
// them, 54 us (6.5 TB/s).
template <int NU, bool kScatter, bool kWarpRow>
__global__ void __launch_bounds__(256)
    quantize_kernel(const uint4* __restrict__ x, int64_t rows, int units,
                    const int32_t* __restrict__ map, int k, uint4* __restrict__ xq,
                    float* __restrict__ xs, uint32_t* zero, int64_t zero_words, bool early) {
    __shared__ uint32_t s_max[8];
    if (early) launch_dependents();
    grid_dependency_wait();
    const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int threads = kWarpRow ? 32 : blockDim.x;
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                                 : (int64_t)blockIdx.x;
    if (kScatter) {
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < zero_words;
             i += (int64_t)gridDim.x * blockDim.x)
            zero[i] = 0u;
        if (kWarpRow && row >= rows) return;
    } else if (row >= min(rows, (int64_t)__ldg(map))) {
        return;
    }
    const uint4* src = x + row * units * 2;
    uint4 v[NU > 0 ? NU : 1][2];
    const Quant q = read_row<NU, kWarpRow>(src, units, tid, threads, v, s_max);
    const int copies = kScatter ? k : 1;
    for (int s = 0; s < copies; ++s) {
        const int64_t dst = kScatter ? (int64_t)__ldg(map + row * k + s) : row;
        if (dst >= 0) write_row<NU>(src, units, tid, threads, v, q, dst, xq, xs);
    }
}

// Token lists and quantised rows of a small batch (T * k <= kSmallSlots) in one launch:
// block t counts, over all slots, where its token's k rows go (slots of a lower
// expert, and earlier slots of the same one), and the blocks share the offsets.  The
// same lists as the index kernels give, without the 4 us of their launch.
constexpr int kSmallSlots = 1024;
constexpr int kSmallThreads = 256;

template <int NU>
__global__ void __launch_bounds__(kSmallThreads)
    small_dispatch_kernel(const int32_t* __restrict__ idx, const uint4* __restrict__ x, int T,
                          int E, int k, int units, int32_t* __restrict__ offsets,
                          int32_t* __restrict__ perm_tok, int32_t* __restrict__ inv,
                          uint4* __restrict__ xq, float* __restrict__ xs, uint32_t* zero,
                          int64_t zero_words) {
    __shared__ uint32_t s_max[8];
    __shared__ int s_idx[kSmallSlots];
    __shared__ int s_dst[16];
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = blockIdx.x, n = T * k;
    for (int64_t i = (int64_t)t * kSmallThreads + tid; i < zero_words;
         i += (int64_t)T * kSmallThreads)
        zero[i] = 0u;
    for (int j = tid; j < n; j += kSmallThreads) {
        const int e = __ldg(idx + j);
        s_idx[j] = e < E ? e : -1;
    }
    const uint4* src = x + (int64_t)t * units * 2;
    uint4 v[NU > 0 ? NU : 1][2];
    const Quant q = read_row<NU, false>(src, units, tid, kSmallThreads, v, s_max);
    __syncthreads();
    for (int s = warp; s < k; s += kSmallThreads / 32) {
        const int j = t * k + s, e = s_idx[j];
        int before = 0;
        for (int i = lane; i < n; i += 32) {
            const int o = s_idx[i];
            before += (o >= 0 && o < e) || (o == e && i < j);
        }
        before = __reduce_add_sync(kAll, before);
        if (lane == 0) {
            s_dst[s] = e >= 0 ? before : -1;
            inv[j] = e >= 0 ? before : -1;
            if (e >= 0) perm_tok[before] = t;
        }
    }
    for (int e = t + warp * T; e <= E; e += T * (kSmallThreads / 32)) {
        int below = 0;
        for (int i = lane; i < n; i += 32) below += s_idx[i] >= 0 && s_idx[i] < e;
        below = __reduce_add_sync(kAll, below);
        if (lane == 0) offsets[e] = below;
    }
    __syncthreads();
    for (int s = 0; s < k; ++s)
        if (s_dst[s] >= 0)
            write_row<NU>(src, units, tid, kSmallThreads, v, q, s_dst[s], xq, xs);
}

// A warp a row up to 1536 values, when there are rows for it: less than 8 warps of a
// block would have work, or wait for the others (32792 rows of 768: 14 us by warps, 20
// by blocks; 4099 rows of 2048 to 8 places each: 14 and 12).
// `early`: the next kernel may start beside this one.
template <bool kScatter>
int launch_quantize(const void* x, int64_t rows, int cols, const int32_t* map, int k, int8_t* xq,
                    float* xs, uint32_t* zero, int64_t zero_words, bool early, cudaStream_t st) {
    const int units = cols / 16;
    const bool by_warp = units <= 96 && rows >= 1024;
    const int threads = by_warp ? 256 : std::min(256, (units + 31) / 32 * 32);
    const int per = by_warp ? (units + 31) / 32 : (units + threads - 1) / threads;
    const int64_t blocks = by_warp ? (rows + 7) / 8 : rows;
    auto kern = by_warp ? (per <= 1   ? quantize_kernel<1, kScatter, true>
                           : per <= 2 ? quantize_kernel<2, kScatter, true>
                                      : quantize_kernel<4, kScatter, true>)
                        : (per <= 1   ? quantize_kernel<1, kScatter, false>
                           : per <= 2 ? quantize_kernel<2, kScatter, false>
                           : per <= 4 ? quantize_kernel<4, kScatter, false>
                                      : quantize_kernel<0, kScatter, false>);
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(threads), 0, st,
                      static_cast<const uint4*>(x), rows, units, map, k,
                      reinterpret_cast<uint4*>(xq), xs, zero, zero_words, early) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// ------------------------------------------------------------------ weights
// W [E][K][N] bf16 -> Wq [E][N][K] int8.  One block takes 64 channels of one
// expert: a pass over their K rows for the channels' amax (whole 128-byte rows of W),
// then a second pass that quantises 128 rows at a time and turns them through
// shared memory, so that Wq is written in 128-byte runs.  Run once at load time.
constexpr int kWCols = 64;
constexpr int kWRows = 128;

__global__ void __launch_bounds__(256)
    weights_kernel(const uint4* __restrict__ W, int K, int N, int8_t* __restrict__ Wq,
                   float* __restrict__ scale) {
    __shared__ uint32_t s_amax[kWCols];
    __shared__ Quant s_q[kWCols];
    __shared__ __align__(16) uint8_t s_tile[kWCols][kWRows + 16];
    grid_dependency_wait();
    const int blocks_n = (N + kWCols - 1) / kWCols;
    const int e = blockIdx.x / blocks_n;
    const int n0 = (blockIdx.x - e * blocks_n) * kWCols;
    const int chunk = threadIdx.x & 7;   // 8 columns each
    const int r0 = threadIdx.x >> 3;     // 32 rows a step
    const bool in = n0 + chunk * 8 < N;  // N is a multiple of 8
    const uint4* src = W + ((int64_t)e * K * N + n0) / 8 + chunk;
    const int64_t pitch = N / 8;
    if (threadIdx.x < kWCols) s_amax[threadIdx.x] = 0u;
    uint32_t m[4] = {0u, 0u, 0u, 0u};
    if (in) {
#pragma unroll 4
        for (int k = r0; k < K; k += 32) {
            const uint4 v = __ldg(src + k * pitch);
            m[0] = max_abs2(m[0], v.x);
            m[1] = max_abs2(m[1], v.y);
            m[2] = max_abs2(m[2], v.z);
            m[3] = max_abs2(m[3], v.w);
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        atomicMax(&s_amax[chunk * 8 + 2 * j], m[j] & 0xffffu);
        atomicMax(&s_amax[chunk * 8 + 2 * j + 1], m[j] >> 16);
    }
    __syncthreads();
    if (threadIdx.x < kWCols) {
        const Quant q = make_quant(s_amax[threadIdx.x]);
        s_q[threadIdx.x] = q;
        if (n0 + (int)threadIdx.x < N) scale[(int64_t)e * N + n0 + threadIdx.x] = q.scale;
    }
    __syncthreads();
    Quant q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = s_q[chunk * 8 + j];
    for (int k0 = 0; k0 < K; k0 += kWRows) {
#pragma unroll
        for (int s = 0; s < kWRows / 32; ++s) {
            const int k = k0 + s * 32 + r0;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (in && k < K) v = __ldg(src + k * pitch);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t one = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
                s_tile[chunk * 8 + j][s * 32 + r0] =
                    q[j].r == 0.0f ? (uint8_t)0 : (uint8_t)quantize2(one, q[j]);
            }
        }
        __syncthreads();
        // 64 channels x 128 bytes: 8 threads of 16 bytes a channel, two channels a thread
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = s * 32 + r0;
            const int k = k0 + chunk * 16;
            if (n0 + c < N && k < K)
                *reinterpret_cast<uint4*>(Wq + ((int64_t)e * N + n0 + c) * K + k) =
                    *reinterpret_cast<const uint4*>(&s_tile[c][chunk * 16]);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ token lists
// The index kernel of the dispatch for more experts: the same cluster of C CTAs and the
// same contiguous runs of slots per warp, with a counter for each (warp, expert) in
// shared memory.  The warps take the experts in turn and scan an expert's counters
// over the CTA's 32 warps; thread e reads the other CTAs' totals of expert e through
// distributed shared memory, and a scan over the experts gives their first rows.
// Stable, deterministic, no atomics on positions.
constexpr int kIndexThreads = 1024;
constexpr int kIndexWarps = 32;
constexpr int kMaxE = 512;
constexpr int kMaxCluster = 8;
constexpr int kSlotsPerWarp = 64;
constexpr int kBatch = 8;

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Lanes of the warp with this lane's expert e (of E <= 2^bits), none for e < 0: one ballot
// for each bit of the number.  (The match instruction takes longer the more numbers it
// finds; with 128 experts it made the kernel 16 us for 32792 slots.)
__device__ __forceinline__ unsigned lanes_with(int e, int bits) {
    unsigned same = __ballot_sync(kAll, e >= 0);
    for (int b = 0; b < bits; ++b) {
        const unsigned set = __ballot_sync(kAll, (e >> b) & 1);
        same &= ((e >> b) & 1) ? set : ~set;
    }
    return e >= 0 ? same : 0u;
}

__global__ void __launch_bounds__(kIndexThreads, 1)
    index_many_kernel(const int32_t* __restrict__ idx, int n, int E, int bits, int k,
                      int32_t* __restrict__ offsets, int32_t* __restrict__ perm_tok,
                      int32_t* __restrict__ inv) {
    extern __shared__ int s_pos[];  // [32][E + 1]: counts, then positions within the CTA
    __shared__ int s_total[kMaxE];  // this CTA's rows of each expert
    __shared__ int s_base[kMaxE];   // the expert's first row in this CTA
    __shared__ int s_warp[kIndexWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)sm100::cluster_ctarank();
    const int C = (int)cluster_ctas();
    const int pitch = E | 1;  // odd: an expert's 32 counters lie in 32 banks
    int* pos = s_pos + warp * pitch;
    for (int e = lane; e < E; e += 32) pos[e] = 0;
    __syncwarp();
    grid_dependency_wait();
    const int nwarps = kIndexWarps * C;
    const int per_warp = ((n + nwarps - 1) / nwarps + 31) / 32 * 32;
    const int j0 = min(n, (rank * kIndexWarps + warp) * per_warp);
    const int j1 = min(n, j0 + per_warp);
    const unsigned lt = (1u << lane) - 1u;
    const bool one_batch = per_warp <= 32 * kBatch;  // pass 2 reuses pass 1's ids
    int ids[kBatch];
    for (int base = j0; base < j1; base += 32 * kBatch) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = base + u * 32 + lane;
            ids[u] = j < j1 ? __ldg(idx + j) : -1;
            if (ids[u] >= E) ids[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * 32 >= j1) break;
            const unsigned same = lanes_with(ids[u], bits);
            if (ids[u] >= 0 && (same & lt) == 0) pos[ids[u]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = warp; e < E; e += kIndexWarps) {  // lane = warp of the CTA
        const int c = s_pos[lane * pitch + e];
        int incl = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(kAll, incl, off);
            if (lane >= off) incl += o;
        }
        s_pos[lane * pitch + e] = incl - c;
        if (lane == 31) s_total[e] = incl;
    }
    sm100::cluster_sync_all();
    int before = 0, total = 0;
    if (tid < E) {
        const uint32_t at = sm100::smem_u32(&s_total[tid]);
        for (int c = 0; c < C; ++c) {
            const int t = ld_cluster_s32(sm100::map_to_cta(at, (uint32_t)c));
            if (c < rank) before += t;
            total += t;
        }
    }
    int incl = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kAll, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (tid < E) {
        int start = incl - total;
        for (int w = 0; w < warp; ++w) start += s_warp[w];
        s_base[tid] = start + before;
        if (rank == 0) {
            offsets[tid] = start;
            if (tid == E - 1) offsets[E] = start + total;
        }
    }
    __syncthreads();
    for (int base = j0; base < j1; base += 32 * kBatch) {
        if (!one_batch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int j = base + u * 32 + lane;
                ids[u] = j < j1 ? __ldg(idx + j) : -1;
                if (ids[u] >= E) ids[u] = -1;
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * 32 >= j1) break;
            const int j = base + u * 32 + lane;
            const int e = ids[u];
            const unsigned same = lanes_with(e, bits);
            int p = -1;
            if (e >= 0) {
                p = pos[e] + s_base[e] + __popc(same & lt);
                perm_tok[p] = j / k;
            }
            if (j < j1) inv[j] = p;
            __syncwarp();
            if (e >= 0 && (same & lt) == 0) pos[e] += __popc(same);
            __syncwarp();
        }
    }
    sm100::cluster_sync_all();  // nobody leaves while its totals may still be read
}

int launch_index(const moe_shape& s, const int32_t* idx, int32_t* offsets, int32_t* perm_tok,
                 int32_t* inv, cudaStream_t stream) {
    if (s.E <= 32) return launch_dispatch_index(s, idx, offsets, perm_tok, inv, stream);
    const int64_t n = (int64_t)s.T * s.k;
    int C = 1;
    while (C < kMaxCluster && n > (int64_t)C * kIndexWarps * kSlotsPerWarp) C *= 2;
    const int smem = kIndexWarps * (s.E + 1) * 4;
    int bits = 0;
    while ((1 << bits) < s.E) ++bits;
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(index_many_kernel),
                             kIndexWarps * (kMaxE + 1) * 4))
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kIndexThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, index_many_kernel, idx, (int)n, (int)s.E, bits, (int)s.k, offsets,
                              perm_tok, inv) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// ------------------------------------------------------------------ combine
// One thread per (token, 8 columns); the k rows' loads are issued before any is used.
template <int KMAX>
__global__ void __launch_bounds__(256)
    combine_kernel(const uint4* __restrict__ o, const int32_t* __restrict__ inv,
                   const float* __restrict__ gate, int T, int d8, int k, uint4* __restrict__ y) {
    grid_dependency_wait();
    const int64_t total = (int64_t)T * d8;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t t = i / d8;
        const int c = (int)(i - t * d8);
        uint4 v[KMAX];
        float g[KMAX];
        bool has[KMAX];
#pragma unroll
        for (int s = 0; s < KMAX; ++s) {
            const int row = s < k ? __ldg(inv + t * k + s) : -1;
            has[s] = row >= 0;
            if (has[s]) {
                g[s] = __ldg(gate + t * k + s);
                v[s] = __ldg(o + (int64_t)row * d8 + c);
            }
        }
        float acc[8];
        bool first = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
#pragma unroll
        for (int s = 0; s < KMAX; ++s) {
            if (!has[s]) continue;
            const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = __fmul_rn(g[s], (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]));
                acc[j] = first ? p : __fadd_rn(acc[j], p);
            }
            first = false;
        }
        y[i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                          pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
    }
}

}  // namespace int8rows

int launch_dispatch_quantize(const moe_shape& s, const int32_t* idx, const void* x,
                             int32_t* offsets, int32_t* perm_tok, int32_t* inv, int8_t* xq,
                             float* xs, uint32_t* zero, int64_t zero_words, cudaStream_t stream) {
    using namespace int8rows;
    if (s.T > 0 && (int64_t)s.T * s.k <= kSmallSlots) {
        const int units = s.d / 16;
        const int per = (units + kSmallThreads - 1) / kSmallThreads;
        auto kern = per <= 1   ? small_dispatch_kernel<1>
                    : per <= 2 ? small_dispatch_kernel<2>
                    : per <= 4 ? small_dispatch_kernel<4>
                               : small_dispatch_kernel<0>;
        return launch_pdl(kern, dim3(s.T), dim3(kSmallThreads), 0, stream, idx,
                          static_cast<const uint4*>(x), s.T, s.E, s.k, units, offsets, perm_tok,
                          inv, reinterpret_cast<uint4*>(xq), xs, zero, zero_words) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    }
    const int rc = launch_index(s, idx, offsets, perm_tok, inv, stream);
    if (rc || s.T == 0) return rc;
    return launch_quantize<true>(x, s.T, s.d, inv, s.k, xq, xs, zero, zero_words, false,
                                 stream);
}

int launch_quantize_rows(const void* h, int max_rows, int cols, const int32_t* n_rows, int8_t* hq,
                         float* hs, cudaStream_t stream) {
    // The down product loads its first weights before it waits for these rows.  Few rows: it may
    // start beside them.  Change of the whole call, us, over d_ff = 768 to 5120: 8 experts, 256 to 2048
    // rows -0.1 to -1.5; 64 experts -3.7 to +1.0 (d_ff = 1424: +0.1 to +2.8).  Many rows of many
    // experts are held up by its CTAs: 8192 rows of 64 experts -0.9 to +4.6 (of 8: -0.2 to -2.7).
    return int8rows::launch_quantize<false>(h, max_rows, cols, n_rows, 1, hq, hs, nullptr, 0,
                                            max_rows <= 2048, stream);
}

int launch_quantize_weights(int E, int K, int N, const void* W, int8_t* Wq, float* scale,
                            cudaStream_t stream) {
    using namespace int8rows;
    const int64_t blocks = (int64_t)E * ((N + kWCols - 1) / kWCols);
    return launch_pdl(weights_kernel, dim3((unsigned)blocks), dim3(256), 0, stream,
                      static_cast<const uint4*>(W), K, N, Wq, scale) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

int launch_combine_bf16(const moe_shape& s, const void* o, const int32_t* inv, const float* gate,
                        void* y, cudaStream_t stream) {
    using namespace int8rows;
    const int64_t work = (int64_t)s.T * (s.d / 8);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((work + 255) / 256,
                                                                 (int64_t)device_sm_count() * 8));
    auto kern = s.k <= 2   ? combine_kernel<2>
                : s.k <= 4 ? combine_kernel<4>
                : s.k <= 8 ? combine_kernel<8>
                           : combine_kernel<16>;
    return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, static_cast<const uint4*>(o), inv,
                      gate, s.T, s.d / 8, s.k, static_cast<uint4*>(y)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace moe
