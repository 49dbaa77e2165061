// expert_int8.cu -- the experts' products in 8-bit integers on the 5th-generation
// tensor cores.
//
// Two launches of one persistent, warp-specialised kernel, with the rows of h
// quantised in between (int8_rows.cu):
//   gate/up (kSwiGLU):  A = xq [R, d],     B = W1q[e] | W3q[e]  ->  h bf16
//   down:               A = hq [R, d_ff],  B = W2q[e]           ->  o bf16
// with C = A B^T summed exactly in int32 (tcgen05.mma kind::i8 into TMEM) and
// scaled in the epilogue: (float(C) * row scale) * channel scale, three float32
// roundings, then SiLU(a) b for the first product and one rounding to bf16.
//
// Both operands are K-major: a stage holds 128 bytes (128 values) of K for 128 rows
// of A and 256 rows of B, written by TMA with the 128-byte swizzle.  A K, an
// output width or a row count that ends inside a box reads zeros there.
//
// Work is cut along K (the integers' sum does not depend on its order): the units
// are (tile, 128 values of K), tile-major, and every CTA takes an equal run
// of them.  A run that covers a whole tile writes its output; one that covers a part
// stores its int32 sums in the workspace and counts its units on the tile's counter,
// and whoever counts last adds the other parts and writes the output.  Nobody
// waits for another CTA, the result is the same whoever comes last, and the few
// tiles of a decode batch still load every SM alike.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "expert_int8.cuh"
#include "expert_math.cuh"
#include "int8_rows.cuh"
#include "sm100.cuh"
#include "tma_map.cuh"

namespace moe {
namespace int8gemm {

using namespace sm100;

constexpr int kBM = 128;                            // rows of a tile (TMEM lanes)
constexpr int kBK = 128;                            // values (= bytes) of K per stage
constexpr int kAccCols = 256;                       // B rows of a tile
constexpr int kStages = 4;
constexpr int kABytes = kBM * kBK;                  // 16 KB
constexpr int kBHalf = (kAccCols / 2) * kBK;        // 16 KB: one box of 128 B rows
constexpr int kStageBytes = kABytes + 2 * kBHalf;   // 48 KB
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kEpiWarps = 8;                        // two for each 32 rows of a tile
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxE = 512;
constexpr int kMaxGrid = 160;                       // CTAs at most (bounds the workspace)
constexpr int kEpiBufBytes = 2048;                  // 32 rows x 32 bf16
constexpr int kEpiScaleBytes = 512;                 // channel scales of a warp's columns
constexpr int kEpiBytes = kEpiWarps * (kEpiBufBytes + kEpiScaleBytes);
constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + kEpiBytes + 1024;

struct Params {
    const int32_t* offsets;   // [E+1]
    const float* row_scale;   // [R]
    const float* scale_a;     // [E, n_out]: s1, or s2
    const float* scale_b;     // [E, n_out]: s3
    __nv_bfloat16* out;       // [R, n_out]
    int* cnt;                 // units counted per tile and epilogue warp
    uint4* part;              // slots of part_rows x 256 int32 sums, two for each CTA
    int* err;
    uint64_t timeout_ns;
    int E, R, K, n_out;
    int tile_cols;            // output columns of a tile (128 or 256)
    int part_rows;            // rows of a slot: the most a tile (pair: a CTA's tile) can have
    int group_m;              // m-tiles per rasterisation group
    int stall_after;
};

// Exclusive prefix over the experts of their m-tiles of `rows` rows, by one warp.
// Offsets are held to 0 .. R, so that no tile lies outside the R rows.
__device__ __forceinline__ void tile_prefix(const int32_t* offsets, int E, int R, int rows,
                                            int* s_off, int* s_mt, int lane) {
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < E) {
            lo = min(max(offsets[e], 0), R);
            hi = min(max(offsets[e + 1], 0), R);
            s_off[e] = lo;
            if (e == E - 1) s_off[E] = hi;
        }
        const int mine = (max(0, hi - lo) + rows - 1) / rows;
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (e < E) s_mt[e] = carry + incl - mine;
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_mt[E] = carry;
}

struct Tile {
    int e, row0, rows, n0;
};

// Tile t of the expert-major order.  Within an expert the m-tiles are walked in
// groups of `group_m`, column by column, m fastest, so that tiles which run together share
// weight slices and a group's rows stay in L2 for all columns.  `e` is a cursor
// that only moves forward: tiles are asked for in ascending order.
__device__ __forceinline__ Tile locate(int t, int& e, const int* s_mt, const int* s_off,
                                       int n_tiles, int tile_cols, int tile_rows, int group_m) {
    while (t >= n_tiles * s_mt[e + 1]) ++e;
    const int local = t - n_tiles * s_mt[e];
    const int mt = s_mt[e + 1] - s_mt[e];
    const int m0 = mt > group_m ? local / (group_m * n_tiles) * group_m : 0;
    const int gm = min(group_m, mt - m0);
    const int r = local - m0 * n_tiles;
    const int n = r / gm;
    Tile ti;
    ti.e = e;
    ti.row0 = s_off[e] + (m0 + r - n * gm) * tile_rows;
    ti.rows = min(tile_rows, s_off[e + 1] - ti.row0);
    ti.n0 = n * tile_cols;
    return ti;
}

// ------------------------------------------------------------------ epilogue
// Eight warps: warp (q, h) takes rows 32 q .. 32 q + 31 of the tile (the TMEM lanes
// it may read) and half h of its output columns, 64 (gate/up) or 128 (down).
struct Epi {
    uint8_t* buf;    // staging of one 32 x 32 bf16 block
    float* scales;   // channel scales of this warp's columns: 64 + 64, or 128
    int q, h, lane;
};

__device__ __forceinline__ Epi make_epi(uint8_t* base, int warp, int lane) {
    const int w = warp - 2;
    return Epi{base + w * kEpiBufBytes,
               reinterpret_cast<float*>(base + kEpiWarps * kEpiBufBytes + w * kEpiScaleBytes),
               warp & 3, w >> 2, lane};
}

// This lane's four of the warp's channel scales; x0: the warp's first output column.
// Called before the wait for the accumulator, which then covers the load.
template <bool kSwiGLU, typename P>
__device__ __forceinline__ float4 load_scales(const P& p, int e, int x0, int lane) {
    const float* src = kSwiGLU && lane >= 16 ? p.scale_b : p.scale_a;
    const int col = x0 + 4 * (kSwiGLU ? lane & 15 : lane);
    if (col >= p.n_out) return make_float4(0.f, 0.f, 0.f, 0.f);
    return __ldg(reinterpret_cast<const float4*>(src + (int64_t)e * p.n_out + col));
}

// Slot of a worker's part of a tile: the worker's run of units starts (which = 0)
// or ends (1) in the tile.  Within a slot, 4 columns of all rows lie together.
__device__ __forceinline__ uint4* part_slot(uint4* slots, int worker, int which, int rows) {
    return slots + ((int64_t)(2 * worker + which) * rows) * (kAccCols / 4);
}

// The other workers' sums of a tile (first .. last except self, `step` slots pairs
// apart); none if last < first.
struct Parts {
    uint4* slots;
    int first, last, self, step, rows, row;
    bool first_is_tail;  // worker `first` holds the tile at the end of its run
};

// Workers owning units [lo, hi) of `units` dealt evenly to `active` workers.
__device__ __forceinline__ void find_parts(Parts& parts, int64_t lo, int64_t hi, int64_t units,
                                           int64_t active) {
    parts.first = (int)(((lo + 1) * active - 1) / units);
    parts.last = (int)((hi * active - 1) / units);
    parts.first_is_tail = units * parts.first / active < lo;
}

// Stores this lane's row of the sums in TMEM columns [c0, c1) to `slot`.
__device__ __forceinline__ void store_part(uint4* slot, uint32_t taddr, int c0, int c1, int rows,
                                           int row, bool valid) {
#pragma unroll 1
    for (int c = c0; c < c1; c += 32) {
        uint32_t r[32];
        tmem_ld_32cols(taddr + c, r);
        tmem_ld_wait();
        if (valid) {
            uint4* dst = slot + (int64_t)(c >> 2) * rows + row;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                __stcg(dst + (int64_t)j * rows,
                       make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
        }
    }
}

// Counts `done` units of a tile's rows of this warp, whose sums are stored;
// whether they were the last of `all`.
__device__ __forceinline__ bool count_part(int* cnt, int done, int all, int lane) {
    __threadfence();  // the sums before the count
    __syncwarp();
    int before = 0;
    if (lane == 0) before = atomicAdd(cnt, done);
    before = __shfl_sync(0xffffffffu, before, 0);
    __threadfence();  // the count before the others' sums
    return before + done == all;
}

// r[j] = the tile's int32 sums of 32 columns of this lane's row.
__device__ __forceinline__ void load_sums(uint32_t taddr, int c, uint32_t (&r)[32],
                                          const Parts& parts, bool valid) {
    tmem_ld_32cols(taddr + c, r);
    tmem_ld_wait();
    if (valid) {
        for (int w = parts.first; w <= parts.last; ++w) {
            if (w == parts.self) continue;
            const uint4* slot = part_slot(parts.slots, w * parts.step,
                                          w == parts.first && parts.first_is_tail ? 1 : 0,
                                          parts.rows) + (int64_t)(c >> 2) * parts.rows + parts.row;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 v = __ldcg(slot + (int64_t)j * parts.rows);
                r[4 * j] += v.x;
                r[4 * j + 1] += v.y;
                r[4 * j + 2] += v.z;
                r[4 * j + 3] += v.w;
            }
        }
    }
}

// r[j] = float(sum) * row scale * channel scale, for 32 columns.
__device__ __forceinline__ void scale_32(uint32_t (&r)[32], float rs, const float* s) {
    const float4* s4 = reinterpret_cast<const float4*>(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 c = s4[j];
        r[4 * j] = __float_as_uint(__int2float_rn((int)r[4 * j]) * rs * c.x);
        r[4 * j + 1] = __float_as_uint(__int2float_rn((int)r[4 * j + 1]) * rs * c.y);
        r[4 * j + 2] = __float_as_uint(__int2float_rn((int)r[4 * j + 2]) * rs * c.z);
        r[4 * j + 3] = __float_as_uint(__int2float_rn((int)r[4 * j + 3]) * rs * c.w);
    }
}

// Output columns [x0, x0 + ncols) of one row a lane: sums from the accumulator's
// columns from c0 (and, kSwiGLU, c0 + b_off for the up product), scaled by rs and
// the warp's channel scales.  When all 32 rows of the warp belong to the expert
// (`tma`), 32 x 32 blocks leave as TMA stores through the staging buffer;
// otherwise rows are stored one by one.
template <bool kSwiGLU>
__device__ __forceinline__ void write_output(const Params& p, const CUtensorMap* map,
                                             const Epi& ep, uint32_t taddr, int c0, int b_off,
                                             int x0, int ncols, int64_t grow, int y0, bool valid,
                                             bool tma, float rs, const Parts& parts) {
    const int lane = ep.lane;
#pragma unroll 1
    for (int c = 0; c < ncols; c += 32) {
        const int n = ncols - c;
        uint32_t ra[32];
        load_sums(taddr, c0 + c, ra, parts, valid);
        scale_32(ra, rs, ep.scales + c);
        if constexpr (kSwiGLU) {
            uint32_t rb[32];
            load_sums(taddr, c0 + b_off + c, rb, parts, valid);
            scale_32(rb, rs, ep.scales + 64 + c);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                ra[j] = __float_as_uint(
                    silu_times(__uint_as_float(ra[j]), __uint_as_float(rb[j])));
        }
        uint32_t packed[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            packed[j] = pack_bf16x2(__uint_as_float(ra[2 * j]), __uint_as_float(ra[2 * j + 1]));
        if (tma) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            uint8_t* rowp = ep.buf + lane * 64;
            const int sw = (lane >> 1) & 3;  // 64-byte swizzle: chunk ^= address bits 7..8
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(rowp + ((j ^ sw) << 4)) =
                    make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2],
                               packed[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, ep.buf, x0 + c, y0);
                bulk_commit_group();
            }
        } else if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + grow * p.n_out + x0 + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (8 * j < n)
                    dst[j] = make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2],
                                        packed[4 * j + 3]);
        }
    }
}

// ------------------------------------------------------------------ the kernel
// Roles (320 threads, one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer,
// warps 2..9 epilogue.  Four stages of 48 KB; two TMEM accumulators,
// so that a tile's epilogue overlaps the next tile's products.
template <bool kSwiGLU>
__global__ void __launch_bounds__(kThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                  const __grid_constant__ CUtensorMap tmB1,
                  const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full_bar[kStages], empty_bar[kStages];
    __shared__ uint64_t acc_full[2], acc_empty[2], drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_off[kMaxE + 1], s_mt[kMaxE + 1];
    __shared__ volatile int s_abort;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], kEpiWarps);
        }
        mbar_init(&drain_bar, 1);
        fence_barrier_init();
        s_abort = 0;
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB0);
        if (kSwiGLU) tma_prefetch_map(&tmB1);
        tma_prefetch_map(&tmOut);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    grid_dependency_wait();
    if (warp == 0) tile_prefix(p.offsets, p.E, p.R, kBM, s_off, s_mt, lane);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_slot;

    const int n_tiles = (p.n_out + p.tile_cols - 1) / p.tile_cols;
    const int kb_count = (p.K + kBK - 1) / kBK;
    const int64_t units = (int64_t)s_mt[p.E] * n_tiles * kb_count;
    const int64_t active = min((int64_t)gridDim.x, units);
    const int64_t me = blockIdx.x;
    const int64_t u0 = me < active ? units * me / active : 0;
    const int64_t u1 = me < active ? units * (me + 1) / active : 0;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0, issued = 0, e = 0;
            uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
            bool ok = true;
            for (int64_t u = u0; u < u1 && ok;) {
                const int t = (int)(u / kb_count);
                int kb = (int)(u - (int64_t)t * kb_count);
                const int kb1 = (int)min((int64_t)kb_count, kb + (u1 - u));
                const Tile ti = locate(t, e, s_mt, s_off, n_tiles, p.tile_cols, kBM, p.group_m);
                u += kb1 - kb;
                for (; kb < kb1; ++kb) {
                    if (p.stall_after >= 0 && issued >= p.stall_after) {
                        ok = false;  // test hook: behave like a producer that died
                        break;
                    }
                    if (!stage_wait(&empty_bar[stage], phase ^ 1u, p.timeout_ns, s_abort)) {
                        record_error(p.err, kDeviceTimeoutBase | kRoleProducer);
                        ok = false;
                        break;
                    }
                    uint8_t* sA = smem + stage * kStageBytes;
                    uint8_t* sB = sA + kABytes;
                    mbar_arrive_expect_tx(&full_bar[stage], kStageBytes);
                    tma_load_3d(sB, &tmB0, &full_bar[stage], kb * kBK, ti.n0, ti.e);
                    if (kSwiGLU)
                        tma_load_3d(sB + kBHalf, &tmB1, &full_bar[stage], kb * kBK, ti.n0, ti.e);
                    else
                        tma_load_3d(sB + kBHalf, &tmB0, &full_bar[stage], kb * kBK,
                                    ti.n0 + kAccCols / 2, ti.e);
                    tma_load_2d(sA, &tmA, &full_bar[stage], kb * kBK, ti.row0);
                    issued_mask |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) s_abort = 1;
            // every copy this thread issued lands before the CTA may exit
            for (int s = 0; s < kStages; ++s)
                if (issued_mask & (1u << s))
                    (void)mbar_wait(&full_bar[s], (issued_parity >> s) & 1u, p.timeout_ns);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMA issuer
            const uint32_t idesc = idesc_s8_s32(kBM, kAccCols);
            const uint64_t adesc0 = desc_kmajor_sw128(smem_u32(smem));
            const uint64_t bdesc0 = desc_kmajor_sw128(smem_u32(smem) + kABytes);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = u0; u < u1 && ok;) {
                const int first = (int)(u % kb_count);
                const int kb1 = (int)min((int64_t)kb_count, first + (u1 - u));
                u += kb1 - first;
                if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.timeout_ns) || s_abort) {
                    record_error(p.err, kDeviceTimeoutBase | kRoleMma);
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + acc * kAccCols;
                for (int kb = first; kb < kb1; ++kb) {
                    if (!stage_wait(&full_bar[stage], phase, p.timeout_ns, s_abort)) {
                        record_error(p.err, kDeviceTimeoutBase | kRoleMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t soff = (uint64_t)((uint32_t)(stage * kStageBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        tc_mma_s8(d_tmem, adesc0 + soff + kk * (32 >> 4),
                                  bdesc0 + soff + kk * (32 >> 4), idesc,
                                  kb != first || kk != 0);
                    tc_commit(&empty_bar[stage]);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                tc_commit(&acc_full[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok) s_abort = 1;
            // every MMA this thread issued completes before TMEM is released
            tc_commit(&drain_bar);
            (void)mbar_wait(&drain_bar, 0, p.timeout_ns);
        }
    } else {
        // ---------------------------------------------------- epilogue
        const Epi ep = make_epi(smem + kStages * kStageBytes, warp, lane);
        constexpr int kCols = kSwiGLU ? 64 : 128;  // output columns of a warp
        const int row = ep.q * 32 + lane;
        int acc = 0, e = 0;
        uint32_t acc_phase = 0;
        for (int64_t u = u0; u < u1;) {
            const int t = (int)(u / kb_count);
            const int kb = (int)(u - (int64_t)t * kb_count);
            const int done = (int)min((int64_t)kb_count - kb, u1 - u);
            const bool at_start = u == u0;
            u += done;
            const Tile ti = locate(t, e, s_mt, s_off, n_tiles, p.tile_cols, kBM, p.group_m);
            const int x0 = ti.n0 + ep.h * kCols;
            const int ncols = min(kCols, p.n_out - x0);
            const bool valid = row < ti.rows;
            const int64_t grow = (int64_t)ti.row0 + row;
            const float4 sc = load_scales<kSwiGLU>(p, ti.e, x0, lane);
            const float rs = valid ? __ldg(p.row_scale + grow) : 0.0f;
            const bool got = mbar_wait(&acc_full[acc], acc_phase, p.timeout_ns);
            if (!got || s_abort) {
                if (!got) record_error(p.err, kDeviceTimeoutBase | kRoleEpilogue);
                s_abort = 1;
                break;
            }
            tc_fence_after_sync();
            reinterpret_cast<float4*>(ep.scales)[lane] = sc;
            __syncwarp();
            const uint32_t taddr = tmem_base + acc * kAccCols + ((uint32_t)(ep.q * 32) << 16);
            const int c0 = ep.h * kCols;
            const int b_off = kSwiGLU ? kAccCols / 2 : 0;
            Parts parts{p.part, 0, -1, (int)me, 1, p.part_rows, row, false};
            // warp-uniform: this warp has rows and columns
            bool write = ep.q * 32 < ti.rows && ncols > 0;
            if (write && done < kb_count) {
                // a part of the tile's K: store the sums, count, and finish if last
                uint4* slot = part_slot(p.part, (int)me, at_start ? 0 : 1, p.part_rows);
                store_part(slot, taddr, c0, c0 + ncols, p.part_rows, row, valid);
                if (kSwiGLU)
                    store_part(slot, taddr, b_off + c0, b_off + c0 + ncols, p.part_rows, row,
                               valid);
                write = count_part(p.cnt + (int64_t)t * kEpiWarps + warp - 2, done, kb_count, lane);
                const int64_t lo = (int64_t)t * kb_count;
                if (write) find_parts(parts, lo, lo + kb_count, units, active);
            }
            if (write)
                write_output<kSwiGLU>(p, &tmOut, ep, taddr, c0, b_off, x0, ncols, grow,
                                      ti.row0 + ep.q * 32, valid, ep.q * 32 + 32 <= ti.rows, rs,
                                      parts);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        // the staging buffers outlive every store that reads them
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ------------------------------------------------------------------ CTA pairs
// A cluster of two CTAs shares each tile's products (cta_group::2): 256 rows by
// 256 columns, CTA r holding rows 128 r .. 128 r + 127 of A and half of the B rows, and
// receiving its own rows of C in its TMEM.  A stage is 32 KB a CTA, so six fit,
// and an SM reads half the B bytes of a single CTA's tile.  Gate/up: CTA r
// holds W1 rows n0 + 64 r .. + 63 and the same W3 rows, so that the accumulator's
// columns are a(0..63) b(0..63) a(64..127) b(64..127).  An expert's last rows
// are a tile like the others (its MMA takes as long with 128 rows as with 256).
//
// Tiles are dealt round-robin while they fill whole rounds of the pairs: tiles that
// run together then share weight slices and rows in L2 (a run of tiles per pair, as
// in the single-CTA kernel, re-reads each slice from DRAM for every m-tile once the
// pairs' slices together exceed L2).  The tiles of the last, partial round are cut
// along K over all pairs, as above.
//
// Synchronisation: both CTAs' loads count on the leader's full barriers; the
// leader's MMA thread commits consumed stages and finished accumulators to both
// CTAs' barriers; the epilogue warps of both arrive on the leader's acc_empty
// barriers.  Cluster barriers at the start (barriers initialised) and the end
// (before TMEM is freed) are reached by every thread; every other wait is bounded.
constexpr int kPairRows = 256;
constexpr int kPairStages = 6;
constexpr int kPairBBytes = (kAccCols / 2) * kBK;          // 16 KB: this CTA's 128 B rows
constexpr int kPairStageBytes = kABytes + kPairBBytes;     // 32 KB
constexpr size_t kPairSmemBytes = (size_t)kPairStages * kPairStageBytes + kEpiBytes + 1024;
constexpr int kMaxPairs = kMaxGrid / 2;

// The work of pair `me`: whole tiles me, me + pairs, ... of the full rounds, then
// units [u0, u1) of the remaining tiles.  next() steps through both.
struct PairWork {
    int pairs, rounds, round, kb_count, rest0;  // rest0: first tile of the partial round
    int64_t u, u0, u1, units;
    // the current segment
    int t, kb0, kb1;

    __device__ __forceinline__ PairWork(int me, int n_pairs, int tiles, int kbs) {
        pairs = n_pairs;
        rounds = tiles / n_pairs;
        round = 0;
        kb_count = kbs;
        rest0 = rounds * n_pairs;
        units = (int64_t)(tiles - rest0) * kbs;
        // fewer units than pairs: one each, for as many pairs as there are units
        const int64_t active = min((int64_t)n_pairs, units);
        u0 = me < active ? units * me / active : 0;
        u1 = me < active ? units * (me + 1) / active : 0;
        u = u0;
        t = me - n_pairs;
    }
    __device__ __forceinline__ bool next() {
        if (round < rounds) {
            ++round;
            t += pairs;
            kb0 = 0;
            kb1 = kb_count;
            return true;
        }
        if (u >= u1) return false;
        const int r = (int)(u / kb_count);
        kb0 = (int)(u - (int64_t)r * kb_count);
        kb1 = (int)min((int64_t)kb_count, kb0 + (u1 - u));
        t = rest0 + r;
        u += kb1 - kb0;
        return true;
    }
    __device__ __forceinline__ bool whole() const { return kb1 - kb0 == kb_count; }
    // whether the current part is the first of this pair's units
    __device__ __forceinline__ bool at_start() const { return u - (kb1 - kb0) == u0; }
};

template <bool kSwiGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1,
                const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full_bar[kPairStages], empty_bar[kPairStages];
    __shared__ uint64_t acc_full[2], acc_empty[2], drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_off[kMaxE + 1], s_mt[kMaxE + 1];
    __shared__ volatile int s_abort;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int me = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 2 * kEpiWarps);
        }
        mbar_init(&drain_bar, 1);
        fence_barrier_init();
        s_abort = 0;
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB0);
        if (kSwiGLU) tma_prefetch_map(&tmB1);
        tma_prefetch_map(&tmOut);
    }
    if (warp == 1) {
        tmem_alloc_pair(&tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    grid_dependency_wait();
    if (warp == 0) tile_prefix(p.offsets, p.E, p.R, kPairRows, s_off, s_mt, lane);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // the peer's barriers are initialised before anyone signals them
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_slot;

    const int n_tiles = (p.n_out + p.tile_cols - 1) / p.tile_cols;
    const int kb_count = (p.K + kBK - 1) / kBK;
    PairWork work(me, npairs, s_mt[p.E] * n_tiles, kb_count);

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            int stage = 0, issued = 0, e = 0;
            uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
            bool ok = true;
            const uint32_t leader_full0 = map_to_cta(smem_u32(&full_bar[0]), 0);
            while (ok && work.next()) {
                const Tile ti = locate(work.t, e, s_mt, s_off, n_tiles, p.tile_cols, kPairRows,
                                       p.group_m);
                const int arow = ti.row0 + rank * kBM;
                for (int kb = work.kb0; kb < work.kb1; ++kb) {
                    if (p.stall_after >= 0 && issued >= p.stall_after) {
                        ok = false;  // test hook: both producers stop at the same stage
                        break;
                    }
                    if (!stage_wait(&empty_bar[stage], phase ^ 1u, p.timeout_ns, s_abort)) {
                        record_error(p.err, kDeviceTimeoutBase | kRoleProducer);
                        ok = false;
                        break;
                    }
                    uint8_t* sA = smem + stage * kPairStageBytes;
                    uint8_t* sB = sA + kABytes;
                    const uint32_t bar = leader_full0 + stage * (uint32_t)sizeof(uint64_t);
                    if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * kPairStageBytes);
                    if (kSwiGLU) {
                        tma_load_3d_pair(sB, &tmB0, bar, kb * kBK, ti.n0 + rank * 64, ti.e);
                        tma_load_3d_pair(sB + kPairBBytes / 2, &tmB1, bar, kb * kBK,
                                         ti.n0 + rank * 64, ti.e);
                    } else {
                        tma_load_3d_pair(sB, &tmB0, bar, kb * kBK, ti.n0 + rank * 128, ti.e);
                    }
                    tma_load_2d_pair(sA, &tmA, bar, kb * kBK, arow);
                    issued_mask |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    ++issued;
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) s_abort = 1;
            // the leader's barriers count both CTAs' bytes: once every phase it
            // armed has completed, no copy of either CTA is in flight
            if (leader)
                for (int s = 0; s < kPairStages; ++s)
                    if (issued_mask & (1u << s))
                        (void)mbar_wait(&full_bar[s], (issued_parity >> s) & 1u, p.timeout_ns);
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ------------------------------------------------ MMA issuer (leader only)
            const uint32_t idesc = idesc_s8_s32(kPairRows, kAccCols);
            const uint64_t adesc0 = desc_kmajor_sw128(smem_u32(smem));
            const uint64_t bdesc0 = desc_kmajor_sw128(smem_u32(smem) + kABytes);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            while (ok && work.next()) {
                if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.timeout_ns) || s_abort) {
                    record_error(p.err, kDeviceTimeoutBase | kRoleMma);
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + acc * kAccCols;
                // the next stage's barrier is looked at before this stage's MMAs
                // are issued, so that its wait overlaps them
                bool ready = mbar_try_wait(&full_bar[stage], phase);
                for (int kb = work.kb0; kb < work.kb1; ++kb) {
                    if (!ready && !stage_wait(&full_bar[stage], phase, p.timeout_ns, s_abort)) {
                        record_error(p.err, kDeviceTimeoutBase | kRoleMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const int cur = stage;
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    ready = kb + 1 < work.kb1 && mbar_try_wait(&full_bar[stage], phase);
                    const uint64_t soff = (uint64_t)((uint32_t)(cur * kPairStageBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        tc_mma_s8_pair(d_tmem, adesc0 + soff + kk * (32 >> 4),
                                       bdesc0 + soff + kk * (32 >> 4), idesc,
                                       kb != work.kb0 || kk != 0);
                    tc_commit_pair_mc(smem_u32(&empty_bar[cur]), 0x3);
                }
                if (!ok) break;
                tc_commit_pair_mc(smem_u32(&acc_full[acc]), 0x3);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok) s_abort = 1;
            tc_commit_pair(smem_u32(&drain_bar));
            (void)mbar_wait(&drain_bar, 0, p.timeout_ns);
        }
    } else {
        // ---------------------------------------------------- epilogue (both CTAs)
        const Epi ep = make_epi(smem + kPairStages * kPairStageBytes, warp, lane);
        constexpr int kCols = kSwiGLU ? 64 : 128;
        const int row = ep.q * 32 + lane;
        int acc = 0, e = 0;
        uint32_t acc_phase = 0;
        const uint32_t leader_acc_empty0 = map_to_cta(smem_u32(&acc_empty[0]), 0);
        while (work.next()) {
            const Tile ti = locate(work.t, e, s_mt, s_off, n_tiles, p.tile_cols, kPairRows,
                                   p.group_m);
            const int x0 = ti.n0 + ep.h * kCols;
            const int ncols = min(kCols, p.n_out - x0);
            const int row0 = rank * kBM + ep.q * 32;  // this warp's first row of the tile
            const bool valid = row0 + lane < ti.rows;
            const int64_t grow = (int64_t)ti.row0 + row0 + lane;
            const float4 sc = load_scales<kSwiGLU>(p, ti.e, x0, lane);
            const float rs = valid ? __ldg(p.row_scale + grow) : 0.0f;
            const bool got = mbar_wait(&acc_full[acc], acc_phase, p.timeout_ns);
            if (!got || s_abort) {
                if (!got) record_error(p.err, kDeviceTimeoutBase | kRoleEpilogue);
                s_abort = 1;
                break;
            }
            tc_fence_after_sync();
            reinterpret_cast<float4*>(ep.scales)[lane] = sc;
            __syncwarp();
            const uint32_t taddr = tmem_base + acc * kAccCols + ((uint32_t)(ep.q * 32) << 16);
            const int c0 = ep.h * 128;
            // a CTA's slots: worker 2 pair + rank
            Parts parts{p.part + (int64_t)rank * 2 * p.part_rows * (kAccCols / 4), 0, -1, me, 2,
                        p.part_rows, row, false};
            bool write = row0 < ti.rows && ncols > 0;
            if (write && !work.whole()) {
                uint4* slot = part_slot(parts.slots, 2 * me, work.at_start() ? 0 : 1, p.part_rows);
                store_part(slot, taddr, c0, c0 + 128, p.part_rows, row, valid);
                const int r = work.t - work.rest0;
                write = count_part(p.cnt + ((int64_t)r * 2 + rank) * kEpiWarps + warp - 2,
                                   work.kb1 - work.kb0, kb_count, lane);
                if (write)
                    find_parts(parts, (int64_t)r * kb_count, (int64_t)(r + 1) * kb_count,
                               work.units, min((int64_t)npairs, work.units));
            }
            if (write)
                write_output<kSwiGLU>(p, &tmOut, ep, taddr, c0, kSwiGLU ? 64 : 0, x0, ncols, grow,
                                      ti.row0 + row0, valid, row0 + 32 <= ti.rows, rs, parts);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_acc_empty0 + acc * (uint32_t)sizeof(uint64_t));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncwarp();
    __syncthreads();
    cluster_sync_all();  // both CTAs are done with the pair's MMAs and tensor memory
    tc_fence_after_sync();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// ------------------------------------------------------------------ host side
bool rows_map(CUtensorMap* map, const void* base, int64_t rows, int cols, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)cols};
    const uint32_t box[2] = {(uint32_t)kBK, (uint32_t)box_rows};
    return make_map(map, base, 1, 2, dims, strides, box, 128);
}

bool weights_map(CUtensorMap* map, const void* base, int E, int n, int k, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
    const uint64_t strides[2] = {(uint64_t)k, (uint64_t)n * (uint64_t)k};
    const uint32_t box[3] = {(uint32_t)kBK, (uint32_t)box_rows, 1};
    return make_map(map, base, 1, 3, dims, strides, box, 128);
}

bool output_map(CUtensorMap* map, const void* base, int64_t rows, int cols) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)cols * 2};
    const uint32_t box[2] = {32, 32};
    return make_map(map, base, 2, 2, dims, strides, box, 64);
}

// Pairs that can be resident at once (a cluster lies within one GPC); per device.
template <bool kSwiGLU>
int resident_pairs() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cached[dev] == 0) {
        auto kern = pair_kernel<kSwiGLU>;
        if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)kPairSmemBytes))
            return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxGrid);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kPairSmemBytes;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kern), &cfg) !=
                cudaSuccess || n <= 0) {
            (void)cudaGetLastError();
            return 0;
        }
        cached[dev] = std::min(n, kMaxPairs);
    }
    return cached[dev];
}

// Rows from which tiles run on CTA pairs.
constexpr int64_t kPairMinRows = 512;

template <bool kSwiGLU>
int launch_product(const moe_shape& s, const int8_t* a, const int8_t* b0, const int8_t* b1,
                   Params p, cudaStream_t st) {
    const int64_t R = (int64_t)s.T * s.k;
    const bool pairs = R >= kPairMinRows;
    CUtensorMap ma, mb0, mb1, mo;
    const int b_rows = pairs && kSwiGLU ? 64 : 128;
    if (!rows_map(&ma, a, R, p.K, kBM) || !weights_map(&mb0, b0, s.E, p.n_out, p.K, b_rows) ||
        !weights_map(&mb1, b1, s.E, p.n_out, p.K, b_rows) || !output_map(&mo, p.out, R, p.n_out))
        return MOE_ERR_CUDA;
    if (pairs) {
        // m-tiles per group: their rows within 32 MB of the 126 MB L2, and at least 8
        p.group_m = (int)std::max<int64_t>(8, (int64_t(32) << 20) / ((int64_t)kPairRows * p.K));
        const int n = resident_pairs<kSwiGLU>();
        if (n <= 0) return MOE_ERR_CUDA;
        return launch_pdl(pair_kernel<kSwiGLU>, dim3(2 * n), dim3(kThreads), kPairSmemBytes, st, ma,
                          mb0, mb1, mo, p) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    }
    p.group_m = 1 << 20;
    auto kern = stream_kernel<kSwiGLU>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)kSmemBytes))
        return MOE_ERR_CUDA;
    const int grid = std::min(kMaxGrid, device_sm_count());
    return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, st, ma, mb0, mb1, mo, p) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace int8gemm

Int8Workspace int8_workspace(const moe_shape& s) {
    using namespace int8gemm;
    const size_t R = (size_t)s.T * s.k;
    const size_t mtiles = R / kBM + std::min<size_t>(R, s.E);
    const size_t rows = std::min<size_t>(kBM, R);
    Int8Workspace w{};
    size_t off = kWsHeaderBytes;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    // counters: of every tile, or, on CTA pairs, of the tiles of one partial round
    const bool pairs = (int64_t)R >= kPairMinRows;
    w.cnt1 = take(4 * kEpiWarps * (pairs ? 2 * kMaxPairs : mtiles * ((s.d_ff + 127) / 128)));
    w.cnt2 = take(4 * kEpiWarps * (pairs ? 2 * kMaxPairs : mtiles * ((s.d + 255) / 256)));
    w.zero_bytes = off;
    w.part = take(2 * (size_t)kMaxGrid * rows * kAccCols * 4);
    w.hs = take(R * 4);
    w.hq = take(R * s.d_ff);
    w.h = take(R * s.d_ff * 2);
    w.total = off;
    return w;
}

int expert_products_int8(const moe_shape& s, const int8_t* xq, const float* xs,
                         const int32_t* offsets, const Int8Experts& w, void* o, void* ws, int* err,
                         uint64_t timeout_ns, int stall_after, cudaStream_t stream) {
    using namespace int8gemm;
    const Int8Workspace L = int8_workspace(s);
    char* base = static_cast<char*>(ws);
    Params p{};
    p.offsets = offsets;
    p.row_scale = xs;
    p.scale_a = w.s1;
    p.scale_b = w.s3;
    p.out = reinterpret_cast<__nv_bfloat16*>(base + L.h);
    p.cnt = reinterpret_cast<int*>(base + L.cnt1);
    p.part = reinterpret_cast<uint4*>(base + L.part);
    p.err = err;
    p.timeout_ns = timeout_ns;
    p.E = s.E;
    p.R = s.T * s.k;
    p.K = s.d;
    p.n_out = s.d_ff;
    p.tile_cols = kAccCols / 2;
    p.part_rows = (int)std::min<int64_t>(kBM, (int64_t)s.T * s.k);
    p.stall_after = stall_after;
    int rc = launch_product<true>(s, xq, w.W1, w.W3, p, stream);
    if (rc) return rc;
    int8_t* hq = reinterpret_cast<int8_t*>(base + L.hq);
    float* hs = reinterpret_cast<float*>(base + L.hs);
    rc = launch_quantize_rows(base + L.h, (int)((int64_t)s.T * s.k), s.d_ff, offsets + s.E, hq, hs,
                              stream);
    if (rc) return rc;
    p.row_scale = hs;
    p.scale_a = w.s2;
    p.scale_b = nullptr;
    p.out = static_cast<__nv_bfloat16*>(o);
    p.cnt = reinterpret_cast<int*>(base + L.cnt2);
    p.K = s.d_ff;
    p.n_out = s.d;
    p.tile_cols = kAccCols;
    return launch_product<false>(s, hq, w.W2, w.W2, p, stream);
}

}  // namespace moe
