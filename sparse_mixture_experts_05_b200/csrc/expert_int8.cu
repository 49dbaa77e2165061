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
constexpr int kThreads = 192;
constexpr int kMaxE = 512;
constexpr int kMaxGrid = 160;                       // CTAs at most (bounds the workspace)
constexpr int kEpiBufBytes = 2048;                  // 32 rows x 32 bf16
constexpr int kEpiBytes = 4 * 2 * kEpiBufBytes;     // two buffers for each epilogue warp
constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + kEpiBytes + 1024;

struct Params {
    const int32_t* offsets;   // [E+1]
    const float* row_scale;   // [R]
    const float* scale_a;     // [E, n_out]: s1, or s2
    const float* scale_b;     // [E, n_out]: s3
    __nv_bfloat16* out;       // [R, n_out]
    int* cnt;                 // [tiles][4]: units counted per tile and 32 rows
    uint4* part;              // [2 grid] slots of part_rows x 256 int32 sums
    int* err;
    uint64_t timeout_ns;
    int E, R, K, n_out;
    int tile_cols;            // output columns of a tile (128 or 256)
    int part_rows;            // rows of a slot: the most a tile can have
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

// Tile t of the expert-major order (within an expert column by column, m fastest,
// so that the tiles of one weight slice follow each other).  `e` is a cursor that
// only moves forward: tiles are asked for in ascending order.
__device__ __forceinline__ Tile locate(int t, int& e, const int* s_mt, const int* s_off,
                                       int n_tiles, int tile_cols, int tile_rows) {
    while (t >= n_tiles * s_mt[e + 1]) ++e;
    const int local = t - n_tiles * s_mt[e];
    const int mt = s_mt[e + 1] - s_mt[e];
    const int n = local / mt;
    Tile ti;
    ti.e = e;
    ti.row0 = s_off[e] + (local - n * mt) * tile_rows;
    ti.rows = min(tile_rows, s_off[e + 1] - ti.row0);
    ti.n0 = n * tile_cols;
    return ti;
}

// ------------------------------------------------------------------ epilogue
struct EpiStage {
    uint8_t* base;
    uint32_t next;
};

// Other CTAs' sums of a tile (CTAs first .. last except self); none if last < first.
struct Parts {
    const uint4* slots;
    int first, last, self, rows, row;
    bool first_is_tail;  // CTA `first` holds the tile at the end of its run
};

__device__ __forceinline__ const uint4* part_slot(const uint4* slots, int cta, int which,
                                                  int rows) {
    return slots + ((int64_t)(2 * cta + which) * rows) * (kAccCols / 4);
}

// r[j] = the tile's int32 sums of 32 columns of this lane's row.
__device__ __forceinline__ void load_sums(uint32_t taddr, int c, uint32_t (&r)[32],
                                          const Parts& parts, bool valid) {
    tmem_ld_32cols(taddr + c, r);
    tmem_ld_wait();
    if (valid) {
        for (int cta = parts.first; cta <= parts.last; ++cta) {
            if (cta == parts.self) continue;
            const uint4* slot = part_slot(parts.slots, cta,
                                          cta == parts.first && parts.first_is_tail ? 1 : 0,
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

// r[j] = float(sum) * row scale * channel scale, for 32 columns of which `n` exist.
__device__ __forceinline__ void scale_32(uint32_t (&r)[32], float rs, const float* __restrict__ s,
                                         int n) {
    const float4* s4 = reinterpret_cast<const float4*>(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 c = 4 * j < n ? __ldg(s4 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
        r[4 * j] = __float_as_uint(__int2float_rn((int)r[4 * j]) * rs * c.x);
        r[4 * j + 1] = __float_as_uint(__int2float_rn((int)r[4 * j + 1]) * rs * c.y);
        r[4 * j + 2] = __float_as_uint(__int2float_rn((int)r[4 * j + 2]) * rs * c.z);
        r[4 * j + 3] = __float_as_uint(__int2float_rn((int)r[4 * j + 3]) * rs * c.w);
    }
}

// Output columns [x0, x0 + ncols) of one row a lane: sums from TMEM columns taddr
// (and, kSwiGLU, taddr + b_off for the up product).  When all 32 rows of the warp
// belong to the expert (`tma`), 32 x 32 blocks leave as TMA stores through two
// staging buffers; otherwise rows are stored one by one.
template <bool kSwiGLU>
__device__ __forceinline__ void write_output(const Params& p, const CUtensorMap* map, EpiStage& st,
                                             uint32_t taddr, uint32_t b_off, int e, int x0,
                                             int ncols, int64_t grow, int y0, bool valid, bool tma,
                                             float rs, const Parts& parts, int lane) {
    const float* sa = p.scale_a + (int64_t)e * p.n_out + x0;
    const float* sb = kSwiGLU ? p.scale_b + (int64_t)e * p.n_out + x0 : nullptr;
#pragma unroll 1
    for (int c = 0; c < ncols; c += 32) {
        const int n = ncols - c;
        uint32_t ra[32];
        load_sums(taddr, c, ra, parts, valid);
        scale_32(ra, rs, sa + c, n);
        if constexpr (kSwiGLU) {
            uint32_t rb[32];
            load_sums(taddr, (int)b_off + c, rb, parts, valid);
            scale_32(rb, rs, sb + c, n);
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
            uint8_t* buf = st.base + st.next * kEpiBufBytes;
            if (lane == 0) bulk_wait_group_read<1>();
            __syncwarp();
            uint8_t* rowp = buf + lane * 64;
            const int sw = (lane >> 1) & 3;  // 64-byte swizzle: chunk ^= address bits 7..8
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(rowp + ((j ^ sw) << 4)) =
                    make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2],
                               packed[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, buf, x0 + c, y0);
                bulk_commit_group();
            }
            st.next ^= 1u;
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
// Roles (192 threads, one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer,
// warps 2..5 epilogue (32 rows each).  Four stages of 48 KB; two TMEM accumulators,
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
            mbar_init(&acc_empty[a], 4);
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
                const Tile ti = locate(t, e, s_mt, s_off, n_tiles, p.tile_cols, kBM);
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
        // ---------------------------------------------------- epilogue (warps 2..5)
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int row = q * 32 + lane;
        EpiStage st{smem + kStages * kStageBytes + q * 2 * kEpiBufBytes, 0u};
        int acc = 0, e = 0;
        uint32_t acc_phase = 0;
        for (int64_t u = u0; u < u1;) {
            const int t = (int)(u / kb_count);
            const int kb = (int)(u - (int64_t)t * kb_count);
            const int done = (int)min((int64_t)kb_count - kb, u1 - u);
            const bool at_start = u == u0;
            u += done;
            const Tile ti = locate(t, e, s_mt, s_off, n_tiles, p.tile_cols, kBM);
            const bool got = mbar_wait(&acc_full[acc], acc_phase, p.timeout_ns);
            if (!got || s_abort) {
                if (!got) record_error(p.err, kDeviceTimeoutBase | kRoleEpilogue);
                s_abort = 1;
                break;
            }
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + acc * kAccCols + ((uint32_t)(q * 32) << 16);
            const bool valid = row < ti.rows;
            const int ncols = min(p.tile_cols, p.n_out - ti.n0);
            Parts parts{p.part, 0, -1, (int)me, p.part_rows, row, false};
            bool write = q * 32 < ti.rows;  // warp-uniform: this warp has rows
            if (write && done < kb_count) {
                // a part of the tile's K: store the sums, count, and finish if last
                uint4* slot = const_cast<uint4*>(part_slot(p.part, (int)me, at_start ? 0 : 1,
                                                           p.part_rows)) + row;
#pragma unroll 1
                for (int c = 0; c < kAccCols; c += 32) {
                    if ((kSwiGLU ? c & (kAccCols / 2 - 1) : c) >= ncols) continue;
                    uint32_t r[32];
                    tmem_ld_32cols(taddr + c, r);
                    tmem_ld_wait();
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            __stcg(slot + (int64_t)((c >> 2) + j) * p.part_rows,
                                   make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
                    }
                }
                __threadfence();  // the sums before the count
                __syncwarp();
                int before = 0;
                if (lane == 0) before = atomicAdd(p.cnt + (int64_t)t * 4 + q, done);
                before = __shfl_sync(0xffffffffu, before, 0);
                write = before + done == kb_count;
                if (write) {
                    __threadfence();  // the count before the others' sums
                    const int64_t lo = (int64_t)t * kb_count;
                    parts.first = (int)(((lo + 1) * active - 1) / units);
                    parts.last = (int)(((lo + kb_count) * active - 1) / units);
                    parts.first_is_tail = units * parts.first / active < lo;
                }
            }
            if (write) {
                const bool tma = q * 32 + 32 <= ti.rows;
                const int64_t grow = (int64_t)ti.row0 + row;
                const float rs = valid ? __ldg(p.row_scale + grow) : 0.0f;
                write_output<kSwiGLU>(p, &tmOut, st, taddr, kAccCols / 2, ti.e, ti.n0, ncols, grow,
                                      ti.row0 + q * 32, valid, tma, rs, parts, lane);
            }
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

template <bool kSwiGLU>
int launch_product(const moe_shape& s, const int8_t* a, const int8_t* b0, const int8_t* b1,
                   const Params& p, cudaStream_t st) {
    const int64_t R = (int64_t)s.T * s.k;
    CUtensorMap ma, mb0, mb1, mo;
    if (!rows_map(&ma, a, R, p.K, kBM) || !weights_map(&mb0, b0, s.E, p.n_out, p.K, kAccCols / 2) ||
        !weights_map(&mb1, b1, s.E, p.n_out, p.K, kAccCols / 2) ||
        !output_map(&mo, p.out, R, p.n_out))
        return MOE_ERR_CUDA;
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
    w.cnt1 = take(mtiles * ((s.d_ff + 127) / 128) * 16);
    w.cnt2 = take(mtiles * ((s.d + 255) / 256) * 16);
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
