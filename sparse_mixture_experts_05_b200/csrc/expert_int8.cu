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
// Tiles go to single CTAs (stream_kernel, 128 rows) or to CTA pairs (pair_kernel,
// 256 rows); plan_of() has the rule and what was measured.
//
// The few tiles of a small batch may be cut along K, because the integers' sum does
// not depend on its order: the units are (tile, 128 values of K), tile-major, and
// every CTA takes an equal run of them.  A run that covers a whole tile writes its
// output; one that covers a part stores its int32 sums in the workspace and counts
// its units on the tile's counter, and whoever counts last adds the parts and
// writes the output.  Nobody waits for another CTA, the result is the same whoever
// comes last, and every SM reads the same share of the weights.
//
// What bounds them: a small batch the weights' bytes (16 tokens at d = 4096, d_ff =
// 14336, 8 experts: 151 + 81 us for 0.94 + 0.47 GB, 6.2 and 5.8 TB/s); a large one the
// tensor cores under the power limit (4096 tokens: 720 + 340 us where a launch stands alone, 2.67 and
// 2.83 Pop/s; calls one after another take 1300 us with the 50 of h's rows in between); many
// small experts both, with rows padded to 128 (2051 tokens, 64 experts, d = 2048, d_ff = 1424,
// top-6: 103 + 69 us).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "expert_int8.cuh"
#include "int8_rows.cuh"
#include "sm100.cuh"
#include "tma_map.cuh"

namespace moe {
namespace int8gemm {

using namespace sm100;

constexpr int kBM = 128;                            // rows of a tile (TMEM lanes)
constexpr int kBK = 128;                            // values (= bytes) of K per stage
constexpr int kAccCols = 256;                       // B rows of a tile
constexpr int kStages = 4;  // with few rows 5 or 6 fit: no faster (16 tokens 250 us either way)
constexpr int kABytes = kBM * kBK;                  // 16 KB
constexpr int kBHalf = (kAccCols / 2) * kBK;        // 16 KB: one box of 128 B rows
constexpr int kStageBytes = kABytes + 2 * kBHalf;   // 48 KB
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kEpiWarps = 8;                        // two for each 32 rows of a tile
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxE = 512;
constexpr int kMaxGrid = 160;                       // CTAs at most (bounds the workspace)
constexpr int kEpiBufBytes = 2048;                  // 16 rows x 64 bf16
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
    int tile_cols;            // pairs: output columns of a tile (128 or 256)
    int part_rows;            // rows of a slot: the most a tile can have
    int group_m;              // m-tiles per rasterisation group
    int stall_after;
    int may_cut;              // tiles may be cut along K
    int a_rows;               // rows of an A box
};

// Offsets, held to 0 .. R so that no tile lies outside the R rows, and the exclusive
// prefix over the experts of their m-tiles of `rows` rows, held to the most that
// ascending offsets can give (what the counters have room for).  All threads of the CTA.
__device__ __forceinline__ void tile_prefix(const int32_t* offsets, int E, int R, int rows,
                                            int* s_off, int* s_mt) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) s_off[e] = min(max(__ldcg(offsets + e), 0), R);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int most = R / rows + min(R, E);
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int mine = e < E ? (max(0, s_off[e + 1] - s_off[e]) + rows - 1) / rows : 0;
            int incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            if (e < E) s_mt[e] = min(carry + incl - mine, most);
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) s_mt[E] = min(carry, most);
    }
}

struct Tile {
    int e, row0, rows, n0;
};

// Tile t of the expert-major order.  Within an expert the m-tiles are walked in
// groups of `group_m`, column by column, m fastest, so that tiles which run together share
// weight slices and a group's rows stay in L2 for all columns.  `e` is a cursor:
// the tiles asked for mostly ascend.
__device__ __forceinline__ Tile locate(int t, int& e, const int* s_mt, const int* s_off,
                                       int n_tiles, int tile_cols, int tile_rows, int group_m) {
    while (t < n_tiles * s_mt[e]) --e;
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
    uint8_t* buf;    // staging of one 16 x 64 bf16 block
    float* scales;   // channel scales of this warp's columns: 64 + 64, or 128
    int q, h, lane;
};

__device__ __forceinline__ Epi make_epi(uint8_t* base, int warp, int lane) {
    const int w = warp - 2;
    return Epi{base + w * kEpiBufBytes,
               reinterpret_cast<float*>(base + kEpiWarps * kEpiBufBytes + w * kEpiScaleBytes),
               warp & 3, w >> 2, lane};
}

// What a warp reads of a tile from memory: four channel scales and the row scale for
// every lane.  Loaded a tile ahead.  The row scales are written by a kernel beside which the down
// product may already run: no read-only loads of them.
struct TileScales {
    float4 channel;
    float row;
};

// x0: the warp's first output column; row0 .. row0 + rows - 1: its rows.
template <bool kSwiGLU, typename P>
__device__ __forceinline__ TileScales load_scales(const P& p, int e, int x0, int row0, int rows,
                                                  int lane) {
    TileScales s;
    const float* src = kSwiGLU && lane >= 16 ? p.scale_b : p.scale_a;
    const int col = x0 + 4 * (kSwiGLU ? lane & 15 : lane);
    s.channel = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < p.n_out)
        s.channel = __ldg(reinterpret_cast<const float4*>(src + (int64_t)e * p.n_out + col));
    s.row = lane < rows ? __ldcg(p.row_scale + row0 + lane) : 0.0f;
    return s;
}

// A part of a tile's sums over K: int32 [rows][256].  A worker (CTA) has two slots,
// for the tile that its run of units starts in (which = 0) and the one it ends in (1).
__device__ __forceinline__ uint4* part_slot(uint4* slots, int worker, int which, int rows) {
    return slots + ((int64_t)(2 * worker + which) * rows) * (kAccCols / 4);
}

// The workers that hold parts of a tile.
struct Parts {
    int first, last;
    bool first_is_tail;  // worker `first` holds the tile at the end of its run
};

// Workers owning units [lo, hi) of `units` dealt evenly to `active` workers.
__device__ __forceinline__ Parts find_parts(int64_t lo, int64_t hi, int64_t units,
                                            int64_t active) {
    Parts parts;
    parts.first = (int)(((lo + 1) * active - 1) / units);
    parts.last = (int)((hi * active - 1) / units);
    parts.first_is_tail = units * parts.first / active < lo;
    return parts;
}

// Stores this lane's row of the sums in TMEM columns [c0, c1) to `slot`.
__device__ __forceinline__ void store_part(uint4* slot, uint32_t taddr, int c0, int c1, int row,
                                           bool valid) {
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        uint32_t r[16];
        tmem_ld_16cols(taddr + c, r);
        tmem_ld_wait();
        if (valid) {
            uint4* dst = slot + row * (kAccCols / 4) + (c >> 2);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                __stcg(dst + j, make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
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

// Four columns of one row summed over all parts (`at`: their place in a slot).
__device__ __forceinline__ int4 sum_parts(uint4* slots, const Parts& parts, int rows, int at) {
    int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 2
    for (int w = parts.first; w <= parts.last; ++w) {
        const uint4 v = __ldcg(
            part_slot(slots, w, w == parts.first && parts.first_is_tail ? 1 : 0, rows) + at);
        sum.x += (int)v.x;
        sum.y += (int)v.y;
        sum.z += (int)v.z;
        sum.w += (int)v.w;
    }
    return sum;
}

// float(sum) * row scale * channel scale of two neighbouring columns.
__device__ __forceinline__ float2 scaled(int s0, int s1, float2 rs, float2 channel) {
    const float2 f = make_float2(__int2float_rn(s0), __int2float_rn(s1));
    return __fmul2_rn(__fmul2_rn(f, rs), channel);
}

// SiLU(a) b = a / (1 + e^-a) b, off by at most 10 2^-24 of its value whatever a is: expf within
// two ulps, the sum and the product half an ulp each, the quick division within two.  Below
// a = -87.3 the divisor passes 2^126 and the quotient is 0 (its true value is under |a| 2^-126).
// ex2.approx and rcp.approx of packed pairs, 6 instructions an element, are off by another |a| 2^-24
// and no more than 2 % faster (1024 tokens, d = 1024, d_ff = 3584, 8 experts: 61.4 and 62.5 us;
// 2051 tokens to 64 experts 212 and 214; 4096 tokens of d = 4096 alike); the IEEE division with its
// branch costs 4 to 40 % (87.9, 257 and 1400 us).
__device__ __forceinline__ float silu_times(float a, float b) {
    return __fmul_rn(__fdividef(a, __fadd_rn(1.0f, expf(-a))), b);
}
__device__ __forceinline__ float2 silu_times2(float2 a, float2 b) {
    return make_float2(silu_times(a.x, b.x), silu_times(a.y, b.y));
}

// Output columns [x0, x0 + ncols) of the warp's 32 rows (`rows` of them exist; y0
// is the first): sums from the accumulator's columns from c0 (and, kSwiGLU, c0 +
// b_off for the up product) of this lane's row, scaled by rs and the warp's channel
// scales.  64 columns are packed at a time and turned in shared memory, 16 rows
// after 16, so that eight lanes store 128 consecutive bytes of a row: whole cache lines
// (32-byte pieces cost the down product of many small experts 10 us of 90).
template <bool kSwiGLU>
__device__ __forceinline__ void write_output(const Params& p, const Epi& ep, uint32_t taddr, int c0,
                                             int b_off, int x0, int ncols, int y0, int rows,
                                             float rs) {
    const int lane = ep.lane;
    const float2 rs2 = make_float2(rs, rs);
    // 16-byte piece j of staged row r lies at piece j ^ (r % 8): no bank conflicts
    uint8_t* put = ep.buf + (lane & 15) * 128;
    const int put_sw = lane & 7;
    const int piece = lane & 7, r0 = lane >> 3;
    __nv_bfloat16* dst = p.out + (int64_t)(y0 + r0) * p.n_out + x0 + piece * 8;
    uint32_t ra[16], rb[16];
    tmem_ld_16cols(taddr + c0, ra);
    if constexpr (kSwiGLU) tmem_ld_16cols(taddr + c0 + b_off, rb);
#pragma unroll 1
    for (int b = 0; b < ncols; b += 64) {
        uint32_t packed[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = b + 16 * i;
            const float2* sa = reinterpret_cast<const float2*>(ep.scales + c);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float2 o = scaled((int)ra[2 * j], (int)ra[2 * j + 1], rs2, sa[j]);
                if constexpr (kSwiGLU)
                    o = silu_times2(o, scaled((int)rb[2 * j], (int)rb[2 * j + 1], rs2, sa[32 + j]));
                packed[8 * i + j] = pack_bf16x2(o.x, o.y);
            }
            if (c + 16 < ncols) {  // the next sums, on their way while these are stored
                tmem_ld_16cols(taddr + c0 + c + 16, ra);
                if constexpr (kSwiGLU) tmem_ld_16cols(taddr + c0 + b_off + c + 16, rb);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if ((lane >> 4) == half) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(put + ((j ^ put_sw) << 4)) = make_uint4(
                        packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
            }
            __syncwarp();
            if (b + piece * 8 < ncols) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 4 + r0;
                    if (half * 16 + r < rows)
                        *reinterpret_cast<uint4*>(dst + (int64_t)(half * 16 + i * 4) * p.n_out +
                                                  b) =
                            *reinterpret_cast<const uint4*>(ep.buf + r * 128 +
                                                            ((piece ^ (r & 7)) << 4));
                }
            }
            __syncwarp();
        }
    }
}

// The same for a tile whose sums lie in parts in the workspace: a lane takes four
// columns of a row, so that all parts' loads are in flight together.  `rs` is lane
// r's row scale; `prow` the warp's first row in a slot.
// kBatch steps of rows have their loads issued together.
template <bool kSwiGLU, int kBatch>
__device__ __forceinline__ void write_parts(const Params& p, const Epi& ep, const Parts& parts,
                                            int c0, int b_off, int x0, int ncols, int y0, int prow,
                                            int rows, float rs) {
    constexpr int kQuads = kSwiGLU ? 16 : 32;  // lanes a row takes
    constexpr int kStep = 32 / kQuads;         // rows of the warp at a time
    const int quad = min(ep.lane & (kQuads - 1), ncols / 4 - 1);
    const bool mine = (ep.lane & (kQuads - 1)) == quad;
    rows = min(rows, 32);
    const float4 sa = reinterpret_cast<const float4*>(ep.scales)[quad];
    const float4 sb = reinterpret_cast<const float4*>(ep.scales)[kSwiGLU ? 16 + quad : quad];
#pragma unroll 1
    for (int r0 = ep.lane / kQuads; r0 - ep.lane / kQuads < rows; r0 += kStep * kBatch) {
        int4 a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int at = (prow + min(r0 + i * kStep, rows - 1)) * (kAccCols / 4) + (c0 >> 2) + quad;
            a[i] = sum_parts(p.part, parts, p.part_rows, at);
            if constexpr (kSwiGLU) b[i] = sum_parts(p.part, parts, p.part_rows, at + (b_off >> 2));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kStep;
            const float row = __shfl_sync(0xffffffffu, rs, r & 31);
            const float2 rs2 = make_float2(row, row);
            float2 lo = scaled(a[i].x, a[i].y, rs2, make_float2(sa.x, sa.y));
            float2 hi = scaled(a[i].z, a[i].w, rs2, make_float2(sa.z, sa.w));
            if constexpr (kSwiGLU) {
                lo = silu_times2(lo, scaled(b[i].x, b[i].y, rs2, make_float2(sb.x, sb.y)));
                hi = silu_times2(hi, scaled(b[i].z, b[i].w, rs2, make_float2(sb.z, sb.w)));
            }
            if (mine && r < rows)
                *reinterpret_cast<uint2*>(p.out + (int64_t)(y0 + r) * p.n_out + x0 + 4 * quad) =
                    make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(hi.x, hi.y));
        }
    }
    __syncwarp();
}

// The work of CTA `me` of `grid`: whole tiles me, me + grid, ..., or, where `may_cut`
// and that spares the busiest CTA enough, an equal run of the units (tile, 128 values of K).
// Enough, in units of about 0.5 us: 12.5 for storing and adding parts at all, 2 for each row of a
// tile (of the mean of them) and another fifth for each part of it, since whoever adds them
// takes row after row and part after part, and a quarter for each row of the batch, which are all
// stored.  Over 436 products of 1 to 500 rows, 1 to 64 experts, K 512 to 14000, the better way
// is missed by 0.25 % of the call in the mean, by 23 % at the most (with 14 and 3/8 a
// row of the batch alone: 4 % and fivefold).  Whole / cut, us, of the whole call:
// down product of K = 14336, 8 experts, 2 rows 99 / 75, 8 rows 203 / 196, 32 rows 256 / 267; of K =
// 8192, 4 experts, 2 rows 49 / 38, 8 rows 60 / 56, 64 rows 65 / 97; of K = 9184, one expert,
// 24 rows 51 / 196; gate/up product of K = 4096, 8 experts, 32 rows 258 / 255, 64 rows 262 / 267;
// of K = 3312, one expert, 22 rows 31 / 185.
// Of a run, the parts of tiles at its two ends come first, so that whoever adds a
// tile's parts has whole tiles to hide that behind.
struct Run {
    int64_t u, u0, u1, skip, units, active;
    int kb_count, step;
    int t, kb0, kb1;  // the current tile and its part

    __device__ __forceinline__ Run(int me, int grid, int m_tiles, int n_tiles, int kbs, bool may_cut,
                                   int rows) {
        const int tiles = m_tiles * n_tiles;
        kb_count = kbs;
        units = (int64_t)tiles * kbs;
        active = min((int64_t)grid, units);
        const int64_t rounds = (tiles + grid - 1) / grid;
        const float spared = (float)(rounds * kbs) - (float)units / (float)active;
        const float tile_rows = (float)rows / (float)m_tiles;
        const float parts = (float)active / (float)tiles;
        const float enough = 12.5f + tile_rows * (2.0f + 0.2f * parts) + 0.25f * (float)rows;
        if (!may_cut || !(spared > enough)) {  // (no tiles: NaN)
            u0 = (int64_t)me * kbs;
            u1 = units;
            skip = (int64_t)(grid - 1) * kbs;
        } else {
            u0 = me < active ? units * me / active : 0;
            u1 = me < active ? units * (me + 1) / active : 0;
            skip = 0;
        }
        u = u0;
        step = 0;
    }
    __device__ __forceinline__ bool next() {
        if (step == 0) {  // the part at the start, if the run starts inside a tile
            step = 1;
            kb0 = (int)(u0 % kb_count);
            if (u0 < u1 && kb0 != 0) {
                t = (int)(u0 / kb_count);
                kb1 = (int)min((int64_t)kb_count, kb0 + (u1 - u0));
                u = u0 + kb1 - kb0;
                return true;
            }
        }
        if (step == 1) {  // the part at the end
            step = 2;
            kb1 = (int)(u1 % kb_count);
            if (u < u1 && kb1 != 0) {
                t = (int)(u1 / kb_count);
                kb0 = 0;
                return true;
            }
        }
        // the whole tiles in between
        if (u + kb_count > u1) return false;
        t = (int)(u / kb_count);
        kb0 = 0;
        kb1 = kb_count;
        u += kb_count + skip;
        return true;
    }
    __device__ __forceinline__ bool starts() const { return (int64_t)t * kb_count + kb0 == u0; }
};

// ------------------------------------------------------------------ the kernel
// Roles (320 threads, one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer, the
// others epilogue.  Four stages of 48 KB; two TMEM accumulators,
// so that a tile's epilogue overlaps the next tile's products.  The down product's weights
// depend on nothing that the kernel before it (h's quantisation) writes, nor do the offsets:
// its producers load the first stages' weights before they wait for that kernel.  (This needs the
// kernel before that, the gate/up product, to have ended: it may not let its dependents start
// early, or the offsets' and weights' writers could still be at work when the down product reads them.)
template <bool kSwiGLU>
__global__ void __launch_bounds__(kThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                  const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ Params p) {
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
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (kSwiGLU) grid_dependency_wait();  // the down product waits further below
    tile_prefix(p.offsets, p.E, p.R, kBM, s_off, s_mt);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_slot;

    constexpr int kTileCols = kSwiGLU ? kAccCols / 2 : kAccCols;  // output columns of a tile
    const int n_tiles = (p.n_out + kTileCols - 1) / kTileCols;
    const int kb_count = (p.K + kBK - 1) / kBK;
    Run run(blockIdx.x, gridDim.x, s_mt[p.E], n_tiles, kb_count, p.may_cut != 0, s_off[p.E]);
    if (!kSwiGLU && warp != 0) grid_dependency_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0, issued = 0, e = 0;
            uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
            bool ok = true;
            int ahead = 0;  // stages whose weights are on their way already
            if constexpr (!kSwiGLU) {
                Run begin = run;
                if (p.stall_after < 0 && begin.next()) {
                    const Tile ti = locate(begin.t, e, s_mt, s_off, n_tiles, kTileCols, kBM,
                                           p.group_m);
                    for (; ahead < kStages && begin.kb0 + ahead < begin.kb1; ++ahead) {
                        uint8_t* sB = smem + ahead * kStageBytes + kABytes;
                        const int x = (begin.kb0 + ahead) * kBK;
                        mbar_arrive_expect_tx(&full_bar[ahead], p.a_rows * kBK + 2 * kBHalf);
                        tma_load_3d(sB, &tmB0, &full_bar[ahead], x, ti.n0, ti.e);
                        tma_load_3d(sB + kBHalf, &tmB0, &full_bar[ahead], x,
                                    ti.n0 + kAccCols / 2, ti.e);
                    }
                }
                grid_dependency_wait();
            }
            while (ok && run.next()) {
                const Tile ti = locate(run.t, e, s_mt, s_off, n_tiles, kTileCols, kBM,
                                       p.group_m);
                for (int kb = run.kb0; kb < run.kb1; ++kb) {
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
                    if (kSwiGLU || issued >= ahead) {
                        mbar_arrive_expect_tx(&full_bar[stage], p.a_rows * kBK + 2 * kBHalf);
                        // rows of W1 and of W3, or two halves of W2's
                        tma_load_3d(sB, &tmB0, &full_bar[stage], kb * kBK, ti.n0, ti.e);
                        tma_load_3d(sB + kBHalf, kSwiGLU ? &tmB1 : &tmB0, &full_bar[stage],
                                    kb * kBK, kSwiGLU ? ti.n0 : ti.n0 + kAccCols / 2, ti.e);
                    }
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
            while (ok && run.next()) {
                if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.timeout_ns) || s_abort) {
                    record_error(p.err, kDeviceTimeoutBase | kRoleMma);
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + acc * kAccCols;
                for (int kb = run.kb0; kb < run.kb1; ++kb) {
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
                                  kb != run.kb0 || kk != 0);
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
        constexpr int kCols = kTileCols / 2;  // output columns of a warp
        constexpr int b_off = kSwiGLU ? kAccCols / 2 : 0;
        const int c0 = ep.h * kCols;
        const int row0 = ep.q * 32;
        int acc = 0, e = 0;
        uint32_t acc_phase = 0;
        Tile ti{};
        TileScales sc{};
        bool more = run.next();
        if (more) {
            ti = locate(run.t, e, s_mt, s_off, n_tiles, kTileCols, kBM, p.group_m);
            sc = load_scales<kSwiGLU>(p, ti.e, ti.n0 + c0, ti.row0 + row0, ti.rows - row0, lane);
        }
        while (more) {
            const bool got = mbar_wait(&acc_full[acc], acc_phase, p.timeout_ns);
            if (!got || s_abort) {
                if (!got) record_error(p.err, kDeviceTimeoutBase | kRoleEpilogue);
                s_abort = 1;
                break;
            }
            tc_fence_after_sync();
            reinterpret_cast<float4*>(ep.scales)[lane] = sc.channel;
            __syncwarp();
            const Tile now = ti;
            const float rs = sc.row;
            const int t = run.t, done = run.kb1 - run.kb0;
            const bool starts = run.starts();
            more = run.next();
            if (more) {  // the next tile's scales load behind this one's work
                ti = locate(run.t, e, s_mt, s_off, n_tiles, kTileCols, kBM, p.group_m);
                sc = load_scales<kSwiGLU>(p, ti.e, ti.n0 + c0, ti.row0 + row0, ti.rows - row0,
                                          lane);
            }
            const uint32_t taddr = tmem_base + acc * kAccCols + ((uint32_t)row0 << 16);
            const int x0 = now.n0 + c0;
            const int ncols = min(kCols, p.n_out - x0);
            if (row0 < now.rows && ncols > 0) {  // warp-uniform: this warp has rows and columns
                if (done == kb_count) {
                    write_output<kSwiGLU>(p, ep, taddr, c0, b_off, x0, ncols, now.row0 + row0,
                                          now.rows - row0, rs);
                } else {
                    // a part of the tile's K: store the sums, count, and finish if last
                    uint4* slot =
                        part_slot(p.part, blockIdx.x, starts ? 0 : 1, p.part_rows);
                    const bool valid = row0 + lane < now.rows;
                    store_part(slot, taddr, c0, c0 + ncols, row0 + lane, valid);
                    if (kSwiGLU)
                        store_part(slot, taddr, b_off + c0, b_off + c0 + ncols, row0 + lane,
                                          valid);
                    if (count_part(p.cnt + (int64_t)t * kEpiWarps + warp - 2, done, kb_count,
                                   lane)) {
                        const int64_t lo = (int64_t)t * kb_count;
                        const Parts parts = find_parts(lo, lo + kb_count, run.units, run.active);
                        if (now.rows - row0 <= 2)
                            write_parts<kSwiGLU, 1>(p, ep, parts, c0, b_off, x0, ncols,
                                                    now.row0 + row0, row0, now.rows - row0, rs);
                        else
                            write_parts<kSwiGLU, 4>(p, ep, parts, c0, b_off, x0, ncols,
                                                    now.row0 + row0, row0, now.rows - row0, rs);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
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
// Tiles are dealt round-robin: tiles that run together then share weight slices and
// rows in L2 (a run of tiles per pair, as in the single-CTA kernel, re-reads each
// slice from DRAM for every m-tile once the pairs' slices together exceed L2).  Cutting
// the last, partial round along K as above measured slower: storing and adding parts
// of 256 rows took about 25 us, more than a whole tile of K = 3584 (layer of 1024
// tokens, d = 1024, d_ff = 3584: 58 + 28 us against 30 + 18).
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

template <bool kSwiGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ Params p) {
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
    }
    if (warp == 1) {
        tmem_alloc_pair(&tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    if (kSwiGLU) grid_dependency_wait();
    tile_prefix(p.offsets, p.E, p.R, kPairRows, s_off, s_mt);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // the peer's barriers are initialised before anyone signals them
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_slot;

    const int n_tiles = (p.n_out + p.tile_cols - 1) / p.tile_cols;
    const int kb_count = (p.K + kBK - 1) / kBK;
    const int tiles = s_mt[p.E] * n_tiles;
    if (!kSwiGLU && warp != 0) grid_dependency_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            int stage = 0, issued = 0, e = 0;
            uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
            bool ok = true;
            const uint32_t leader_full0 = map_to_cta(smem_u32(&full_bar[0]), 0);
            int ahead = 0;  // stages whose weights are on their way already
            if constexpr (!kSwiGLU) {
                if (p.stall_after < 0 && me < tiles) {
                    const Tile ti = locate(me, e, s_mt, s_off, n_tiles, p.tile_cols, kPairRows,
                                           p.group_m);
                    for (; ahead < kPairStages && ahead < kb_count; ++ahead) {
                        if (leader) mbar_arrive_expect_tx(&full_bar[ahead], 2 * kPairStageBytes);
                        tma_load_3d_pair(smem + ahead * kPairStageBytes + kABytes, &tmB0,
                                         leader_full0 + ahead * (uint32_t)sizeof(uint64_t),
                                         ahead * kBK, ti.n0 + rank * 128, ti.e);
                    }
                }
                grid_dependency_wait();
            }
            for (int t = me; t < tiles && ok; t += npairs) {
                const Tile ti = locate(t, e, s_mt, s_off, n_tiles, p.tile_cols, kPairRows,
                                       p.group_m);
                const int arow = ti.row0 + rank * kBM;
                for (int kb = 0; kb < kb_count; ++kb) {
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
                    const bool fresh = kSwiGLU || issued >= ahead;
                    if (leader && fresh)
                        mbar_arrive_expect_tx(&full_bar[stage], 2 * kPairStageBytes);
                    if (kSwiGLU) {
                        tma_load_3d_pair(sB, &tmB0, bar, kb * kBK, ti.n0 + rank * 64, ti.e);
                        tma_load_3d_pair(sB + kPairBBytes / 2, &tmB1, bar, kb * kBK,
                                         ti.n0 + rank * 64, ti.e);
                    } else if (fresh) {
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
            for (int t = me; t < tiles && ok; t += npairs) {
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
                for (int kb = 0; kb < kb_count; ++kb) {
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
                    ready = kb + 1 < kb_count && mbar_try_wait(&full_bar[stage], phase);
                    const uint64_t soff = (uint64_t)((uint32_t)(cur * kPairStageBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        tc_mma_s8_pair(d_tmem, adesc0 + soff + kk * (32 >> 4),
                                       bdesc0 + soff + kk * (32 >> 4), idesc,
                                       (kb | kk) != 0);
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
        const int row0 = rank * kBM + ep.q * 32;  // this warp's first row of a tile
        int acc = 0, e = 0;
        uint32_t acc_phase = 0;
        const uint32_t leader_acc_empty0 = map_to_cta(smem_u32(&acc_empty[0]), 0);
        Tile ti{};
        TileScales sc{};
        if (me < tiles) {
            ti = locate(me, e, s_mt, s_off, n_tiles, p.tile_cols, kPairRows, p.group_m);
            sc = load_scales<kSwiGLU>(p, ti.e, ti.n0 + ep.h * kCols, ti.row0 + row0,
                                      ti.rows - row0, lane);
        }
        for (int t = me; t < tiles; t += npairs) {
            const bool got = mbar_wait(&acc_full[acc], acc_phase, p.timeout_ns);
            if (!got || s_abort) {
                if (!got) record_error(p.err, kDeviceTimeoutBase | kRoleEpilogue);
                s_abort = 1;
                break;
            }
            tc_fence_after_sync();
            reinterpret_cast<float4*>(ep.scales)[lane] = sc.channel;
            __syncwarp();
            const Tile now = ti;
            const float rs = sc.row;
            if (t + npairs < tiles) {  // the next tile's scales load behind this one's work
                ti = locate(t + npairs, e, s_mt, s_off, n_tiles, p.tile_cols, kPairRows,
                            p.group_m);
                sc = load_scales<kSwiGLU>(p, ti.e, ti.n0 + ep.h * kCols, ti.row0 + row0,
                                          ti.rows - row0, lane);
            }
            const int x0 = now.n0 + ep.h * kCols;
            const int ncols = min(kCols, p.n_out - x0);
            if (row0 < now.rows && ncols > 0)
                write_output<kSwiGLU>(
                    p, ep, tmem_base + acc * kAccCols + ((uint32_t)(ep.q * 32) << 16), ep.h * 128,
                    kSwiGLU ? 64 : 0, x0, ncols, now.row0 + row0, now.rows - row0, rs);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_acc_empty0 + acc * (uint32_t)sizeof(uint64_t));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
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
    return make_byte_map(map, base, 2, dims, strides, box);
}

bool weights_map(CUtensorMap* map, const void* base, int E, int n, int k, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
    const uint64_t strides[2] = {(uint64_t)k, (uint64_t)n * (uint64_t)k};
    const uint32_t box[3] = {(uint32_t)kBK, (uint32_t)box_rows, 1};
    return make_byte_map(map, base, 3, dims, strides, box);
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
        cached[dev] = n;
    }
    return cached[dev];
}

// How the rows of a call are worked on.
//  kCut: single CTAs, tiles cut along K where that pays; kDealt: single CTAs, whole
//  tiles; kPairs: CTA pairs, whole tiles.
enum Plan { kCut, kDealt, kPairs };

// From 512 routed rows there are enough tiles, and enough rows for parts to be dear
// (512 tokens, d = 4096, d_ff = 14336, 8 experts, top-2: 163 us whole, 278 cut).
// Pairs read a third fewer bytes into the SMs for the same products but pad rows to
// 256, not 128.  Down product, change of the whole call with pairs for single CTAs over 13 to 39
// shapes each (4 to 32 experts, 128 to 2048 rows of each, d = 1024 to 4096): K = 1424 -3 %, 2048
// 0, 2560 -1 %, 3584 -3 %, 4096 -1 %, 5120 -3 % in the mean, between -17 and +10 % (the worst
// at every K is 8 experts of 512 rows give or take 20, 2 or 3 tiles of 256 each); K = 768 and 240 rows
// of each of 128 experts 77 us single, 98 in pairs.  So nothing is won for sure below K = 3500.  Gate/up
// product, K = 4096 and 5120: 1024 rows of an expert +1 to -6 %, 1280 0 to -3 %, 1536 0 to -1 %, 2048
// -1 to -4 %, 3584 -1 to -3 %; 128 rows 163 us single, 184 in pairs; K = 2048 and 192 rows 97 and 101.
Plan plan_of(const moe_shape& s, int K, bool swiglu) {
    const int64_t R = (int64_t)s.T * s.k;
    if (R < 512) return kCut;
    return K >= 3500 && (!swiglu || R >= (int64_t)1536 * s.E) ? kPairs : kDealt;
}

// m-tiles per group: their rows within 32 MB of the 126 MB L2, and at least 2048 rows.
int group_of(int tile_rows, int K) {
    return (int)std::max<int64_t>(2048 / tile_rows, (int64_t(32) << 20) / ((int64_t)tile_rows * K));
}

template <bool kSwiGLU>
int launch_pairs(const moe_shape& s, const int8_t* a, const int8_t* b0, const int8_t* b1, Params p,
                 cudaStream_t st) {
    CUtensorMap ma, mb0, mb1;
    const int b_rows = kSwiGLU ? 64 : 128;
    if (!rows_map(&ma, a, p.R, p.K, kBM) || !weights_map(&mb0, b0, s.E, p.n_out, p.K, b_rows) ||
        !weights_map(&mb1, b1, s.E, p.n_out, p.K, b_rows))
        return MOE_ERR_CUDA;
    p.group_m = group_of(kPairRows, p.K);
    const int n = resident_pairs<kSwiGLU>();
    if (n <= 0) return MOE_ERR_CUDA;
    return launch_pdl(pair_kernel<kSwiGLU>, dim3(2 * n), dim3(kThreads), kPairSmemBytes, st, ma,
                      mb0, mb1, p) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <bool kSwiGLU>
int launch_single(const moe_shape& s, const int8_t* a, const int8_t* b0, const int8_t* b1, Params p,
                  bool may_cut, cudaStream_t st) {
    // a box has as many rows as there are, in eights: rows past the tensor's end are
    // filled with zeros at a price (5 experts' weights, 8 rows: 135 us with boxes of
    // 128 rows, 110 with 8)
    p.a_rows = (int)std::min<int64_t>(kBM, (p.R + 7) / 8 * 8);
    p.may_cut = may_cut;
    p.part_rows = (int)std::min<int64_t>(kBM, p.R);
    p.group_m = group_of(kBM, p.K);
    CUtensorMap ma, mb0, mb1;
    if (!rows_map(&ma, a, p.R, p.K, p.a_rows) ||
        !weights_map(&mb0, b0, s.E, p.n_out, p.K, kAccCols / 2) ||
        !weights_map(&mb1, b1, s.E, p.n_out, p.K, kAccCols / 2))
        return MOE_ERR_CUDA;
    auto kern = stream_kernel<kSwiGLU>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)kSmemBytes))
        return MOE_ERR_CUDA;
    const int grid = std::min(kMaxGrid, device_sm_count());
    return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, st, ma, mb0, mb1, p) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <bool kSwiGLU>
int launch_product(const moe_shape& s, const int8_t* a, const int8_t* b0, const int8_t* b1,
                   const Params& p, cudaStream_t st) {
    switch (plan_of(s, p.K, kSwiGLU)) {
        case kCut: return launch_single<kSwiGLU>(s, a, b0, b1, p, true, st);
        case kDealt: return launch_single<kSwiGLU>(s, a, b0, b1, p, false, st);
        default: return launch_pairs<kSwiGLU>(s, a, b0, b1, p, st);
    }
}

}  // namespace int8gemm

Int8Workspace int8_workspace(const moe_shape& s) {
    using namespace int8gemm;
    const size_t R = (size_t)s.T * s.k;
    Int8Workspace w{};
    size_t off = kWsHeaderBytes;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    // counters of the tiles that may be cut, and two slots of parts for each CTA
    size_t slots = 0;
    auto counters = [&](int K, int n_out, bool swiglu) -> size_t {
        if (plan_of(s, K, swiglu) != kCut) return 0;
        const size_t cols = swiglu ? kAccCols / 2 : kAccCols;
        slots = 2 * (size_t)kMaxGrid * std::min<size_t>(kBM, R) * kAccCols * 4;
        return (R / kBM + std::min<size_t>(R, s.E)) * ((n_out + cols - 1) / cols) * kEpiWarps * 4;
    };
    w.cnt1 = take(counters(s.d, s.d_ff, true));
    w.cnt2 = take(counters(s.d_ff, s.d, false));
    w.zero_bytes = off;
    w.part = take(slots);
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
