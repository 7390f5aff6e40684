// tn_grouped_kernel: matrix products grouped by expert, ragged row ranges
// given by offsets in device memory, with both gradients.  The 8-bit kernels
// (i8_kernel.cuh) share its schedule, epilogue, split sums and operand copies.
//
// Rows t of expert e are the ones with offsets[e] <= t < offsets[e + 1].
//     product  C[t, m]     = sum_k A[e, m, k] B[t, k]
//     grad_b   dB[t, k]    = sum_m dC[t, m] A[e, m, k]
//     grad_a   dA[e, m, k] = sum_{t of e} dC[t, m] B[t, k]
// (C, dB and dA row-major; sums in FP32 in tensor memory, rounded once.)
//
// One structure for the three.  The MMA's M side ("L", TMEM lanes) runs over
// the result's contiguous index (m, k, k) and its N side ("R", TMEM columns)
// over the result's rows (t, t, m).  The N side of a tcgen05.mma takes any
// multiple of 16 (32 for a CTA pair), so a group's last tile, or a group of a
// few rows, costs MMAs of its own size, not of a whole tile's; a group's rows
// are cut into tiles of equal height.  Which index of an operand is the sum's
// decides its layout in shared memory: contiguous along the sum, it is K-major
// (rows of 128 bytes along the sum); contiguous across it, MN-major (rows of
// 64 elements across, one for each term).  The TMA writes both with the same
// 128-byte swizzle, and the tensor core reads both.
//              L                         R
//   product    A   (K-major)             B   (K-major)
//   grad_b     A   (MN-major)            dC  (K-major)
//   grad_a     B   (MN-major)            dC  (MN-major)
//
// Ragged ends: a row of another group that a box of the N side takes along
// only reaches accumulator columns that are not stored.  In grad_a the rows
// are the sum, so there the tensor maps of each group (made on the device by
// grouped_maps_kernel) end where the group ends, and the TMA fills with zeros.
//
// Roles, barriers, bounded waits and the programmatic-dependent-launch
// protocol are the general kernel's (tn_gemm_kernel.cuh): warp 0 loads, warp 1
// issues the MMAs, warps 2-9 read the accumulator and store.
//
// Measured on GB300, back to back on inputs that change.  Few rows are bound by the
// read of the weights: 8 rows over 8 of 32 experts of 2048 x 2048 15.6 us (4.3 TB/s;
// 128 tiles leave 24 SMs idle, and some 4 us are start and epilogue), 1021 rows over 16
// of 4096 x 1024 28.2 us (4.8 TB/s; 3.4 waves take the time of 4).  Weight gradients of
// few rows are bound by their stores, which alone take 37 us for 134 MB (3.6 TB/s): 32
// experts of 1024 x 2048, 3001 rows 37.5 us.  Many rows are bound by the tensor cores
// under the power cap: 16384 rows over 8 of 8192 x 4096 691 us (1590 TFLOP/s), the
// gradients 1390 (8192 rows, 14336 x 4096) and 1490 (16384 rows, 4096 x 4096).
#pragma once

#include "grouped_ptx.cuh"
#include "grouped_sinks.cuh"
#include "repack_kernel.cuh"
#include "tn_gemm_kernel.cuh"

namespace tn {

constexpr int kGrMaxExperts = 1024;
constexpr int kGrBlock = 64;                 // terms of the sum per block: 128 bytes of 16-bit elements
constexpr int kGrRaster = 8;                 // R tiles per raster group
constexpr int kGrChunk = 32;                 // accumulator columns per epilogue step
constexpr int kGrStageBytes = kGrChunk * 64; // one epilogue warp's staging: 32 rows of 32 16-bit results

// (kGrI8: the 8-bit kernels' product; tn_grouped_kernel has no such form.)  The
// others read what one of the first three reads and end otherwise (grouped_sinks.cuh).
enum GroupedOp : int {
    kGrProduct = 0, kGrGradB = 1, kGrGradA = 2, kGrI8 = 3,
    kGrGated = 4,            // a product of gate and up rows, act(gate) * up stored
    kGrLossStats = 5,        // a product whose columns' softmax statistics are stored
    kGrLossGrad = 6,         // a product whose softmax's loss gradient is stored
    kGrGradBAdd = 7,         // a token gradient in parts, added up in FP32
    kGrGradAOne = 8,         // a weight gradient of one group, times a scale
    kGrGradBScaled = 9,      // the first two gradients, times a scale
    kGrGradAScaled = 10,
    kGrLossGradLong = 11     // kGrLossGrad for sums of several segments (below)
};
constexpr int kGrOps = 12;

// The one of the first three that an operation reads its operands as.
__host__ __device__ constexpr int grouped_reads(int op)
{
    return op == kGrGated || op == kGrLossStats || op == kGrLossGrad || op == kGrLossGradLong ? kGrProduct
           : op == kGrGradBAdd || op == kGrGradBScaled ? kGrGradB
           : op == kGrGradAOne || op == kGrGradAScaled ? kGrGradA : op;
}

// Weight gradients by expert: the groups' rows have tensor maps of their own.
__host__ __device__ constexpr bool grouped_has_maps(int op) { return op == kGrGradA || op == kGrGradAScaled; }

constexpr int kI8RowsL = 128, kI8Rows = 64;  // the 8-bit kernel's tile (i8_kernel.cuh)
constexpr int kGrEpiWarps = 8;               // epilogue warps: two per quarter of the TMEM lanes
constexpr int kGrThreads = 64 + 32 * kGrEpiWarps;

// The loss's statistics hold sums in their epilogue, whose warps therefore get most of
// the registers: they are whole warpgroups (two warps before them are idle).  Sums
// of more than kGrSegment blocks are cut: the tensor cores' running sum drops what is
// below its last bit, towards zero, at every step of 16 terms, so a long sum is short
// by some 8e-10 of itself a term (measured: 3.3e-6 at 4096 terms, and 1024 at a time
// 0.9e-6), all logits alike, which the loss keeps.  The segments' sums are added in FP32,
// rounded to nearest.  The loss's gradient cuts its logits alike: it takes them against the log-sum-exp
// of the statistics' logits, and a token whose target has all but 1e-4 of the mass has a gradient of
// 1e-4, of which a logit of 30 that is 3e-6 of itself off on one side alone would leave nothing.  (Sums
// of one segment are the same in the kernel without, which is shorter: 1021 tokens over 32003 classes of 1024
// with gradients take 3.6 us less.)
template <int kOp>
struct GroupedWarps {
    static constexpr bool kSegmented = kOp == kGrLossStats || kOp == kGrLossGradLong;
    static constexpr int kEpi = kGrEpiWarps, kFirst = kSegmented ? 4 : 2;
    static constexpr int kThreads = 32 * (kFirst + kEpi), kTurns = kEpi / 4;
    // (the block's registers, shared out anew: the launch is refused where it was compiled for fewer)
    static constexpr int kRegs = 168, kRegsLead = 56, kRegsEpi = 224;
    static_assert(!kSegmented || 32 * (kFirst * kRegsLead + kEpi * kRegsEpi) <= kThreads * kRegs,
                  "no more registers than the block is launched with");
};
constexpr int kGrSegment = 16;

// kGroup CTAs compute a tile of 128 * kGroup (L) x kRows (R).  Its rows are one
// MMA N side up to 256, or (kRows = 512) two halves that share the L operand,
// the first of 256 rows: a quarter fewer bytes per MMA out of L2.  A half's
// accumulator is one of two TMEM buffers, which the halves of all tiles use in
// turn, so the epilogue of one overlaps the MMAs of the next.
template <int kGroup, int kRows>
struct GroupedCfg {
    static constexpr int kHalfRows = kRows < 256 ? kRows : 256;
    static constexpr int kHalves = kRows / kHalfRows;
    static constexpr int kRowsL = 128;                       // per CTA
    static constexpr int kRowsR = kHalfRows / kGroup;        // per CTA and half
    static constexpr int kTileL = kRowsL * kGroup;
    static constexpr int kLBytes = kRowsL * 128;
    static constexpr int kRBytes = kRowsR * 128;
    static constexpr int kBlockBytes = kLBytes + kHalves * kRBytes;
    // Blocks per stage, each with a barrier of its own that its loads complete on;
    // the stage is given back as a whole.  Two, where they fit: what a stage costs
    // beside its bytes (a wait, an election and a commit or an arming on either
    // side, some 350 cycles) is then paid half as often.
    static constexpr int kAtoms = kHalves == 1 ? 2 : 1;
    static constexpr int kStageBytes = kAtoms * kBlockBytes;
    static constexpr int kStages = 196608 / kStageBytes;
    static constexpr int kGran = 16 * kGroup;                // the MMA's N is a multiple of it
    static constexpr uint32_t kAccCols = kHalfRows;
    static constexpr uint32_t kTmemCols = 2 * kAccCols;      // two accumulators: an epilogue overlaps the next tile
    // full[S][atoms], empty[S], accfull[2], accempty[2], drain, never
    static constexpr int kNumBarriers = (kAtoms + 1) * kStages + 6;
    static constexpr int kTables = 2 * (kGrMaxExperts + 8) * 4;   // group starts, units before each group
    static constexpr int kStaging = kGrEpiWarps * kGrStageBytes;
    static constexpr int kSmemBytes = 1024 /* alignment slack */ + kStages * kStageBytes + kStaging + kNumBarriers * 8 +
                                      32 + kStages * kAtoms * 4 + kTables;
    static_assert(kSmemBytes <= 232448, "exceeds the 227 KiB shared memory of one CTA");
};

struct GroupedParams {
    // product: L {K, M, E} box {64, 128, 1}, R {K, T} boxes {64, 16 (i + 1)};
    // grad_b:  L {K, M, E} box {64, 64, 1},  R {M, T} boxes {64, 16 (i + 1)}
    CUtensorMap tmap_l, tmap_r[8];
    const CUtensorMap *group_maps;   // grad_a: [E][2], R {M, T_e} and L {K, T_e}, boxes {64, 64}
    const int32_t *offsets;          // E + 1 row starts, or NULL: one group of all T rows
    uint16_t *out;                   // row r of group e's range at out + e * out_stride + r * out_ld
    int64_t out_ld, out_stride;
    int32_t E, T;
    int32_t l_extent;                // the result's contiguous extent
    int32_t r_extent;                // grad_a: the result's rows per expert (M)
    int32_t red;                     // terms of the sum (grad_a: the group's rows instead)
    uint32_t fmt, out_fmt;           // operands and result: 0 f16, 1 bf16
    int32_t split;                   // single CTAs: a cluster of this many shares a tile's sum (1, 2, 4 or 8)
    uint32_t out_vec;                // every row of the result starts on a 16-byte boundary
    const float *scale_l;            // 8-bit product: [E][l_extent] and [T] (else NULL)
    const float *scale_r;
    uint32_t flags;                  // kFlagStall* (test hooks)
    uint64_t wait_limit_ns;
    // The operations from kGrGated on:
    int32_t tile_rows;               // rows of the result in a tile at most
    int32_t parts;                   // kGrGradBAdd: the sum's parts, each a result of its own
    SinkParams sink;
};

// Waiter::wait by a converged warp, with one answer for all its lanes.
__device__ __forceinline__ bool wait_warp(const Waiter &w, uint32_t bar, uint32_t parity, int site)
{
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *w.abort_flag != 0u)) return false;
        if (__any_sync(0xffffffffu, ptx::globaltimer() - t0 > w.limit)) {
            if (ptx::elect_one()) w.raise(site);
            __syncwarp();
            return false;
        }
    }
}

// ------------------------------------------------------------------ schedule
// Rows [start[e], start[e + 1]) belong to group e.  Offsets are read as if each
// were at least the ones before it and at most T, so a table that is not
// ascending, or that passes T, never leads outside the operands.
struct GroupedTile {
    int32_t e, l0, r0;      // group, first index of the L side, first row within the group's range
    int32_t rows;           // rows of the result in this tile
    int32_t n_mma[2];       // MMA N of either half (0: no second half)
    int32_t red;            // terms of the sum
};

// Tiles of up to r rows that `rows` rows make.  (rows + r - 1 may pass 2^31 - 1.)
__host__ __device__ constexpr int32_t row_tiles(int32_t rows, int32_t r) { return rows > 0 ? (rows - 1) / r + 1 : 0; }
static_assert(row_tiles(0x7FFFFF00, 512) == 0x400000 && row_tiles(512, 512) == 1 && row_tiles(0, 512) == 0,
              "up to 2^31 - 256 rows, the most that a call may have");

template <int kOp, int kRows, int kHalfRows, int kTileL, int kGran>
struct GroupedWalk {
    static constexpr int kReads = grouped_reads(kOp);
    static constexpr int kSpan = kOp == kGrGated ? kTileL / 2 : kTileL;    // a gated tile holds gate and up rows
    const int32_t *start, *before;      // shared memory
    int32_t l_tiles, r_extent, red;
    int32_t e;
    int32_t most = kRows;               // rows of a tile, at most

    // Tile u (u never decreases over the calls, or there is one group).
    __device__ __forceinline__ GroupedTile at(int32_t u)
    {
        while (before[e + 1] <= u) ++e;
        GroupedTile t;
        const int32_t group_rows = start[e + 1] - start[e];
        const int32_t rows = kReads == kGrGradA ? r_extent : group_rows;
        const int32_t tiles = row_tiles(rows, kOp >= kGrGated ? most : kRows);
        // the rows in steps of kGran, spread evenly: the first `more` tiles have one more
        const int32_t steps = (rows + kGran - 1) / kGran, each = steps / tiles, more = steps - each * tiles;
        int64_t tr, tl;
        tile_coord(u - before[e], tiles, l_tiles, kGrRaster, tr, tl);
        t.e = e;
        t.l0 = static_cast<int32_t>(tl) * kSpan;
        const int32_t r = static_cast<int32_t>(tr);
        t.r0 = (r * each + (r < more ? r : more)) * kGran;
        const int32_t padded = (each + (r < more ? 1 : 0)) * kGran;
        t.rows = rows - t.r0 < padded ? rows - t.r0 : padded;
        t.n_mma[0] = padded < kHalfRows ? padded : kHalfRows;
        t.n_mma[1] = padded - t.n_mma[0];
        t.red = kReads == kGrGradA ? group_rows : red;
        return t;
    }
};

// Descriptor of an MN-major operand with the 128-byte swizzle: each term's 64
// elements are a row of 128 bytes, 8 terms 1024 bytes further on (the stride
// offset), the next 64 elements across a block of kGrBlock terms further on
// (the leading offset).
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kGrBlock * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t q)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(q)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z, int32_t q)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(q)
        : "memory");
}

// Makes a tensor map that another kernel wrote usable by this thread's TMA
// instructions.
__device__ __forceinline__ void acquire_tensormap(const CUtensorMap *map)
{
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(map))
                 : "memory");
}

// The group tables in shared memory, by all threads of the CTA.
template <int kOp, int kRows, int kCtaThreads = GroupedWarps<kOp>::kThreads>
__device__ __forceinline__ void grouped_tables(const GroupedParams &p, int32_t l_tiles, int32_t *start, int32_t *before)
{
    constexpr int kReads = grouped_reads(kOp);
    const int32_t E = p.E, T = p.T, most = kOp >= kGrGated ? p.tile_rows : kRows;
    for (int32_t i = threadIdx.x; i <= E; i += kCtaThreads) {
        const int32_t o = p.offsets ? p.offsets[i] : (i == 0 ? 0 : T);
        start[i] = o < 0 ? 0 : (o > T ? T : o);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        // each lane a run of entries: the running maximum of the starts, then the
        // running sum of the groups' tiles
        const int lane = threadIdx.x;
        const int32_t per = (E + 1 + 31) / 32;
        const int32_t i0 = lane * per < E + 1 ? lane * per : E + 1;
        const int32_t i1 = i0 + per < E + 1 ? i0 + per : E + 1;
        int32_t top = 0;
        for (int32_t i = i0; i < i1; ++i) top = start[i] > top ? start[i] : top;
        int32_t run = top;
        for (int d = 1; d < 32; d *= 2) {
            const int32_t o = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d && o > run) run = o;
        }
        int32_t m = __shfl_up_sync(0xffffffffu, run, 1);
        if (lane == 0) m = 0;
        for (int32_t i = i0; i < i1; ++i) {
            m = start[i] > m ? start[i] : m;
            start[i] = m;
        }
        __syncwarp();
        int32_t sum = 0;
        for (int32_t i = i0; i < i1 && i < E; ++i) {
            const int32_t rows = kReads == kGrGradA ? p.r_extent : start[i + 1] - start[i];
            sum += row_tiles(rows, most) * l_tiles;
        }
        int32_t acc = sum;
        for (int d = 1; d < 32; d *= 2) {
            const int32_t o = __shfl_up_sync(0xffffffffu, acc, d);
            if (lane >= d) acc += o;
        }
        acc -= sum;
        for (int32_t i = i0; i < i1; ++i) {
            before[i] = acc;
            if (i < E) {
                const int32_t rows = kReads == kGrGradA ? p.r_extent : start[i + 1] - start[i];
                acc += row_tiles(rows, most) * l_tiles;
            }
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ epilogue
// The accumulator holds the result transposed (its lanes are the result's
// contiguous index).  A warp takes its 32 lanes by 32 columns as 8 x 8
// fragments, stores them transposed to its staging rows of 64 bytes, and
// writes those out 16 bytes a lane, whole 32-byte sectors.  The 16-byte pieces
// of two staging rows share a 128-byte line and are permuted within it, so that
// neither side meets a bank twice.  One warp runs this with little to overlap,
// so what counts is instructions: about 60 a step.
struct GroupedStore {
    uint32_t base;            // the warp's staging rows
    uint32_t st0, ld0;        // this lane's first staging addresses (others are fixed offsets from them)
    int lane;
    int32_t wide;             // of this warp's 32 lanes, those inside the result
    bool vec;                 // 16-byte stores: all 32 lanes, on 16-byte boundaries
    int64_t ld;               // the result's row stride, elements
    float scale_l[4];         // 8-bit product: of lanes 8 i + lane / 4

    __device__ __forceinline__ void init(uint32_t s_mine, int lane_)
    {
        base = s_mine;
        lane = lane_;
        auto piece = [&](int row, int c) {        // address of 16-byte piece c (0 .. 3) of a staging row
            return s_mine + (row >> 1) * 128 + (((((row & 1) << 2) | c) ^ ((row >> 1) & 3)) << 4);
        };
        st0 = piece(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1);
        ld0 = piece(lane >> 2, lane & 3);
    }

    // Columns v of one step, the result's rows from out on (this warp's first
    // element of the step's first row), `rows` of them to store; scale_r: the
    // scale of the step's first row.
    template <bool kBf16, bool kScaled>
    __device__ __forceinline__ void step(const uint32_t (&v)[2][16], uint16_t *out, int32_t rows,
                                         const float *scale_r) const
    {
        uint32_t h[2][4][2];                      // [half of the lanes][8 columns][8 lanes]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s0 = 1.0f, s1 = 1.0f;
            if constexpr (kScaled) {
                const int32_t r = 8 * i + 2 * (lane & 3);
                if (r < rows) s0 = __ldg(scale_r + r);
                if (r + 1 < rows) s1 = __ldg(scale_r + r + 1);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x0 = __uint_as_float(v[q >> 1][4 * i + 2 * (q & 1)]);
                float x1 = __uint_as_float(v[q >> 1][4 * i + 2 * (q & 1) + 1]);
                if constexpr (kScaled) {
                    x0 = x0 * scale_l[q] * s0;
                    x1 = x1 * scale_l[q] * s1;
                }
                h[q >> 1][i][q & 1] = kBf16 ? ptx::pack_bf16x2(x0, x1) : ptx::pack_f16x2(x0, x1);
            }
        }
        __syncwarp();                             // the last step's pieces have been read
#pragma unroll
        for (int q = 0; q < 2; ++q)               // lanes 16 q .. : pieces 2 q, 2 q + 1
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                ptx::stmatrix_x4_trans((st0 ^ (32u * q)) + 512u * i, h[q][i][0], h[q][i][1], h[q][i + 1][0],
                                       h[q][i + 1][1]);
        __syncwarp();
        if (vec) {
            uint16_t *dst = out + (lane >> 2) * ld + 8 * (lane & 3);
            if (rows >= kGrChunk) {
                uint4 x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = ptx::ld_shared_v4(ld0 + 512u * q);
#pragma unroll
                for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(dst + 8 * q * ld) = x[q];
            } else {
#pragma unroll 1
                for (int q = 0; 8 * q + (lane >> 2) < rows; ++q, dst += 8 * ld)
                    *reinterpret_cast<uint4 *>(dst) = ptx::ld_shared_v4(ld0 + 512u * q);
            }
        } else if (lane < wide) {
            // rows that are not aligned, or end inside this warp's 32: an element a lane,
            // so that a warp's store is one stretch of a row
            uint16_t *dst = out + lane;
            const int32_t n = rows < kGrChunk ? rows : kGrChunk;
#pragma unroll 8
            for (int32_t r = 0; r < n; ++r) {
                dst[r * ld] = ptx::ld_shared_u16(base + (r >> 1) * 128 +
                                                 (((((r & 1) << 2) | (lane >> 3)) ^ ((r >> 1) & 3)) << 4) + 2 * (lane & 7));
            }
        }
    }

    // The steps first, first + 2, ... of a half's columns (from TMEM address
    // t_row on; out, rows and scale_r as for step 0), the next one's columns on
    // their way while one is stored; read_all() once all have been read.
    template <bool kBf16, bool kScaled, class ReadAll>
    __device__ __forceinline__ void half(uint32_t t_row, int32_t first, int32_t steps, uint16_t *out, int32_t rows,
                                         const float *scale_r, ReadAll read_all) const
    {
        each_step(t_row, first, steps, read_all, [&](int32_t s, const uint32_t (&v)[2][16]) {
            const int32_t c = s * kGrChunk;
            step<kBf16, kScaled>(v, out + c * ld, rows - c, kScaled ? scale_r + c : nullptr);
        });
    }

    // The same, store(s, columns of step s) for each.
    template <class ReadAll, class Store>
    static __device__ __forceinline__ void each_step(uint32_t t_row, int32_t first, int32_t steps, ReadAll read_all,
                                                     Store store)
    {
        auto load = [&](int32_t s, uint32_t (&v)[2][16]) {
            ptx::tmem_ld_16x256b_x4(t_row + s * kGrChunk, v[0]);
            ptx::tmem_ld_16x256b_x4(t_row + (16u << 16) + s * kGrChunk, v[1]);
        };
        auto landed = [&](uint32_t (&v)[2][16]) {
            ptx::tmem_ld_wait_all();
            ptx::reg_dependency(v[0]);
            ptx::reg_dependency(v[1]);
        };
        uint32_t va[2][16], vb[2][16];
        int32_t s = first;
        if (s < steps) {
            load(s, va);
            landed(va);
        }
        while (true) {
            if (s + 2 >= steps) {
                read_all();
                if (s < steps) store(s, va);
                return;
            }
            load(s + 2, vb);
            store(s, va);
            landed(vb);
            s += 2;
            if (s + 2 >= steps) {
                read_all();
                store(s, vb);
                return;
            }
            load(s + 2, va);
            store(s, vb);
            landed(va);
            s += 2;
        }
    }
};

// ------------------------------------------------------------------ split sums
// Few tiles with long sums leave most SMs idle.  Then a cluster of 2, 4 or 8
// single CTAs takes a tile (and just one: the host asks for no more tiles than
// clusters), each CTA a part of the sum.  The tile's 32 x 32 pieces of the
// accumulator are shared out over the CTAs: each leaves the others' pieces of its
// own partial sum, as the registers that they are read into, in its ring, whose
// loads and MMAs are all done, and adds up its own out of the others' rings, in
// the order of the ranks, so that a result never depends on timing.
struct SplitSum {
    uint32_t ring;            // shared address, the same in every CTA
    int32_t split, rank;      // CTAs of the cluster (a power of two), this one's rank

    // Piece (quarter of the lanes, step of the columns).
    __device__ __forceinline__ bool mine(int quarter, int step) const { return ((quarter + 4 * step) & (split - 1)) == rank; }
    __device__ __forceinline__ uint32_t at(int quarter, int step, int lane) const
    {
        return ring + static_cast<uint32_t>(quarter + 4 * step) * 4096u + lane * 16u;
    }
    __device__ __forceinline__ void leave(uint32_t addr, const uint32_t (&v)[2][16]) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ptx::st_shared_v4(addr + (4 * h + i) * 512u, v[h][4 * i], v[h][4 * i + 1], v[h][4 * i + 2], v[h][4 * i + 3]);
    }
    // v: this CTA's own part of the piece, then the sum.
    __device__ __forceinline__ void add_others(uint32_t addr, uint32_t (&v)[2][16]) const
    {
        float sum[2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[h][i] = 0.0f;
#pragma unroll 1
        for (int32_t q = 0; q < split; ++q) {
            const uint32_t from = ptx::mapa_shared(addr, q);
            uint4 x[2][4];
            if (q != rank) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[h][i] = ptx::ld_cluster_v4(from + (4 * h + i) * 512u);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[h][i] = make_uint4(v[h][4 * i], v[h][4 * i + 1], v[h][4 * i + 2], v[h][4 * i + 3]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[h][4 * i] += __uint_as_float(x[h][i].x);
                    sum[h][4 * i + 1] += __uint_as_float(x[h][i].y);
                    sum[h][4 * i + 2] += __uint_as_float(x[h][i].z);
                    sum[h][4 * i + 3] += __uint_as_float(x[h][i].w);
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) v[h][i] = __float_as_uint(sum[h][i]);
    }
};

// A piece's columns out of TMEM.
__device__ __forceinline__ void load_piece(uint32_t t_addr, uint32_t (&v)[2][16])
{
    ptx::tmem_ld_16x256b_x4(t_addr, v[0]);
    ptx::tmem_ld_16x256b_x4(t_addr + (16u << 16), v[1]);
    ptx::tmem_ld_wait_all();
    ptx::reg_dependency(v[0]);
    ptx::reg_dependency(v[1]);
}

template <int kOp, int kGroup, int kRows>
__global__ void __launch_bounds__(GroupedWarps<kOp>::kThreads, 1) tn_grouped_kernel(const __grid_constant__ GroupedParams p)
{
    using Cfg = GroupedCfg<kGroup, kRows>;
    using Warps = GroupedWarps<kOp>;
    constexpr bool kSegmented = Warps::kSegmented, kShareRegs = kSegmented && kRows > 64;
    static_assert(!kSegmented || (Cfg::kHalves == 1 && kGrSegment % Cfg::kAtoms == 0), "segments are whole stages");
    constexpr int kStages = Cfg::kStages, kAtoms = Cfg::kAtoms;
    constexpr int kReads = grouped_reads(kOp);
    constexpr bool kLMajorK = kReads == kGrProduct, kRMajorK = kReads != kGrGradA;
    constexpr bool kSinks = kOp >= kGrGated;      // the epilogue is one of grouped_sinks.cuh's

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_ring = ptx::smem_addr(smem);
    const uint32_t s_staging = s_ring + kStages * Cfg::kStageBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * Cfg::kStageBytes + Cfg::kStaging);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::kNumBarriers);
    volatile uint32_t *abort_flag = tmem_holder + 1;
    volatile uint32_t *issued_count = tmem_holder + 2;    // fills this CTA's producer issued
    volatile uint32_t *producer_done = tmem_holder + 3;   // set once this CTA's producer issues no more
    // [kStages][kAtoms]: this CTA's bytes of the block in the stage's last fill
    volatile uint32_t *fill_bytes = tmem_holder + 8;
    int32_t *start = reinterpret_cast<int32_t *>(tmem_holder + 8 + kStages * kAtoms);
    int32_t *before = start + kGrMaxExperts + 8;
    const uint32_t abort_addr = ptx::smem_addr(const_cast<uint32_t *>(abort_flag));
    const uint32_t count_addr = ptx::smem_addr(const_cast<uint32_t *>(issued_count));
    const uint32_t done_addr = ptx::smem_addr(const_cast<uint32_t *>(producer_done));
    const uint32_t fill_addr = ptx::smem_addr(const_cast<uint32_t *>(fill_bytes));
    const uint32_t bar0 = ptx::smem_addr(bars);
    constexpr int kEmpty0 = kStages * kAtoms, kAcc0 = kEmpty0 + kStages;
    auto full_bar = [&](int s, int a) { return bar0 + 8u * (s * kAtoms + a); };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kEmpty0 + s); };
    auto accfull_bar = [&](int b) { return bar0 + 8u * (kAcc0 + b); };
    auto accempty_bar = [&](int b) { return bar0 + 8u * (kAcc0 + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (kAcc0 + 4);
    const uint32_t never_bar = bar0 + 8u * (kAcc0 + 5);   // nothing ever arrives (test stalls)

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t pos = kGroup == 2 ? ptx::cluster_ctarank() : 0u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            for (int a = 0; a < kAtoms; ++a) {
                ptx::mbar_init(full_bar(s, a), 1);
                fill_bytes[s * kAtoms + a] = 0u;
            }
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accfull_bar(b), 1);
            ptx::mbar_init(accempty_bar(b), Warps::kEpi * kGroup);
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::mbar_init(never_bar, 1);
        *abort_flag = 0u;
        *issued_count = 0u;
        *producer_done = 0u;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (!grouped_has_maps(kOp) && threadIdx.x == 32 && p.red > 0) {
        ptx::prefetch_tensormap(&p.tmap_l);
        ptx::prefetch_tensormap(&p.tmap_r[kReads == kGrGradA ? 0 : Cfg::kRowsR / 16 - 1]);
    }
    if (warp == 1) {
        ptx::tmem_alloc<kGroup>(ptx::smem_addr(tmem_holder), Cfg::kTmemCols);
        ptx::tmem_relinquish_alloc_permit<kGroup>();
    }
    ptx::tc_fence_before_sync();
    if constexpr (kGroup == 2)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    const Waiter w{abort_flag, abort_addr, pos, static_cast<uint32_t>(kGroup), p.wait_limit_ns};

    // Every thread's first global access is behind this wait: the offsets, and
    // in grad_a the maps, may be the previous kernel's.
    ptx::griddep_wait();
    constexpr int kSpan = kOp == kGrGated ? Cfg::kTileL / 2 : Cfg::kTileL, kCtaSpan = kSpan / kGroup;
    const int32_t l_tiles = (p.l_extent + kSpan - 1) / kSpan;
    grouped_tables<kOp, kRows>(p, l_tiles, start, before);
    constexpr bool kParts = kOp == kGrGradBAdd;
    const int32_t tiles = before[p.E], total = kParts ? tiles * p.parts : tiles;
    // (grad_a's sums are the groups' own rows: not split)
    constexpr bool kMaySplit = kGroup == 1 && kReads != kGrGradA && !kParts;
    static_assert(!kMaySplit || kRows <= 2 * kGrChunk, "the pieces of a split sum are four by two at most");
    const int32_t split = kMaySplit ? p.split : 1;
    const int32_t ctas = kGroup * split;
    const int32_t slot = static_cast<int32_t>(blockIdx.x) / ctas, slots = static_cast<int32_t>(gridDim.x) / ctas;
    const SplitSum parts{s_ring, split, split > 1 ? static_cast<int32_t>(ptx::cluster_ctarank()) : 0};
    // of the blocks of a sum of `blocks`, those before the `rank`th CTA's of the cluster, or
    // before the `rank`th part: whole stages
    auto part = [&](int32_t blocks, int32_t rank) {
        if (!kMaySplit && !kParts) return rank == 0 ? 0 : blocks;
        const int32_t stages = (blocks + kAtoms - 1) / kAtoms;
        const int32_t to = static_cast<int32_t>(static_cast<int64_t>(stages) * rank / (kParts ? p.parts : split)) * kAtoms;
        return to < blocks ? to : blocks;
    };
    GroupedWalk<kOp, kRows, Cfg::kHalfRows, Cfg::kTileL, Cfg::kGran> walk{start, before, l_tiles, p.r_extent, p.red, 0};
    if constexpr (kSinks) walk.most = p.tile_rows;
    auto tile_at = [&](int32_t u) { return walk.at(kParts ? u % tiles : u); };
    auto rank_of = [&](int32_t u) { return kParts ? u / tiles : parts.rank; };
    auto blocks_of = [](int32_t red) { return (red + kGrBlock - 1) / kGrBlock; };
    // what a sink is told beside the place: the part of the sum, or the group
    auto which = [&](const GroupedTile &t, int32_t u) { return kParts ? rank_of(u) : grouped_has_maps(kOp) ? t.e : 0; };
    // a part of a sum that is too short for all of them
    auto no_terms = [&](const GroupedTile &t, int32_t u) {
        return kParts && part(blocks_of(t.red), rank_of(u)) == part(blocks_of(t.red), rank_of(u) + 1);
    };

    bool joins = false;                           // an epilogue warp whose tile's split sum is complete here
    uint32_t kept[2][16];                         // ... of segments: its own part of its piece
    if (warp < Warps::kFirst) {
    if constexpr (kShareRegs) ptx::setmaxnreg_dec<Warps::kRegsLead>();
    if (warp == 0) {
        // ------------------------------------------------ TMA producer (every CTA)
        // A pair's loads all complete on the even CTA's full[s][a], which its own
        // producer arms with both CTAs' bytes.  A block past the end of the sum
        // (the last stage's second) is armed with no bytes.
        {
            int stage = 0;
            uint32_t phase = 0, n_issued = 0;
            bool ok = true;
            if (p.flags & (pos == 0 && parts.rank == 0 ? kFlagStallProducer0 : kFlagStallProducer1))
                ok = wait_warp(w, never_bar, 0u, kSiteStall);
            int32_t mapped = -1;
            for (int32_t u = slot; ok && u < total; u += slots) {
                const GroupedTile t = tile_at(u);
                const int32_t l0 = t.l0 + static_cast<int32_t>(pos) * kCtaSpan;
                int32_t cols[2], r0[2];       // this CTA's R elements of either half, and the first
                uint32_t r_bytes = 0;
#pragma unroll
                for (int h = 0; h < Cfg::kHalves; ++h) {
                    cols[h] = t.n_mma[h] / kGroup;
                    r0[h] = (kReads == kGrGradA ? 0 : start[t.e]) + t.r0 + h * Cfg::kHalfRows +
                            static_cast<int32_t>(pos) * cols[h];
                    r_bytes += kRMajorK ? cols[h] * 128u
                                        : static_cast<uint32_t>((cols[h] + 63) / 64) * (kGrBlock * 128u);
                }
                const uint32_t fill = Cfg::kLBytes + r_bytes;
                // (a weight gradient of one group: the call's own two maps)
                const CUtensorMap *map_l = &p.tmap_l, *map_r = p.tmap_r;
                if constexpr (grouped_has_maps(kOp)) {
                    map_r = p.group_maps + 2 * t.e;
                    map_l = map_r + 1;
                    if (t.e != mapped && t.red > 0) {
                        if (ptx::elect_one()) {       // (the lane that issues the loads)
                            acquire_tensormap(map_r);
                            acquire_tensormap(map_l);
                        }
                        __syncwarp();
                        mapped = t.e;
                    }
                }
                const int32_t sum_blocks = blocks_of(t.red);
                const int32_t begin = part(sum_blocks, rank_of(u)), blocks = part(sum_blocks, rank_of(u) + 1);
                for (int32_t i = begin; i < blocks; i += kAtoms) {
                    if (!wait_warp(w, empty_bar(stage), phase ^ 1u, kSiteEmpty)) {
                        ok = false;
                        break;
                    }
                    ++n_issued;
                    if (ptx::elect_one()) {
#pragma unroll
                    for (int a = 0; a < kAtoms; ++a) {
                        const uint32_t s_l = s_ring + stage * Cfg::kStageBytes + a * Cfg::kBlockBytes;
                        const uint32_t s_r = s_l + Cfg::kLBytes;
                        const int32_t k0 = (i + a) * kGrBlock;
                        const bool past = i + a >= blocks;
                        uint32_t bar = full_bar(stage, a);
                        fill_bytes[stage * kAtoms + a] = past ? 0u : fill;
                        if (pos == 0) ptx::mbar_arrive_expect_tx(bar, past ? 0u : kGroup * fill);
                        if (past) continue;
                        if constexpr (kGroup == 2) bar = ptx::mapa_shared(bar, 0);
                        auto load2 = [&](uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y) {
                            if constexpr (kGroup == 2)
                                ptx::tma_load_2d_pair(dst, map, bar, x, y);
                            else
                                ptx::tma_load_2d(dst, map, bar, x, y);
                        };
                        auto load3 = [&](uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z) {
                            if constexpr (kGroup == 2)
                                tma_load_3d_pair(dst, map, bar, x, y, z);
                            else
                                tma_load_3d(dst, map, bar, x, y, z);
                        };
                        if constexpr (kOp == kGrGated) {
                            // 16 gate rows, then the 16 up rows beside them, four times
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if constexpr (kGroup == 2)
                                    tma_load_4d_pair(s_l + q * 4096u, map_l, bar, k0, l0 + 16 * q, 0, t.e);
                                else
                                    tma_load_4d(s_l + q * 4096u, map_l, bar, k0, l0 + 16 * q, 0, t.e);
                            }
                        } else if constexpr (kLMajorK) {
                            load3(s_l, map_l, k0, l0, t.e);
                        } else if constexpr (kReads == kGrGradB) {
                            load3(s_l, map_l, l0, k0, t.e);
                            load3(s_l + kGrBlock * 128, map_l, l0 + 64, k0, t.e);
                        } else {
                            load2(s_l, map_l, l0, k0);
                            load2(s_l + kGrBlock * 128, map_l, l0 + 64, k0);
                        }
#pragma unroll
                        for (int h = 0; h < Cfg::kHalves; ++h) {
                            if (h > 0 && cols[h] == 0) break;
                            const uint32_t dst = s_r + h * Cfg::kRBytes;
                            if constexpr (kRMajorK) {
                                // one box of just these rows: with boxes of 16 rows a tile of 224 took
                                // twice a full one's time, with one of 128 (the next power of two a CTA)
                                // no less than a full one's
                                load2(dst, map_r + cols[h] / 16 - 1, k0, r0[h]);
                            } else {
                                load2(dst, map_r, r0[h], k0);
                                if (cols[h] > 64) load2(dst + kGrBlock * 128, map_r, r0[h] + 64, k0);
                            }
                        }
                    }
                    *issued_count = n_issued;
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // no more loads from this CTA: the next kernel may start its setup
            if (lane == 0) ptx::griddep_launch_dependents();
            if constexpr (kGroup == 2) {
                // (one lane from here on: the counts below are its own stores or released to it)
                const bool one = ptx::elect_one();
                if (one) ptx::st_release_cluster_u32(ptx::mapa_shared(done_addr, pos), 1u);
                if (one && pos == 0) {
                    // Both producers have stopped (or the limit ran out): let every load that
                    // was issued land before the pair can exit.  Loads go round the stages in
                    // order, and a stage is refilled only after the pair's MMAs read its
                    // previous fill, so the two producers are at most one fill of a stage
                    // apart.  On the normal path both issued every fill; after an abort the
                    // bytes that will not come are taken off the last fill, or the fill that
                    // this CTA did not arm is armed for the bytes that will.
                    uint32_t peer = n_issued;
                    const uint64_t t0 = ptx::globaltimer();
                    bool stopped = true;
                    while (ptx::ld_acquire_cluster_u32(ptx::mapa_shared(done_addr, 1)) == 0u) {
                        if (ptx::globaltimer() - t0 > w.limit) {
                            atomicCAS(&g_tn_status, 0, 4 | (kSitePeerDone << 8));
                            stopped = false;
                            break;
                        }
                    }
                    if (stopped) peer = ptx::ld_relaxed_cluster_u32(ptx::mapa_shared(count_addr, 1));
                    for (int s = 0; s < kStages; ++s) {
                        auto fills = [&](uint32_t n) { return n / kStages + (static_cast<uint32_t>(s) < n % kStages); };
                        const uint32_t mine = fills(n_issued), theirs = fills(peer);
                        const uint32_t last = mine > theirs ? mine : theirs;
                        if (last == 0) continue;
                        if (mine > theirs + 1 || theirs > mine + 1) {      // cannot happen; never guess
                            atomicCAS(&g_tn_status, 0, 4 | (kSiteReconcile << 8));
                            continue;
                        }
                        for (int a = 0; a < kAtoms; ++a) {
                            const int b = s * kAtoms + a;
                            if (mine > theirs && fill_bytes[b])
                                ptx::mbar_complete_tx(full_bar(s, a), fill_bytes[b]);
                            else if (theirs > mine)
                                ptx::mbar_arrive_expect_tx(
                                    full_bar(s, a), ptx::ld_relaxed_cluster_u32(ptx::mapa_shared(fill_addr + 4u * b, 1)));
                            w.drain(full_bar(s, a), (last - 1) & 1u);
                        }
                    }
                }
            } else if (ptx::elect_one()) {
                for (int s = 0; s < kStages; ++s) {
                    const uint32_t passes = n_issued / kStages + (static_cast<uint32_t>(s) < n_issued % kStages ? 1u : 0u);
                    for (int a = 0; a < kAtoms && passes; ++a) w.drain(full_bar(s, a), (passes - 1) & 1u);
                }
            }
        }
    } else if (warp == 1) {
        if (pos == 0) {
            // ------------------------------------------------ MMA issuer (even CTA of a pair)
            int stage = 0;
            uint32_t phase = 0, sub = 0;      // sub: halves so far; half `sub` uses accumulator sub % 2
            bool ok = true, issued_any = false;
            constexpr uint16_t kMask = kGroup == 2 ? 3 : 1;
            constexpr uint32_t kStepL = kLMajorK ? 2 : 128, kStepR = kRMajorK ? 2 : 128;   // 16 terms on, in 16-byte units
            if (p.flags & kFlagStallMma) ok = wait_warp(w, never_bar, 0u, kSiteStall);
            for (int32_t u = slot; ok && u < total; u += slots) {
                const GroupedTile t = tile_at(u);
                if (t.red == 0 || no_terms(t, u)) continue;
                const int halves = Cfg::kHalves == 2 && t.n_mma[1] > 0 ? 2 : 1;
                uint32_t idesc[2], d_tmem[2];
#pragma unroll
                for (int h = 0; h < Cfg::kHalves; ++h) {
                    idesc[h] = ptx::idesc_f32acc(Cfg::kTileL, static_cast<uint32_t>(t.n_mma[h]), p.fmt, p.fmt) |
                               (kLMajorK ? 0u : 1u << 15) | (kRMajorK ? 0u : 1u << 16);
                    d_tmem[h] = tmem_base + ((sub + h) & 1u) * Cfg::kAccCols;
                }
                if (!wait_warp(w, accempty_bar(sub & 1u), ((sub >> 1) & 1u) ^ 1u, kSiteAccEmpty)) break;
                ptx::tc_fence_after_sync();
                const int32_t sum_blocks = blocks_of(t.red);
                const int32_t begin = part(sum_blocks, rank_of(u)), blocks = part(sum_blocks, rank_of(u) + 1);
                // The MMAs of block i, in atom a of stage s, for half h.  Terms past the end
                // of the sum are zeros: whole steps of them are left out.
                auto issue = [&](int s, int a, int32_t i, int h) {
                    const uint32_t s_l = s_ring + s * Cfg::kStageBytes + a * Cfg::kBlockBytes;
                    const uint32_t s_r = s_l + Cfg::kLBytes + h * Cfg::kRBytes;
                    const uint64_t desc_l = kLMajorK ? ptx::desc_kmajor_sw128(s_l) : desc_mnmajor_sw128(s_l);
                    const uint64_t desc_r = kRMajorK ? ptx::desc_kmajor_sw128(s_r) : desc_mnmajor_sw128(s_r);
                    const int32_t left = t.red - i * kGrBlock;
#pragma unroll
                    for (int j = 0; j < kGrBlock / 16; ++j)
                        if (left > 16 * j)
                            ptx::mma_f16<kGroup>(d_tmem[h], desc_l + kStepL * j, desc_r + kStepR * j, idesc[h],
                                                 (kSegmented ? (i - begin) % kGrSegment : i - begin) | j ? 1u : 0u);
                };
                // A tile's second half may have to wait for the epilogue to read its
                // accumulator.  Until then stages are held with only their first half's MMAs
                // issued, at most kStages - 1 of them, so that the producer always has one to
                // fill; the held stages' second halves follow in order.
                const uint32_t bar1 = accempty_bar((sub + 1) & 1u), phase1 = (((sub + 1) >> 1) & 1u) ^ 1u;
                bool free1 = halves == 1;
                int held = 0, held_stage = 0;
                int32_t held_block = 0;
                auto flush = [&]() {
                    ptx::tc_fence_after_sync();
                    for (; held > 0; --held, ++held_block) {
                        if (ptx::elect_one()) {
                            issue(held_stage, 0, held_block, Cfg::kHalves - 1);
                            ptx::mma_commit<kGroup>(empty_bar(held_stage), kMask);
                        }
                        __syncwarp();
                        if (++held_stage == kStages) held_stage = 0;
                    }
                };
                for (int32_t i = begin; ok && i < blocks; i += kAtoms) {
                    if constexpr (kSegmented) {
                        if (i > begin && (i - begin) % kGrSegment == 0) {      // on to the other accumulator
                            if (ptx::elect_one()) ptx::mma_commit<kGroup>(accfull_bar(sub & 1u), kMask);
                            __syncwarp();
                            ++sub;
                            d_tmem[0] = tmem_base + (sub & 1u) * Cfg::kAccCols;
                            if (!wait_warp(w, accempty_bar(sub & 1u), ((sub >> 1) & 1u) ^ 1u, kSiteAccEmpty)) {
                                ok = false;
                                break;
                            }
                            ptx::tc_fence_after_sync();
                        }
                    }
#pragma unroll
                    for (int a = 0; a < kAtoms; ++a) {
                        if (!wait_warp(w, full_bar(stage, a), phase, kSiteLoaded)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after_sync();
                        if (ptx::elect_one()) {
                            issue(stage, a, i + a, 0);
                            // (a tile's last block of one half: the stage is free behind its MMAs)
                            if (Cfg::kHalves == 1 && a == kAtoms - 1) ptx::mma_commit<kGroup>(empty_bar(stage), kMask);
                        }
                        __syncwarp();
                        issued_any = true;
                    }
                    if (!ok) break;
                    if constexpr (Cfg::kHalves == 2) {
                        if (!free1) free1 = __all_sync(0xffffffffu, ptx::mbar_test_wait(bar1, phase1));
                        if (!free1 && held + 1 < kStages && i + 1 < blocks) {
                            if (held == 0) {
                                held_stage = stage;
                                held_block = i;
                            }
                            ++held;
                            if (++stage == kStages) {
                                stage = 0;
                                phase ^= 1u;
                            }
                            continue;
                        }
                        if (!free1 && !(free1 = wait_warp(w, bar1, phase1, kSiteAccEmpty))) {
                            ok = false;
                            break;
                        }
                        if (halves == 2) flush();
                        if (ptx::elect_one()) {
                            if (halves == 2) issue(stage, 0, i, 1);
                            ptx::mma_commit<kGroup>(empty_bar(stage), kMask);
                        }
                        __syncwarp();
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                for (int h = 0; h < halves; ++h, ++sub) {
                    if (ptx::elect_one()) ptx::mma_commit<kGroup>(accfull_bar(sub & 1u), kMask);
                    __syncwarp();
                }
            }
            // every MMA this thread issued completes before TMEM is freed
            if (issued_any && ptx::elect_one()) {
                ptx::mma_commit<kGroup>(drain_bar, 1);
                w.drain(drain_bar, 0u);
            }
        }
    }
    } else {
        // ------------------------------------------------ epilogue (warps 2..9, or 4..11, every CTA)
        if constexpr (kShareRegs) ptx::setmaxnreg_inc<Warps::kRegsEpi>();
        const int quarter = warp & 3;             // TMEM lanes 32*quarter .. +31 are this warp's
        const int turn = (warp - Warps::kFirst) >> 2;        // of the columns' steps, the quarter's two warps take every other one
        GroupedStore store;
        store.init(s_staging + (warp - Warps::kFirst) * kGrStageBytes, lane);
        store.ld = p.out_ld;
        uint32_t sub = 0;                         // halves so far
        bool ok = true;
        const bool out_bf16 = p.out_fmt != 0;
        for (int32_t u = slot; ok && u < total; u += slots) {
            const GroupedTile t = tile_at(u);
            if constexpr (kSegmented && kMaySplit) {
                if (split > 1) {                  // as below, its segments' sums in registers
                    const int32_t sum_blocks = blocks_of(t.red);
                    const int32_t n = part(sum_blocks, parts.rank + 1) - part(sum_blocks, parts.rank);
                    bool got = true;
                    for (int32_t i = 0; got && i < n; i += kGrSegment, ++sub) {
                        got = wait_warp(w, accfull_bar(sub & 1u), (sub >> 1) & 1u, kSiteAccFull);
                        if (!got) break;
                        ptx::tc_fence_after_sync();
                        if (turn * kGrChunk < t.n_mma[0]) {
                            uint32_t v[2][16];
                            load_piece(tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + (sub & 1u) * Cfg::kAccCols +
                                           turn * kGrChunk, v);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int x = 0; x < 16; ++x)
                                    kept[h][x] = i == 0 ? v[h][x]
                                                        : __float_as_uint(__uint_as_float(kept[h][x]) + __uint_as_float(v[h][x]));
                        }
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(accempty_bar(sub & 1u));
                    }
                    joins = got;
                    if (got && turn * kGrChunk < t.n_mma[0] && !parts.mine(quarter, turn))
                        parts.leave(parts.at(quarter, turn, lane), kept);
                    break;
                }
            }
            if (split > 1) {                      // the cluster's one tile, stored further down
                ok = joins = wait_warp(w, accfull_bar(0), 0u, kSiteAccFull);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                for (int s = turn; s * kGrChunk < t.n_mma[0]; s += 2) {
                    if (parts.mine(quarter, s)) continue;
                    uint32_t v[2][16];
                    load_piece(tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + s * kGrChunk, v);
                    parts.leave(parts.at(quarter, s, lane), v);
                }
                break;
            }
            const int32_t l0 = t.l0 + static_cast<int32_t>(pos) * kCtaSpan + kCtaSpan / 4 * quarter;   // this warp's part
            const int64_t row0 = static_cast<int64_t>(kReads == kGrGradA ? 0 : start[t.e]) + t.r0;
            uint16_t *out = p.out + t.e * p.out_stride + row0 * p.out_ld + l0;
            store.wide = p.l_extent - l0 < 32 ? p.l_extent - l0 : 32;
            store.vec = p.out_vec != 0 && store.wide == 32;
            if (t.red == 0 || no_terms(t, u)) {   // an empty sum
                if constexpr (kSinks) {
                    const uint32_t zero[2][16] = {};
                    for (int32_t c = turn * kGrChunk; c < t.rows; c += Warps::kTurns * kGrChunk)
                        Sink<kOp>::step(p, store, zero, l0, row0 + c, t.rows - c, which(t, u));
                } else if (lane < store.wide) {
                    for (int32_t r = turn; r < t.rows; r += 2) out[r * p.out_ld + lane] = 0;
                }
                continue;
            }
            if constexpr (kSegmented) {
                constexpr int kSteps = Cfg::kHalfRows / kGrChunk / Warps::kTurns > 0
                                           ? Cfg::kHalfRows / kGrChunk / Warps::kTurns : 1;
                const int32_t sum_blocks = blocks_of(t.red), steps = (t.n_mma[0] + kGrChunk - 1) / kGrChunk;
                const uint32_t t_lanes = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16);
                auto hand_back = [&]() {
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kGroup == 2)
                            ptx::mbar_arrive_remote(ptx::mapa_shared(accempty_bar(sub & 1u), 0));
                        else
                            ptx::mbar_arrive(accempty_bar(sub & 1u));
                    }
                };
                float sum[kSteps][2][16];
                for (int32_t i = 0; i < sum_blocks; i += kGrSegment, ++sub) {
                    ok = wait_warp(w, accfull_bar(sub & 1u), (sub >> 1) & 1u, kSiteAccFull);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint32_t t_acc = t_lanes + (sub & 1u) * Cfg::kAccCols;
                    const bool last = i + kGrSegment >= sum_blocks;
                    // (a sum of one segment stays where it is)
                    if (!last || i > 0) {
#pragma unroll
                        for (int q = 0; q < kSteps; ++q) {
                            const int32_t s = turn + q * Warps::kTurns;
                            if (s >= steps) break;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t addr = t_acc + (static_cast<uint32_t>(16 * h) << 16) + s * kGrChunk;
                                uint32_t v[16];
                                ptx::tmem_ld_16x256b_x4(addr, v);
                                ptx::tmem_ld_wait_all();
                                ptx::reg_dependency(v);
#pragma unroll
                                for (int x = 0; x < 16; ++x)
                                    sum[q][h][x] = i == 0 ? __uint_as_float(v[x]) : sum[q][h][x] + __uint_as_float(v[x]);
                                if (last) {       // back to where the last segment was
#pragma unroll
                                    for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(sum[q][h][x]);
                                    ptx::tmem_st_16x256b_x4(addr, v);
                                }
                            }
                        }
                        if (!last) {
                            hand_back();
                            continue;
                        }
                        ptx::tmem_st_wait();
                    }
#pragma unroll 1
                    for (int32_t s = turn; s < steps; s += Warps::kTurns) {
                        const int32_t c = s * kGrChunk;
                        uint32_t v[2][16];
                        load_piece(t_acc + c, v);
                        if (s + Warps::kTurns >= steps) hand_back();
                        Sink<kOp>::step(p, store, v, l0, row0 + c, t.rows - c, 0);
                    }
                    if (turn >= steps) hand_back();
                }
            } else {
#pragma unroll 1
            for (int half = 0; half < Cfg::kHalves; ++half) {
                const int32_t first = half * Cfg::kHalfRows;       // the half's first row within the tile
                const int32_t n_mma = half == 0 ? t.n_mma[0] : t.n_mma[1];
                if (half > 0 && n_mma == 0) break;
                ok = wait_warp(w, accfull_bar(sub & 1u), (sub >> 1) & 1u, kSiteAccFull);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint32_t t_row =
                    tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + (sub & 1u) * Cfg::kAccCols;
                const int32_t steps = (n_mma + kGrChunk - 1) / kGrChunk;
                auto hand_back = [&]() {          // this warp has read its part of the accumulator
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kGroup == 2)
                            ptx::mbar_arrive_remote(ptx::mapa_shared(accempty_bar(sub & 1u), 0));
                        else
                            ptx::mbar_arrive(accempty_bar(sub & 1u));
                    }
                };
                uint16_t *dst = out + first * p.out_ld;
                const int32_t rows = t.rows - first;
                if constexpr (kSinks)
                    GroupedStore::each_step(t_row, turn, steps, hand_back, [&](int32_t s, const uint32_t (&v)[2][16]) {
                        const int32_t c = s * kGrChunk;
                        Sink<kOp>::step(p, store, v, l0, row0 + first + c, rows - c, which(t, u));
                    });
                else if (out_bf16)
                    store.half<true, false>(t_row, turn, steps, dst, rows, nullptr, hand_back);
                else
                    store.half<false, false>(t_row, turn, steps, dst, rows, nullptr, hand_back);
                ++sub;
            }
            }
        }
    }

    __syncwarp();                // .aligned barriers below need converged warps
    if constexpr (kMaySplit) {
        if (split > 1) {
            ptx::cluster_sync();                  // every CTA's pieces are in its ring
            if (joins) {
                const int quarter = warp & 3;
                const GroupedTile t = walk.at(slot);
                const int32_t l0 = t.l0 + kCtaSpan / 4 * quarter;
                GroupedStore store;
                store.init(s_staging + (warp - Warps::kFirst) * kGrStageBytes, lane);
                store.ld = p.out_ld;
                store.wide = p.l_extent - l0 < 32 ? p.l_extent - l0 : 32;
                store.vec = p.out_vec != 0 && store.wide == 32;
                const int64_t row0 = static_cast<int64_t>(start[t.e]) + t.r0;
                uint16_t *out = p.out + row0 * p.out_ld + l0;
                for (int s = (warp - Warps::kFirst) >> 2; s * kGrChunk < t.n_mma[0]; s += Warps::kTurns) {
                    if (!parts.mine(quarter, s)) continue;
                    uint32_t v[2][16];
                    if constexpr (kSegmented) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int x = 0; x < 16; ++x) v[h][x] = kept[h][x];
                    } else {
                        load_piece(tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + s * kGrChunk, v);
                    }
                    parts.add_others(parts.at(quarter, s, lane), v);
                    const int32_t c = s * kGrChunk;
                    if constexpr (kSinks)
                        Sink<kOp>::step(p, store, v, l0, row0 + c, t.rows - c, 0);
                    else if (p.out_fmt != 0)
                        store.step<true, false>(v, out + c * p.out_ld, t.rows - c, nullptr);
                    else
                        store.step<false, false>(v, out + c * p.out_ld, t.rows - c, nullptr);
                }
            }
            __syncwarp();
        }
    }
    ptx::tc_fence_before_sync();
    if (kGroup == 2 || split > 1)
        ptx::cluster_sync();     // no CTA leaves while another may still touch its shared memory
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<kGroup>(tmem_base, Cfg::kTmemCols);
    }
}

// ------------------------------------------------------------------ grad_a's tensor maps
// maps[2 e] and maps[2 e + 1]: the rows of group e of dC and of B, as copies of
// two templates with the group's first row as base and its rows as extent.  One
// warp per group and map.
struct GroupedMapsParams {
    CUtensorMap dc, b;
    CUtensorMap *maps;
    const int32_t *offsets;
    const uint8_t *dc_base, *b_base;
    int64_t dc_row_bytes, b_row_bytes;
    int32_t E, T;
};

[[maybe_unused]] static __global__ void __launch_bounds__(32) grouped_maps_kernel(const __grid_constant__ GroupedMapsParams p)
{
    __shared__ __align__(128) CUtensorMap map;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int32_t e = static_cast<int32_t>(blockIdx.x) >> 1, lane = threadIdx.x;
    const bool second = blockIdx.x & 1;
    // the group's rows, from offsets read as the product's kernel reads them
    auto clamped = [&](int32_t i) {
        const int32_t o = p.offsets[i];
        return o < 0 ? 0 : (o > p.T ? p.T : o);
    };
    int32_t top = 0;
    for (int32_t i = lane; i <= e; i += 32) {
        const int32_t o = clamped(i);
        top = o > top ? o : top;
    }
    const int32_t first = __reduce_max_sync(0xffffffffu, top);
    const int32_t end = max(first, clamped(e + 1));
    if (first == end) return;                     // no rows: the map is not used
    const uint32_t *src = reinterpret_cast<const uint32_t *>(second ? &p.b : &p.dc);
    reinterpret_cast<uint32_t *>(&map)[lane] = src[lane];
    __syncwarp();
    const uint32_t s_map = ptx::smem_addr(&map);
    if (lane == 0) {
        const uint64_t base = reinterpret_cast<uint64_t>(second ? p.b_base + first * p.b_row_bytes
                                                                : p.dc_base + first * p.dc_row_bytes);
        asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(s_map), "l"(base)
                     : "memory");
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(s_map),
                     "r"(static_cast<uint32_t>(end - first))
                     : "memory");
    }
    __syncwarp();
    asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::
                     "l"(reinterpret_cast<uint64_t>(p.maps + 2 * e + second)),
                 "r"(s_map)
                 : "memory");
}

// ------------------------------------------------------------------ copies
// Rows that the TMA cannot address in place, copied to rows that start on 64-byte
// boundaries, the padding zeroed, and 8-bit tokens widened to f16 on the way where the
// kernel wants them so: row r of the copy is row r % rows_per of block r / rows_per.
template <typename Src>
struct WidenJob {
    const Src *src;
    int64_t ld, stride;
    uint8_t *dst;
    int64_t units, unit_bytes;   // 16-byte source units of a row, padding included; bytes of one in the copy
    int64_t rows_per, rows, cols;
    int32_t shift;       // 1 << shift lanes of a warp to a row
    int64_t segs, work;  // segments (kWidenSeg units) of a row; warps' shares in all
    const char *end;     // one past the last row's last element
    const int32_t *offsets;   // blocks are the experts' and only those with rows are read; or NULL
};

// Four 8-bit integers to four halves, exactly.
__device__ __forceinline__ uint32_t f16x2_minus_1152(uint32_t v)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x64806480u));
    return r;
}

// (An integer in the low bits of a float whose exponent makes them its units is a known
// trick.)  In the order 0, 2, 1, 3: what bounds the widening is the integer pipe, and a
// mask is cheaper than byte permutations.  All operands are widened alike, so
// each product still pairs a term with its own.
__device__ __forceinline__ uint2 i8x4_to_f16x4(uint32_t w)
{
    // x ^ 0x80 = x + 128 in the low bits of 1024's mantissa is 1152 + x
    uint32_t a, b;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(a) : "r"(w), "r"(0x00FF00FFu), "r"(0x64806480u));
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(b) : "r"(w >> 8), "r"(0x00FF00FFu), "r"(0x64806480u));
    return make_uint2(f16x2_minus_1152(a), f16x2_minus_1152(b));
}

constexpr int kWidenThreads = 256;
constexpr int kWidenSeg = 256;                   // units (16 source bytes) of a warp's share of a row at most

// Both operands in one launch (either may have no rows).  A warp's share is up to
// 256 units of one row, or several short rows side by side; what is worked out
// for a row is worked out once for all of them.  A row starts wherever its
// elements do, so a unit is cut out of two aligned 16-byte loads, and what it
// took along past the row's end is masked.  Units whose loads would leave the
// operand (its first and last ones) are gathered element by element: none reads
// a byte before its first or after its last element.
template <typename Src>
__global__ void __launch_bounds__(kWidenThreads, 5) widen_rows_kernel(const __grid_constant__ WidenJob<Src> j0,
                                                                      const __grid_constant__ WidenJob<Src> j1)
{
    constexpr int kElems = 16 / sizeof(Src);     // of a unit
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();            // they start once the last of these CTAs has
    const int lane = threadIdx.x & 31;
    const int64_t work = j0.work + j1.work, step = static_cast<int64_t>(gridDim.x) * (kWidenThreads / 32);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kWidenThreads / 32) + (threadIdx.x >> 5); i < work; i += step) {
        const WidenJob<Src> &j = i < j0.work ? j0 : j1;
        const int64_t n = i < j0.work ? i : i - j0.work;
        int64_t first = n, seg = 0;              // the warp's first row (shift 5: the row), its segment
        if (j.segs > 1) {
            first = j.work <= 0xFFFFFFFFll ? static_cast<uint32_t>(n) / static_cast<uint32_t>(j.segs) : n / j.segs;
            seg = n - first * j.segs;
        }
        const int64_t r = (first << (5 - j.shift)) + (lane >> j.shift);
        if (r >= j.rows) continue;
        int64_t e = 0;
        if (j.rows != j.rows_per)                // several blocks
            e = j.rows <= 0xFFFFFFFFll ? static_cast<uint32_t>(r) / static_cast<uint32_t>(j.rows_per) : r / j.rows_per;
        // Rows of expert e run from the largest offset up to its own to the next one,
        // if that is larger: it has none where the next is not above its own.
        // Nothing reads that part of the copy.
        if (j.offsets && max(j.offsets[e + 1], 0) <= max(j.offsets[e], 0)) continue;
        const int64_t u0 = seg * kWidenSeg;      // the share's first unit of its row(s)
        const Src *src = j.src + e * j.stride + (r - e * j.rows_per) * j.ld + u0 * kElems;
        uint8_t *dst = j.dst + (r * j.units + u0) * j.unit_bytes;
        // within the share 32 bits count elements and units
        const int64_t left = j.cols - u0 * kElems, room = j.units - u0;
        const int32_t cols = static_cast<int32_t>(left < kWidenSeg * kElems ? (left > 0 ? left : 0) : kWidenSeg * kElems);
        const int32_t units = static_cast<int32_t>(room < kWidenSeg ? room : kWidenSeg);
        const int32_t s = static_cast<int32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
        const uint4 *aligned = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(src) - s);
        const int32_t bytes = cols * static_cast<int32_t>(sizeof(Src)), lanes = 1 << j.shift;
        const uint32_t sh = 8u * (s & 3);
        // units whose aligned loads stay inside the operand: from lo on, below hi
        const char *begin = reinterpret_cast<const char *>(j.src);
        const int32_t lo = reinterpret_cast<const char *>(aligned) < begin ? 1 : 0;
        const int64_t whole = (j.end - reinterpret_cast<const char *>(aligned)) / 16 - (s == 0 ? 0 : 1);
        const int32_t hi = static_cast<int32_t>(whole < units ? whole : units);
#pragma unroll 2
        for (int32_t c = lane & (lanes - 1); c < units; c += lanes) {
            const int32_t valid = bytes - 16 * c;            // of this unit's bytes
            uint4 x = make_uint4(0, 0, 0, 0);
            if (valid > 0 && c >= lo && c < hi) {
                x = __ldg(aligned + c);
                if (s != 0) {
                    const uint4 y = __ldg(aligned + c + 1);
                    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                    switch (s >> 2) {
                    case 0: x = window16<0>(w, sh); break;
                    case 1: x = window16<1>(w, sh); break;
                    case 2: x = window16<2>(w, sh); break;
                    default: x = window16<3>(w, sh); break;
                    }
                }
                if (valid < 16) {
                    auto keep = [valid](int32_t first) {     // mask of the word from byte `first` on
                        const int32_t n = valid - first;
                        return n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                    };
                    x.x &= keep(0);
                    x.y &= keep(4);
                    x.z &= keep(8);
                    x.w &= keep(12);
                }
            } else if (valid > 0) {
                union {
                    Src v[kElems];
                    uint4 u4;
                } part;
                part.u4 = x;
#pragma unroll
                for (int q = 0; q < kElems; ++q)
                    if (c * kElems + q < cols) part.v[q] = src[c * kElems + q];
                x = part.u4;
            }
            uint4 *to = reinterpret_cast<uint4 *>(dst + c * static_cast<int32_t>(j.unit_bytes));
            if (sizeof(Src) == 1 && j.unit_bytes == 32) {    // to f16
                const uint2 a = i8x4_to_f16x4(x.x), b = i8x4_to_f16x4(x.y), d = i8x4_to_f16x4(x.z), f = i8x4_to_f16x4(x.w);
                to[0] = make_uint4(a.x, a.y, b.x, b.y);
                to[1] = make_uint4(d.x, d.y, f.x, f.y);
            } else {
                to[0] = x;
            }
        }
    }
}

}  // namespace tn
