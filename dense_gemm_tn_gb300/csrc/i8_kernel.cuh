// tn_i8_kernel: the 8-bit integer product (dense, or grouped by expert) for few
// rows per expert, where the read of the weights is what counts, and for few tiles.
//
//     C[t, m] = (sum_k A[e, m, k] B[t, k]) scale_a[e, m] scale_b[t]
//
// The weights are read once, as the 8-bit integers they are, and widened to f16
// (exactly) on the way to the tensor core: GB300 multiplies f16 an order of
// magnitude faster than 8-bit integers.  Widening them in a kernel of its own
// would move five bytes per weight instead of one.
//
// Per CTA: 128 weights' rows (MMA M) by up to 64 tokens (MMA N), single CTAs.
// Warp 0 loads 8-bit tiles of 128 terms by TMA; warps 6-13 widen the weights
// into tensor memory, from where the MMAs of warp 1 take their A operand, and
// the tokens into shared memory (two K-major 128B-swizzled blocks of 64 terms);
// warps 2-5 scale and store.  With the weights widened into shared memory as
// well, a stage's 108 KiB of shared-memory traffic (load, read, write, the
// MMAs' reads) bound it: 820 cycles a stage, against 44 KiB this way.
// Schedule, ragged ends, bounded waits, split sums and the epilogue's steps are the
// grouped kernel's.
//
// Measured on GB300: 16 experts of 4096 x 2048, 515 rows 32.5 us (4.3 TB/s).  512 tiles are
// 3.4 waves and take the time of 4; and between a tile's ends a stage takes 0.43 us from
// memory (8192 x 16 on 128 CTAs, K = 4096 -> 8192: 11.6 -> 18.4 us, 4.9 TB/s; out of L2 0.33
// us a stage).  8192 x 16 x 2048 9.0 us replayed from a graph, where start, epilogue and the
// join of two half sums are some 6 of them (10.7 us called from Python, whose host time
// bounds it); 1024 x 16 x 8192 10.3 us on 64 CTAs.
#pragma once

#include "grouped_kernel.cuh"

namespace tn {

constexpr int kI8EpiWarps = 4;
constexpr int kI8WidenWarps = 8;                             // two teams, which take stages in turn
constexpr int kI8TeamWarps = kI8WidenWarps / 2;
constexpr int kI8Threads = 32 * (2 + kI8EpiWarps + kI8WidenWarps);
constexpr int kI8Block = 128;                                // terms per 8-bit stage: 128 bytes

constexpr int kI8RowsL = 128, kI8Rows = 64;
constexpr int kI8Stage8Bytes = (kI8RowsL + kI8Rows) * 128;   // 8-bit stage: L, then R
constexpr int kI8Stages8 = 6;
constexpr int kI8HalfBytes = kI8Rows * 128;                  // 64 terms of R as f16
constexpr int kI8Stage16Bytes = 2 * kI8HalfBytes;
constexpr int kI8Stages16 = 2;                               // one per team
// TMEM columns: two accumulators, the two f16 stages of L (two terms a column), and
// the sums of runs
constexpr uint32_t kI8ACol0 = 2 * kI8Rows, kI8ACols = kI8Block / 2;
constexpr uint32_t kI8SumCol0 = kI8ACol0 + kI8Stages16 * kI8ACols;
constexpr uint32_t kI8TmemCols = 512;
static_assert(kI8SumCol0 + kI8Rows <= kI8TmemCols, "the TMEM columns of an SM");
// full8[S8], empty8[S8], full16[S16], empty16[S16], accfull[2], accempty[2], drain, never
constexpr int kI8Barriers = 2 * kI8Stages8 + 2 * kI8Stages16 + 6;
constexpr int kI8SmemBytes = 1024 /* alignment slack */ + kI8Stages8 * kI8Stage8Bytes + kI8Stages16 * kI8Stage16Bytes +
                             kI8EpiWarps * kGrStageBytes + kI8Barriers * 8 + 32 + 2 * (kGrMaxExperts + 8) * 4;
static_assert(kI8SmemBytes <= 232448, "exceeds the 227 KiB shared memory of one CTA");

// A tensor core's FP32 sum of 8-bit products is exact while it stays within 2^24,
// which 1024 terms of at most 2^14 each do not leave.  So an accumulator takes a run
// of that many terms and no more: the epilogue adds it to the tile's sum, an integer,
// while the MMAs of the next run go on in the other accumulator.  kI8MaxExact terms
// stay in 32 bits.  The runs of a longer sum are rounded to whole units of 2^s, s > 0,
// so that it does, 2^s being less than a 32768th of the number of terms.
//
// Measured on GB300 against one accumulator for the whole sum, which was off by 1100 in
// sums of 10000 whose halves of 16384 terms cancel: single CTAs 8192 x 16 x 2048 and
// 1024 x 16 x 8192 no difference, 4096 x 192 x 8192 29.8 -> 30.9 us; pairs, K up to 1024,
// no difference, 8192 x 4096 x 8192 313 -> 325, 8 experts of 4096 x 2048 with 4096 rows
// 57.9 -> 62.5.  What it costs there is the widening warps' share of the SM, which have no
// time to spare.  (Sums kept in floats until one comes to 2^24, read with 32-lane loads,
// or held by twelve warps instead of eight were all slower.)
constexpr int kI8Run = 1024 / kI8Block;                      // stages
constexpr int32_t kI8MaxExact = 131071;                      // * 2^14 < 2^31

// 2^-s for a sum of `red` terms.
__device__ __forceinline__ float sum_unit(int32_t red)
{
    int s = 0;
    if (red > kI8MaxExact)
        while (red >> s > 65536) ++s;
    return __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
}

// A piece of a run's sums (floats) as integers, and of a tile's sum as floats.
__device__ __forceinline__ void piece_to_ints(uint32_t (&v)[2][16], float unit)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h][i] = static_cast<uint32_t>(__float2int_rn(__uint_as_float(v[h][i]) * unit));
}

__device__ __forceinline__ void piece_to_floats(uint32_t (&v)[2][16], float unit)
{
    const float back = 1.0f / unit;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h][i] = __float_as_uint(__int2float_rn(static_cast<int32_t>(v[h][i])) * back);
}

// What the CTAs of a cluster left of their parts of a piece at `addr` of their rings,
// added up.
__device__ __forceinline__ void join_piece(const SplitSum &parts, uint32_t addr, uint32_t (&v)[2][16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h][i] = 0u;
#pragma unroll 1
    for (int32_t q = 0; q < parts.split; ++q) {
        const uint32_t from = ptx::mapa_shared(addr, q);
        uint4 x[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[h][i] = ptx::ld_cluster_v4(from + (4 * h + i) * 512u);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[h][4 * i] += x[h][i].x;
                v[h][4 * i + 1] += x[h][i].y;
                v[h][4 * i + 2] += x[h][i].z;
                v[h][4 * i + 3] += x[h][i].w;
            }
    }
}

// A piece's columns to TMEM, from where this warp alone takes them back.
__device__ __forceinline__ void store_piece(uint32_t t_addr, const uint32_t (&v)[2][16])
{
    ptx::tmem_st_16x256b_x4(t_addr, v[0]);
    ptx::tmem_st_16x256b_x4(t_addr + (16u << 16), v[1]);
    ptx::tmem_st_wait();
}

// A lane's row of L, 128 8-bit terms of a swizzled tile, to its TMEM lane's 64
// columns at t_a; v: its first four 16-byte pieces, loaded before.
template <int kPieces = 4>
__device__ __forceinline__ void widen_row_to_tmem(uint32_t row_addr, int lane, uint4 (&v)[4], uint32_t t_a)
{
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int part = 0; part < 4; part += kPieces) {
            uint32_t f[8 * kPieces];
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const uint32_t words[4] = {v[part + c].x, v[part + c].y, v[part + c].z, v[part + c].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint2 x = i8x4_to_f16x4(words[q]);
                    f[8 * c + 2 * q] = x.x;
                    f[8 * c + 2 * q + 1] = x.y;
                }
            }
            if (half == 0) {
#pragma unroll
                for (int c = part; c < part + kPieces; ++c) v[c] = ptx::ld_shared_v4(row_addr + (((4 + c) ^ (lane & 7)) << 4));
            }
            if constexpr (kPieces == 4)
                ptx::tmem_st_32x32b_x32(t_a + 32 * half, f);
            else
                ptx::tmem_st_32x32b_x16(t_a + 32 * half + 8 * part, f);
        }
    }
}

// A lane's part of widening eight rows (r0 .. r0 + 7) of a swizzled 8-bit tile
// into the two swizzled f16 blocks: 16 terms of each 64-term half, two 16-byte
// loads and four 16-byte stores.  An odd row does half 1 first, so that the two
// rows of a shared-memory pass meet no bank twice, in the loads or the stores.
struct WidenRows {
    uint32_t ld[2], st[2];        // offsets of the piece done first and second: its load, its first store

    __device__ __forceinline__ explicit WidenRows(int lane)
    {
        const int row = lane >> 2, c = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int half = (row & 1) ^ i;
            ld[i] = row * 128 + (((4 * half + c) ^ row) << 4);
            st[i] = half * kI8HalfBytes + row * 128 + (((2 * c) ^ row) << 4);
        }
    }
    __device__ __forceinline__ void store(uint32_t dst, int i, const uint4 &w) const
    {
        const uint2 a = i8x4_to_f16x4(w.x), b = i8x4_to_f16x4(w.y), d = i8x4_to_f16x4(w.z), e = i8x4_to_f16x4(w.w);
        ptx::st_shared_v4(dst + st[i], a.x, a.y, b.x, b.y);
        ptx::st_shared_v4(dst + (st[i] ^ 16u), d.x, d.y, e.x, e.y);
    }
};

__global__ void __launch_bounds__(kI8Threads, 1) tn_i8_kernel(const __grid_constant__ GroupedParams p)
{
    constexpr int kS8 = kI8Stages8, kS16 = kI8Stages16;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_ring8 = ptx::smem_addr(smem), s_ring16 = s_ring8 + kS8 * kI8Stage8Bytes;
    const uint32_t s_staging = s_ring16 + kS16 * kI8Stage16Bytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kS8 * kI8Stage8Bytes + kS16 * kI8Stage16Bytes + kI8EpiWarps * kGrStageBytes);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + kI8Barriers);
    volatile uint32_t *abort_flag = tmem_holder + 1;
    int32_t *start = reinterpret_cast<int32_t *>(tmem_holder + 8);
    int32_t *before = start + kGrMaxExperts + 8;
    const uint32_t abort_addr = ptx::smem_addr(const_cast<uint32_t *>(abort_flag));
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full8_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty8_bar = [&](int s) { return bar0 + 8u * (kS8 + s); };
    auto full16_bar = [&](int s) { return bar0 + 8u * (2 * kS8 + s); };
    auto empty16_bar = [&](int s) { return bar0 + 8u * (2 * kS8 + kS16 + s); };
    constexpr int kAcc0 = 2 * kS8 + 2 * kS16;
    auto accfull_bar = [&](int b) { return bar0 + 8u * (kAcc0 + b); };
    auto accempty_bar = [&](int b) { return bar0 + 8u * (kAcc0 + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (kAcc0 + 4);
    const uint32_t never_bar = bar0 + 8u * (kAcc0 + 5);   // nothing ever arrives (test stalls)

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kS8; ++s) {
            ptx::mbar_init(full8_bar(s), 1);
            ptx::mbar_init(empty8_bar(s), kI8TeamWarps);
        }
        for (int s = 0; s < kS16; ++s) {
            ptx::mbar_init(full16_bar(s), kI8TeamWarps);
            ptx::mbar_init(empty16_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accfull_bar(b), 1);
            ptx::mbar_init(accempty_bar(b), kI8EpiWarps);
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::mbar_init(never_bar, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (threadIdx.x == 32 && p.red > 0) {
        ptx::prefetch_tensormap(&p.tmap_l);
        ptx::prefetch_tensormap(&p.tmap_r[0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc<1>(ptx::smem_addr(tmem_holder), kI8TmemCols);
        ptx::tmem_relinquish_alloc_permit<1>();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    const Waiter w{abort_flag, abort_addr, 0u, 1u, p.wait_limit_ns};

    ptx::griddep_wait();                      // every thread's first global access is behind this wait
    const int32_t l_tiles = (p.l_extent + kI8RowsL - 1) / kI8RowsL;
    grouped_tables<kGrI8, kI8Rows, kI8Threads>(p, l_tiles, start, before);
    const int32_t total = before[p.E];
    const int32_t split = p.split;
    const int32_t slot = static_cast<int32_t>(blockIdx.x) / split, slots = static_cast<int32_t>(gridDim.x) / split;
    const SplitSum parts{s_ring8, split, split > 1 ? static_cast<int32_t>(ptx::cluster_ctarank()) : 0};
    GroupedWalk<kGrI8, kI8Rows, kI8Rows, kI8RowsL, 16> walk{start, before, l_tiles, 0, p.red, 0};
    // 8-bit stages of a tile, this CTA's being those from begin on, below blocks
    const int32_t sum_blocks = (p.red + kI8Block - 1) / kI8Block;
    const int32_t begin = sum_blocks * parts.rank / split, blocks = sum_blocks * (parts.rank + 1) / split;
    const bool sums = sum_blocks > kI8Run;    // sums of several runs, as integers
    const float unit = sum_unit(p.red);
    bool joins = false;                       // an epilogue warp whose tile's split sum is complete here

    GroupedStore store;
    // an epilogue warp's part of the result, with its scales
    auto aim = [&](const GroupedTile &t, int quarter) {
        const int32_t l0 = t.l0 + 32 * quarter;
        store.init(s_staging + (warp - 2) * kGrStageBytes, lane);
        store.ld = p.out_ld;
        store.wide = p.l_extent - l0 < 32 ? p.l_extent - l0 : 32;
        store.vec = p.out_vec != 0 && store.wide == 32;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store.scale_l[i] = 8 * i + (lane >> 2) < store.wide
                                   ? __ldg(p.scale_l + static_cast<int64_t>(t.e) * p.l_extent + l0 + 8 * i + (lane >> 2))
                                   : 0.0f;
        return p.out + (static_cast<int64_t>(start[t.e]) + t.r0) * p.out_ld + l0;
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0, n_issued = 0;
        bool ok = true;
        if (p.flags & (parts.rank == 0 ? kFlagStallProducer0 : kFlagStallProducer1))
            ok = wait_warp(w, never_bar, 0u, kSiteStall);
        for (int32_t u = slot; ok && u < total; u += slots) {
            const GroupedTile t = walk.at(u);
            const CUtensorMap *map_r = p.tmap_r + t.n_mma[0] / 16 - 1;
            const int32_t r0 = start[t.e] + t.r0;
            const uint32_t fill = static_cast<uint32_t>(kI8RowsL + t.n_mma[0]) * 128u;
            for (int32_t i = begin; i < blocks; ++i) {
                if (!wait_warp(w, empty8_bar(stage), phase ^ 1u, kSiteEmpty)) {
                    ok = false;
                    break;
                }
                if (ptx::elect_one()) {
                    const uint32_t s_l = s_ring8 + stage * kI8Stage8Bytes;
                    ptx::mbar_arrive_expect_tx(full8_bar(stage), fill);
                    tma_load_3d(s_l, &p.tmap_l, full8_bar(stage), i * kI8Block, t.l0, t.e);
                    ptx::tma_load_2d(s_l + kI8RowsL * 128, map_r, full8_bar(stage), i * kI8Block, r0);
                }
                __syncwarp();
                ++n_issued;
                if (++stage == kS8) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) ptx::griddep_launch_dependents();
        if (ptx::elect_one())
            for (int s = 0; s < kS8; ++s) {       // every issued load lands before the CTA can exit
                const uint32_t passes = n_issued / kS8 + (static_cast<uint32_t>(s) < n_issued % kS8 ? 1u : 0u);
                if (passes) w.drain(full8_bar(s), (passes - 1) & 1u);
            }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        int stage = 0;
        uint32_t phase = 0, sub = 0;              // sub: runs so far; run `sub` uses accumulator sub % 2
        bool ok = true, issued_any = false;
        if (p.flags & kFlagStallMma) ok = wait_warp(w, never_bar, 0u, kSiteStall);
        for (int32_t u = slot; ok && p.red > 0 && u < total; u += slots) {
            const GroupedTile t = walk.at(u);
            const uint32_t idesc = ptx::idesc_f32acc(kI8RowsL, static_cast<uint32_t>(t.n_mma[0]), 0u, 0u);
            for (int32_t i = begin, run = 0; i < blocks; ++i) {      // run: stages of the run so far
                const uint32_t d_tmem = tmem_base + (sub & 1u) * kI8Rows;
                if ((run == 0 && !wait_warp(w, accempty_bar(sub & 1u), ((sub >> 1) & 1u) ^ 1u, kSiteAccEmpty)) ||
                    !wait_warp(w, full16_bar(stage), phase, kSiteLoaded)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after_sync();
                const int32_t left = p.red - i * kI8Block;
                const bool last = i + 1 == blocks || run + 1 == kI8Run;
                if (ptx::elect_one()) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t desc_r =
                            ptx::desc_kmajor_sw128(s_ring16 + stage * kI8Stage16Bytes + half * kI8HalfBytes);
                        const uint32_t a_tmem = tmem_base + kI8ACol0 + stage * kI8ACols + half * (kI8ACols / 2);
#pragma unroll
                        for (int j = 0; j < kGrBlock / 16; ++j)
                            if (left > half * kGrBlock + 16 * j)
                                ptx::mma_f16_ts<1>(d_tmem, a_tmem + 8 * j, desc_r + 2u * j, idesc,
                                                (run | half | j) != 0 ? 1u : 0u);
                    }
                    ptx::mma_commit<1>(empty16_bar(stage));
                    if (last) ptx::mma_commit<1>(accfull_bar(sub & 1u));
                }
                __syncwarp();
                issued_any = true;
                ++run;
                if (last) {
                    run = 0;
                    ++sub;
                }
                if (++stage == kS16) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
        }
        if (issued_any && ptx::elect_one()) {     // every MMA issued completes before TMEM is freed
            ptx::mma_commit<1>(drain_bar);
            w.drain(drain_bar, 0u);
        }
    } else if (warp < 2 + kI8EpiWarps) {
        // ------------------------------------------------ epilogue (warps 2..5)
        const int quarter = warp & 3;
        uint32_t sub = 0;
        for (int32_t u = slot; u < total; u += slots) {
            const GroupedTile t = walk.at(u);
            const int64_t row0 = static_cast<int64_t>(start[t.e]) + t.r0;
            uint16_t *out = aim(t, quarter);
            if (p.red == 0) {                     // an empty sum
                if (lane < store.wide)
                    for (int32_t r = 0; r < t.rows; ++r) out[r * p.out_ld + lane] = 0;
                continue;
            }
            const uint32_t t_lanes = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16);
            bool ok = true;
            for (int32_t i = begin; i < blocks; i += kI8Run, ++sub) {
                const bool last = i + kI8Run >= blocks;
                ok = wait_warp(w, accfull_bar(sub & 1u), (sub >> 1) & 1u, kSiteAccFull);
                if (!ok) break;
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int32_t c = 0; c < t.n_mma[0]; c += kGrChunk) {
                    uint32_t v[2][16];
                    load_piece(t_lanes + (sub & 1u) * kI8Rows + c, v);
                    if (c + kGrChunk >= t.n_mma[0]) {
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(accempty_bar(sub & 1u));
                    }
                    if (sums) {
                        piece_to_ints(v, unit);
                        if (i > begin) {
                            uint32_t so_far[2][16];
                            load_piece(t_lanes + kI8SumCol0 + c, so_far);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int q = 0; q < 16; ++q) v[h][q] += so_far[h][q];
                        }
                        if (!last) {
                            store_piece(t_lanes + kI8SumCol0 + c, v);
                            continue;
                        }
                        if (split > 1) {          // the cluster's one tile, stored further down
                            parts.leave(parts.at(quarter, c / kGrChunk, lane), v);
                            continue;
                        }
                        piece_to_floats(v, unit);
                    }
                    if (p.out_fmt != 0)
                        store.step<true, true>(v, out + c * p.out_ld, t.rows - c, p.scale_r + row0 + c);
                    else
                        store.step<false, true>(v, out + c * p.out_ld, t.rows - c, p.scale_r + row0 + c);
                }
            }
            if (!ok) break;
            joins = split > 1;
            if (joins) break;
        }
    } else {
        // ------------------------------------------------ widening (warps 6..13)
        // Two teams of four warps take the stages in turn, each into an f16 stage of
        // its own: while one waits, loads or stores, the other has the integer pipe.
        // A warp widens the 32 rows of L that are its quarter of the TMEM lanes, a row
        // a lane, and its share of R's groups of eight rows.
        const int team = (warp - 2 - kI8EpiWarps) / kI8TeamWarps, mine = (warp - 2 - kI8EpiWarps) % kI8TeamWarps;
        static_assert(kS16 == 2 && kS8 % 2 == 0, "a team's stages are every other one");
        const int quarter = warp & 3;
        const WidenRows widen(lane);
        const uint32_t row_l = static_cast<uint32_t>(32 * quarter + lane) * 128u;
        const uint32_t t_a = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + kI8ACol0 + team * kI8ACols;
        const uint32_t dst = s_ring16 + team * kI8Stage16Bytes + mine * 1024;
        constexpr int kOwnR = kI8Rows / 8 / kI8TeamWarps;     // groups of R a warp has at most
        bool ok = true;
        int stage8 = team;
        uint32_t phase8 = 0, phase16 = 0, n = 0;              // n: stages so far
        for (int32_t u = slot; ok && p.red > 0 && u < total; u += slots) {
            const int32_t groups_r = walk.at(u).n_mma[0] / 8;
            for (int32_t i = begin; i < blocks; ++i, ++n) {
                if ((n & 1u) != static_cast<uint32_t>(team)) continue;
                ok = wait_warp(w, full8_bar(stage8), phase8, kSiteLoaded);
                if (!ok) break;
                const uint32_t src = s_ring8 + stage8 * kI8Stage8Bytes;
                uint4 v[4], r[kOwnR][2];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = ptx::ld_shared_v4(src + row_l + ((c ^ (lane & 7)) << 4));
#pragma unroll
                for (int g = 0; g < kOwnR; ++g)
                    if (mine + g * kI8TeamWarps < groups_r) {
                        const uint32_t at = src + (kI8RowsL + 8 * (mine + g * kI8TeamWarps)) * 128;
                        r[g][0] = ptx::ld_shared_v4(at + widen.ld[0]);
                        r[g][1] = ptx::ld_shared_v4(at + widen.ld[1]);
                    }
                ok = wait_warp(w, empty16_bar(team), phase16 ^ 1u, kSiteEmpty);
                if (!ok) break;
                ptx::tc_fence_after_sync();                   // the MMAs that read this stage are done
                widen_row_to_tmem(src + row_l, lane, v, t_a);
#pragma unroll
                for (int g = 0; g < kOwnR; ++g)
                    if (mine + g * kI8TeamWarps < groups_r) {
                        widen.store(dst + g * kI8TeamWarps * 1024, 0, r[g][0]);
                        widen.store(dst + g * kI8TeamWarps * 1024, 1, r[g][1]);
                    }
                ptx::fence_proxy_async_smem();                // the MMAs read what was stored
                ptx::tmem_st_wait();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(full16_bar(team));
                    ptx::mbar_arrive(empty8_bar(stage8));
                }
                phase16 ^= 1u;
                stage8 += 2;
                if (stage8 >= kS8) {
                    stage8 -= kS8;
                    phase8 ^= 1u;
                }
            }
        }
    }

    __syncwarp();                // .aligned barriers below need converged warps
    if (split > 1) {
        ptx::cluster_sync();                  // every CTA's pieces are in its ring
        if (joins) {
            const int quarter = warp & 3;
            const GroupedTile t = walk.at(slot);
            const int64_t row0 = static_cast<int64_t>(start[t.e]) + t.r0;
            uint16_t *out = aim(t, quarter);
            for (int s = 0; s * kGrChunk < t.n_mma[0]; ++s) {
                if (!parts.mine(quarter, s)) continue;
                const int32_t c = s * kGrChunk;
                uint32_t v[2][16];
                join_piece(parts, parts.at(quarter, s, lane), v);
                piece_to_floats(v, unit);
                if (p.out_fmt != 0)
                    store.step<true, true>(v, out + c * p.out_ld, t.rows - c, p.scale_r + row0 + c);
                else
                    store.step<false, true>(v, out + c * p.out_ld, t.rows - c, p.scale_r + row0 + c);
            }
        }
        __syncwarp();
    }
    ptx::tc_fence_before_sync();
    if (split > 1)
        ptx::cluster_sync();     // no CTA leaves while another reads its ring
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<1>(tmem_base, kI8TmemCols);
    }
}

// ------------------------------------------------------------------ many rows
// tn_i8_pair_kernel: the same product on CTA pairs, for many rows per expert.
// The weights are again widened on the way, each CTA's 128 rows into its own
// tensor memory; the tokens come widened to f16 (widen_rows_kernel; T x K, where
// widening the weights as well would move five bytes for each of them first).
// Bound by the tensor cores and the widening that feeds them: 8192 x 4096 x 8192 340 us
// with the tokens' widening (1620 TFLOP/s; the f16 rate under the power cap is 1715).
//
// Tiles of 256 (L) x up to 192 (R) rows: two accumulators of 192 columns and two
// stages of widened weights of 64 fill the 512 TMEM columns.  A stage is 128
// terms: 16 KiB of 8-bit weights, which the CTA's own barrier announces to its
// widening warps, and two swizzled blocks of its half of the tokens, announced to
// the even CTA's issuing warp.  The widening warps of both CTAs arrive on the
// even CTA's barrier of the TMEM stage.
constexpr int kIpRows = 192, kIpRowsR = kIpRows / 2;         // per tile, per CTA
constexpr int kIpLBytes = 128 * 128;
constexpr int kIpAtomBytes = kIpRowsR * 128;                 // 64 terms of a CTA's tokens
constexpr int kIpStageBytes = kIpLBytes + 2 * kIpAtomBytes;
constexpr int kIpStages = 4;                                 // (an even number: a team's stages are every other one)
// kRuns: sums of more than one run.  Warps: two teams of four that widen, four of the
// epilogue (kRuns: eight), one for the TMA and one for the MMAs (kRuns: and two that only
// wait, so that warps come in fours).  The sums of 96 columns a thread want more registers
// than an even share, which the others give up.
template <bool kRuns>
struct I8PairCfg {
    static constexpr int kEpiWarps = kRuns ? 8 : 4;
    static constexpr int kTurns = kEpiWarps / 4;             // warps to a quarter of the lanes, which take steps in turn
    static constexpr int kPieces = kIpRows / kGrChunk / kTurns;
    static constexpr int kFirstEpi = 8, kTmaWarp = kFirstEpi + kEpiWarps, kMmaWarp = kTmaWarp + 1;
    static constexpr int kThreads = 32 * (kTmaWarp + (kRuns ? 4 : 2));
    // full8[S], fullr[S], empty[S], fulla[2], emptya[2], accfull[2], accempty[2], drain, never
    static constexpr int kBarriers = 3 * kIpStages + 10;
    static constexpr int kSmemBytes = 1024 /* alignment slack */ + kIpStages * kIpStageBytes + kEpiWarps * kGrStageBytes +
                                      kBarriers * 8 + 32 + kIpStages * 4 + 2 * (kGrMaxExperts + 8) * 4;
    static_assert(kSmemBytes <= 232448, "exceeds the 227 KiB shared memory of one CTA");
};
constexpr int kIpLaunchRegs = 96, kIpRegsLead = 64, kIpRegsWiden = 72, kIpRegsEpi = 136;
static_assert(128 * kIpRegsLead + 256 * kIpRegsWiden + 256 * kIpRegsEpi <= I8PairCfg<true>::kThreads * kIpLaunchRegs,
              "no more registers than the block is launched with");
constexpr uint32_t kIpACol0 = 2 * kIpRows;
constexpr uint32_t kIpTmemCols = 512;
static_assert(kIpACol0 + 2 * kI8ACols == kIpTmemCols, "the TMEM columns are all used");
static_assert(kIpAtomBytes % 1024 == 0, "blocks start on the swizzle's 1024 bytes");

template <bool kRuns>
__global__ void __launch_bounds__(I8PairCfg<kRuns>::kThreads, 1) tn_i8_pair_kernel(const __grid_constant__ GroupedParams p)
{
    using Cfg = I8PairCfg<kRuns>;
    constexpr int kS = kIpStages;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_ring = ptx::smem_addr(smem), s_staging = s_ring + kS * kIpStageBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kS * kIpStageBytes + Cfg::kEpiWarps * kGrStageBytes);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + Cfg::kBarriers);
    volatile uint32_t *abort_flag = tmem_holder + 1;
    volatile uint32_t *issued_count = tmem_holder + 2;    // fills this CTA's producer issued
    volatile uint32_t *producer_done = tmem_holder + 3;   // set once this CTA's producer issues no more
    volatile uint32_t *fill_bytes = tmem_holder + 8;      // [kS]: this CTA's token bytes of the stage's last fill
    int32_t *start = reinterpret_cast<int32_t *>(tmem_holder + 8 + kS);
    int32_t *before = start + kGrMaxExperts + 8;
    const uint32_t abort_addr = ptx::smem_addr(const_cast<uint32_t *>(abort_flag));
    const uint32_t count_addr = ptx::smem_addr(const_cast<uint32_t *>(issued_count));
    const uint32_t done_addr = ptx::smem_addr(const_cast<uint32_t *>(producer_done));
    const uint32_t fill_addr = ptx::smem_addr(const_cast<uint32_t *>(fill_bytes));
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full8_bar = [&](int s) { return bar0 + 8u * s; };
    auto fullr_bar = [&](int s) { return bar0 + 8u * (kS + s); };
    auto empty_bar = [&](int s) { return bar0 + 8u * (2 * kS + s); };
    auto fulla_bar = [&](int t) { return bar0 + 8u * (3 * kS + t); };
    auto emptya_bar = [&](int t) { return bar0 + 8u * (3 * kS + 2 + t); };
    auto accfull_bar = [&](int b) { return bar0 + 8u * (3 * kS + 4 + b); };
    auto accempty_bar = [&](int b) { return bar0 + 8u * (3 * kS + 6 + b); };
    const uint32_t drain_bar = bar0 + 8u * (3 * kS + 8);
    const uint32_t never_bar = bar0 + 8u * (3 * kS + 9);   // nothing ever arrives (test stalls)

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t pos = ptx::cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kS; ++s) {
            ptx::mbar_init(full8_bar(s), 1);
            ptx::mbar_init(fullr_bar(s), 1);
            ptx::mbar_init(empty_bar(s), kI8TeamWarps + 1);      // the weights are read, and the tokens
            fill_bytes[s] = 0u;
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(fulla_bar(b), 2 * kI8TeamWarps);
            ptx::mbar_init(emptya_bar(b), 1);
            ptx::mbar_init(accfull_bar(b), 1);
            ptx::mbar_init(accempty_bar(b), 2 * Cfg::kEpiWarps);
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::mbar_init(never_bar, 1);
        *abort_flag = 0u;
        *issued_count = 0u;
        *producer_done = 0u;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (threadIdx.x == 32 && p.red > 0) {
        ptx::prefetch_tensormap(&p.tmap_l);
        ptx::prefetch_tensormap(&p.tmap_r[kIpRowsR / 16 - 1]);
    }
    if (warp == Cfg::kMmaWarp) {
        ptx::tmem_alloc<2>(ptx::smem_addr(tmem_holder), kIpTmemCols);
        ptx::tmem_relinquish_alloc_permit<2>();
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    const Waiter w{abort_flag, abort_addr, pos, 2u, p.wait_limit_ns};

    ptx::griddep_wait();                      // every thread's first global access is behind this wait
    const int32_t l_tiles = (p.l_extent + 255) / 256;
    grouped_tables<kGrI8, kIpRows, Cfg::kThreads>(p, l_tiles, start, before);
    const int32_t total = before[p.E];
    const int32_t slot = static_cast<int32_t>(blockIdx.x) / 2, slots = static_cast<int32_t>(gridDim.x) / 2;
    GroupedWalk<kGrI8, kIpRows, kIpRows, 256, 32> walk{start, before, l_tiles, 0, p.red, 0};
    const int32_t blocks = (p.red + kI8Block - 1) / kI8Block;       // stages of a tile

    if (warp >= Cfg::kTmaWarp) {
        if constexpr (kRuns) ptx::setmaxnreg_dec<kIpRegsLead>();
        if (warp == Cfg::kTmaWarp) {
            // ------------------------------------------------ TMA producer (both CTAs)
            int stage = 0;
            uint32_t phase = 0, n_issued = 0;
            bool ok = true;
            if (p.flags & (pos == 0 ? kFlagStallProducer0 : kFlagStallProducer1)) ok = wait_warp(w, never_bar, 0u, kSiteStall);
            for (int32_t u = slot; ok && u < total; u += slots) {
                const GroupedTile t = walk.at(u);
                const int32_t cols = t.n_mma[0] / 2;                 // this CTA's tokens
                const CUtensorMap *map_r = p.tmap_r + cols / 16 - 1;
                const int32_t l0 = t.l0 + static_cast<int32_t>(pos) * 128;
                const int32_t r0 = start[t.e] + t.r0 + static_cast<int32_t>(pos) * cols;
                for (int32_t i = 0; i < blocks; ++i) {
                    if (!wait_warp(w, empty_bar(stage), phase ^ 1u, kSiteEmpty)) {
                        ok = false;
                        break;
                    }
                    ++n_issued;
                    if (ptx::elect_one()) {
                        const uint32_t s_l = s_ring + stage * kIpStageBytes, s_r = s_l + kIpLBytes;
                        const uint32_t bar_r = ptx::mapa_shared(fullr_bar(stage), 0);
                        const uint32_t bytes = 2u * cols * 128u;
                        fill_bytes[stage] = bytes;
                        ptx::mbar_arrive_expect_tx(full8_bar(stage), kIpLBytes);
                        tma_load_3d(s_l, &p.tmap_l, full8_bar(stage), i * kI8Block, l0, t.e);
                        if (pos == 0) ptx::mbar_arrive_expect_tx(fullr_bar(stage), 2 * bytes);
                        ptx::tma_load_2d_pair(s_r, map_r, bar_r, i * kI8Block, r0);
                        ptx::tma_load_2d_pair(s_r + kIpAtomBytes, map_r, bar_r, i * kI8Block + kGrBlock, r0);
                        *issued_count = n_issued;
                    }
                    __syncwarp();
                    if (++stage == kS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (lane == 0) ptx::griddep_launch_dependents();
            if (ptx::elect_one()) {
                auto fills = [](uint32_t n, int s) { return n / kS + (static_cast<uint32_t>(s) < n % kS ? 1u : 0u); };
                // this CTA's weights: every issued load lands before the CTA can exit
                for (int s = 0; s < kS; ++s)
                    if (const uint32_t passes = fills(n_issued, s)) w.drain(full8_bar(s), (passes - 1) & 1u);
                ptx::st_release_cluster_u32(ptx::mapa_shared(done_addr, pos), 1u);
                if (pos == 0) {
                    // the pair's tokens, as in tn_grouped_kernel
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
                    for (int s = 0; s < kS; ++s) {
                        const uint32_t mine = fills(n_issued, s), theirs = fills(peer, s);
                        const uint32_t last = mine > theirs ? mine : theirs;
                        if (last == 0) continue;
                        if (mine > theirs + 1 || theirs > mine + 1) {      // cannot happen; never guess
                            atomicCAS(&g_tn_status, 0, 4 | (kSiteReconcile << 8));
                            continue;
                        }
                        if (mine > theirs)
                            ptx::mbar_complete_tx(fullr_bar(s), fill_bytes[s]);
                        else if (theirs > mine)
                            ptx::mbar_arrive_expect_tx(fullr_bar(s),
                                                       ptx::ld_relaxed_cluster_u32(ptx::mapa_shared(fill_addr + 4u * s, 1)));
                        w.drain(fullr_bar(s), (last - 1) & 1u);
                    }
                }
            }
        } else if (warp == Cfg::kMmaWarp) {
            if (pos == 0) {
                // ------------------------------------------------ MMA issuer (even CTA)
                int stage = 0;
                uint32_t phase = 0, sub = 0, n = 0;               // runs (run `sub` uses accumulator sub % 2) and stages so far
                bool ok = true, issued_any = false;
                if (p.flags & kFlagStallMma) ok = wait_warp(w, never_bar, 0u, kSiteStall);
                for (int32_t u = slot; ok && p.red > 0 && u < total; u += slots) {
                    const GroupedTile t = walk.at(u);
                    const uint32_t idesc = ptx::idesc_f32acc(256, static_cast<uint32_t>(t.n_mma[0]), 0u, 0u);
                    for (int32_t i = 0, run = 0; i < blocks; ++i, ++n) {      // run: stages of the run so far
                        const uint32_t team = n & 1u;
                        const uint32_t d_tmem = tmem_base + (sub & 1u) * kIpRows;
                        if ((run == 0 && !wait_warp(w, accempty_bar(sub & 1u), ((sub >> 1) & 1u) ^ 1u, kSiteAccEmpty)) ||
                            !wait_warp(w, fullr_bar(stage), phase, kSiteLoaded) ||
                            !wait_warp(w, fulla_bar(team), (n >> 1) & 1u, kSiteLoaded)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after_sync();
                        const int32_t left = p.red - i * kI8Block;
                        const bool last = i + 1 == blocks || (kRuns && run + 1 == kI8Run);
                        if (ptx::elect_one()) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint64_t desc_r = ptx::desc_kmajor_sw128(s_ring + stage * kIpStageBytes + kIpLBytes +
                                                                               half * kIpAtomBytes);
                                const uint32_t a_tmem = tmem_base + kIpACol0 + team * kI8ACols + half * (kI8ACols / 2);
#pragma unroll
                                for (int j = 0; j < kGrBlock / 16; ++j)
                                    if (left > half * kGrBlock + 16 * j)
                                        ptx::mma_f16_ts<2>(d_tmem, a_tmem + 8 * j, desc_r + 2u * j, idesc,
                                                           (run | half | j) != 0 ? 1u : 0u);
                            }
                            ptx::mma_commit<2>(emptya_bar(team), 3);
                            ptx::mma_commit<2>(empty_bar(stage), 3);
                            if (last) ptx::mma_commit<2>(accfull_bar(sub & 1u), 3);
                        }
                        __syncwarp();
                        issued_any = true;
                        ++run;
                        if (last) {
                            run = 0;
                            ++sub;
                        }
                        if (++stage == kS) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (issued_any && ptx::elect_one()) {             // every MMA issued completes before TMEM is freed
                    ptx::mma_commit<2>(drain_bar, 1);
                    w.drain(drain_bar, 0u);
                }
            }
        }
    } else if (warp < Cfg::kFirstEpi) {
        // ------------------------------------------------ widening (both CTAs)
        if constexpr (kRuns) ptx::setmaxnreg_dec<kIpRegsWiden>();
        const int team = warp / kI8TeamWarps;
        static_assert(kS % 2 == 0, "a team's stages are every other one");
        const int quarter = warp & 3;
        const uint32_t row_l = static_cast<uint32_t>(32 * quarter + lane) * 128u;
        const uint32_t t_a = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + kIpACol0 + team * kI8ACols;
        const uint32_t fulla = ptx::mapa_shared(fulla_bar(team), 0);
        bool ok = true;
        int stage = team;
        uint32_t phase = 0, phase_a = 0, n = 0;               // n: stages so far
        for (int32_t u = slot; ok && p.red > 0 && u < total; u += slots) {
            for (int32_t i = 0; i < blocks; ++i, ++n) {
                if ((n & 1u) != static_cast<uint32_t>(team)) continue;
                ok = wait_warp(w, full8_bar(stage), phase, kSiteLoaded);
                if (!ok) break;
                const uint32_t src = s_ring + stage * kIpStageBytes + row_l;
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = ptx::ld_shared_v4(src + ((c ^ (lane & 7)) << 4));
                ok = wait_warp(w, emptya_bar(team), phase_a ^ 1u, kSiteEmpty);
                if (!ok) break;
                ptx::tc_fence_after_sync();                   // the MMAs that read this TMEM stage are done
                widen_row_to_tmem<kRuns ? 2 : 4>(src, lane, v, t_a);
                ptx::tmem_st_wait();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive_remote(fulla);
                    ptx::mbar_arrive(empty_bar(stage));
                }
                phase_a ^= 1u;
                stage += 2;
                if (stage >= kS) {
                    stage -= kS;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        // The sums of several runs gather in registers, and go back as floats to the
        // accumulator of the last one, out of which a tile is stored.
        if constexpr (kRuns) ptx::setmaxnreg_inc<kIpRegsEpi>();
        constexpr int kTurns = Cfg::kTurns, kPieces = Cfg::kPieces;
        const int quarter = warp & 3, turn = (warp - Cfg::kFirstEpi) >> 2;
        const uint32_t t_lanes = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16);
        const float unit = sum_unit(p.red);
        GroupedStore store;
        store.init(s_staging + (warp - Cfg::kFirstEpi) * kGrStageBytes, lane);
        store.ld = p.out_ld;
        uint32_t sub = 0;                                     // runs so far
        auto acc_full = [&]() {
            const bool ok = wait_warp(w, accfull_bar(sub & 1u), (sub >> 1) & 1u, kSiteAccFull);
            if (ok) ptx::tc_fence_after_sync();
            return ok;
        };
        auto hand_back = [&]() {                              // this warp has read its part of the accumulator
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_remote(ptx::mapa_shared(accempty_bar(sub & 1u), 0));
        };
        for (int32_t u = slot; u < total; u += slots) {
            if constexpr (kRuns) {
                const int32_t n_mma = walk.at(u).n_mma[0];
                uint32_t sum[kPieces][2][16];
#pragma unroll
                for (int s = 0; s < kPieces; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int q = 0; q < 16; ++q) sum[s][h][q] = 0u;
                bool ok;
                int32_t i = 0;
                while (true) {
                    ok = acc_full();
                    if (!ok) break;
#pragma unroll
                    for (int s = 0; s < kPieces; ++s) {
                        const int32_t c = (kTurns * s + turn) * kGrChunk;
                        if (c >= n_mma) break;
                        uint32_t v[2][16];
                        load_piece(t_lanes + (sub & 1u) * kIpRows + c, v);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                sum[s][h][q] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(v[h][q]) * unit));
                    }
                    i += kI8Run;
                    if (i >= blocks) break;
                    hand_back();
                    ++sub;
                }
                if (!ok) break;
#pragma unroll
                for (int s = 0; s < kPieces; ++s) {
                    const int32_t c = (kTurns * s + turn) * kGrChunk;
                    if (c >= n_mma) break;
                    piece_to_floats(sum[s], unit);
                    store_piece(t_lanes + (sub & 1u) * kIpRows + c, sum[s]);
                }
            }
            const GroupedTile t = walk.at(u);
            const int32_t l0 = t.l0 + static_cast<int32_t>(pos) * 128 + 32 * quarter;
            const int64_t row0 = static_cast<int64_t>(start[t.e]) + t.r0;
            uint16_t *out = p.out + row0 * p.out_ld + l0;
            store.wide = p.l_extent - l0 < 32 ? p.l_extent - l0 : 32;
            store.vec = p.out_vec != 0 && store.wide == 32;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store.scale_l[i] = 8 * i + (lane >> 2) < store.wide
                                       ? __ldg(p.scale_l + static_cast<int64_t>(t.e) * p.l_extent + l0 + 8 * i + (lane >> 2))
                                       : 0.0f;
            if constexpr (!kRuns) {
                if (!acc_full()) break;
            }
#pragma unroll 1
            for (int32_t c = turn * kGrChunk; c < t.n_mma[0]; c += kTurns * kGrChunk) {
                uint32_t v[2][16];
                load_piece(t_lanes + (sub & 1u) * kIpRows + c, v);
                if (c + kTurns * kGrChunk >= t.n_mma[0]) hand_back();
                if (p.out_fmt != 0)
                    store.step<true, true>(v, out + c * p.out_ld, t.rows - c, p.scale_r + row0 + c);
                else
                    store.step<false, true>(v, out + c * p.out_ld, t.rows - c, p.scale_r + row0 + c);
            }
            if (turn * kGrChunk >= t.n_mma[0]) hand_back();   // (no columns of its own)
            ++sub;
        }
    }

    __syncwarp();                // .aligned barriers below need converged warps
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();         // no CTA leaves while the other may still touch its shared memory
    if (warp == Cfg::kMmaWarp) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<2>(tmem_base, kIpTmemCols);
    }
}

}  // namespace tn
