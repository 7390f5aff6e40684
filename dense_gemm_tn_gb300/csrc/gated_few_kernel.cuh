// gated_few_kernel: the gated projections (grouped_sinks.cuh) of up to 16 tokens, a
// decode step's, over weights of a few megabytes.  What bounds them is the read of the weights,
// once, and the general kernel's tiles are too coarse for it: 2048 x 2048 are 32 tiles of
// 64 gate and 64 up rows (split four ways, 9.8 us); here they are 128 of 16 and 16, 6.0 us
// with one token (2.8 TB/s; the kernel's start and its join are most of the rest).
//
// A CTA's warps share a tile's rows and split the sum by blocks of 64 terms (128
// bytes of a row).  Each lane copies its own 16-byte pieces of its rows kDepth - 1
// blocks ahead into a ring of its own in shared memory and multiplies them by
// mma.m16n8k16, the tokens on its N side (a warp's own instruction: its operands are
// registers, and its rate is not what bounds).  The warps' sums meet in shared
// memory, in the warps' order.
#pragma once

#include <cstdint>

#include "grouped_sinks.cuh"
#include "w4_kernel.cuh"

namespace tn {

struct GatedFewParams {
    const uint16_t *a;               // E matrices of 2 M rows
    int64_t lda, stride_a;
    const uint16_t *b;               // T tokens
    int64_t ldb;
    const int32_t *offsets;          // E + 1, or NULL: one matrix, all tokens
    uint16_t *h;
    int64_t ldh;
    float *pre;                      // the products, or NULL
    int64_t pre_ld;
    int32_t E, T, M, K;
    int32_t tiles;                   // of 16 gate rows
    int32_t act;
};

constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps, kFewDepth = 2, kFewBlock = 64;
constexpr int kFewRingBytes = kFewWarps * kFewDepth * 8 * 32 * 16;      // a lane: 4 rows, 2 pieces each
constexpr int kFewRowFloats = 36;                                       // 32 rows' sums of a token

template <bool kBf16, int kTilesN>
__global__ void __launch_bounds__(kFewThreads) gated_few_kernel(const __grid_constant__ GatedFewParams p)
{
    extern __shared__ __align__(16) float few_smem[];
    __shared__ int32_t found[3];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int32_t nth = static_cast<int32_t>(blockIdx.x) / p.tiles;     // of the experts with rows
    const int32_t m0 = (static_cast<int32_t>(blockIdx.x) - nth * p.tiles) * 16;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    int32_t e = 0, row0 = 0, rows = p.T;
    if (p.offsets) {
        // the offsets as the general kernel reads them: each at least the ones before it, at most T
        if (warp == 0) {
            int32_t top = 0, left = nth, which = -1, first = 0, end = 0;
            for (int32_t i0 = 0; i0 < p.E && which < 0; i0 += 32) {
                auto at = [&](int32_t i) {
                    const int32_t o = i <= p.E ? p.offsets[i] : 0;
                    return o < 0 ? 0 : o > p.T ? p.T : o;
                };
                int32_t from = max(at(i0 + lane), top);
                for (int d = 1; d < 32; d *= 2) {
                    const int32_t o = __shfl_up_sync(0xffffffffu, from, d);
                    if (lane >= d) from = max(from, o);
                }
                const int32_t to = max(from, at(i0 + lane + 1));
                const uint32_t some = __ballot_sync(0xffffffffu, i0 + lane < p.E && to > from);
                const int32_t n = __popc(some);
                if (left < n) {
                    const int src = __fns(some, 0, left + 1);
                    which = i0 + src;
                    first = __shfl_sync(0xffffffffu, from, src);
                    end = __shfl_sync(0xffffffffu, to, src);
                } else {
                    left -= n;
                    top = __shfl_sync(0xffffffffu, to, 31);
                }
            }
            if (lane == 0) {
                found[0] = which;
                found[1] = first;
                found[2] = end - first;
            }
        }
        __syncthreads();
        e = found[0];
        row0 = found[1];
        rows = found[2];
        if (e < 0) return;
    }

    // rows g, g + 8 of the gate's 16 and of the up rows' (past the last: the last again, not stored)
    const uint16_t *a_row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t m = min(m0 + 8 * (i & 1) + g, p.M - 1) + (i >> 1) * p.M;
        a_row[i] = p.a + e * p.stride_a + m * p.lda + warp * kFewBlock + 8 * t;
    }
    const uint16_t *b_row[kTilesN];
    bool held[kTilesN];
#pragma unroll
    for (int n = 0; n < kTilesN; ++n) {
        held[n] = 8 * n + g < rows;
        b_row[n] = p.b + (row0 + (held[n] ? 8 * n + g : 0)) * p.ldb + warp * kFewBlock + 8 * t;
    }
    const int32_t blocks = (p.K + kFewBlock - 1) / kFewBlock;
    constexpr int kStep = kFewWarps * kFewBlock;
    const uint32_t ring = ptx::smem_addr(few_smem) + (warp * kFewDepth * 8 * 32 + lane) * 16;
    // the block `ahead` turns after block b; terms past the last are zeros
    auto copy = [&](int32_t b, int ahead, int stage) {
        const int32_t left = p.K - (b + ahead * kFewWarps) * kFewBlock - 8 * t;
        if (left > -8 * t) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int32_t bytes = left > 32 * q ? 16 : 0;       // (K is a multiple of 8)
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(ring + ((stage * 4 + i) * 2 + q) * 512),
                                 "l"(bytes ? a_row[i] + ahead * kStep + 32 * q : p.a), "r"(bytes)
                                 : "memory");
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    struct Tokens {
        uint4 v[2][kTilesN];
    };
    auto load = [&](Tokens &x, int32_t b, int ahead) {
        const int32_t left = p.K - (b + ahead * kFewWarps) * kFewBlock - 8 * t;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int n = 0; n < kTilesN; ++n) {
                x.v[q][n] = make_uint4(0, 0, 0, 0);
                if (held[n] && left > 32 * q)
                    x.v[q][n] = __ldg(reinterpret_cast<const uint4 *>(b_row[n] + ahead * kStep + 32 * q));
            }
    };
    float acc[2][kTilesN][4] = {};               // gate and up
    int32_t b = warp;
#pragma unroll
    for (int s = 0; s < kFewDepth - 1; ++s) copy(b, s, s);
    Tokens tokens[2];
    load(tokens[0], b, 0);
#pragma unroll 1
    while (b < blocks) {
#pragma unroll
        for (int s = 0; s < kFewDepth; ++s) {
            if (s > 0 && b + s * kFewWarps >= blocks) break;
            copy(b, s + kFewDepth - 1, (s + kFewDepth - 1) % kFewDepth);
            load(tokens[(s + 1) & 1], b, s + 1);
            const Tokens &x = tokens[s & 1];
            asm volatile("cp.async.wait_group %0;" ::"n"(kFewDepth - 1) : "memory");
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 lo = w4::ld_shared(ring + ((s * 4 + 2 * i) * 2 + q) * 512);
                    const uint4 hi = w4::ld_shared(ring + ((s * 4 + 2 * i + 1) * 2 + q) * 512);
#pragma unroll
                    for (int n = 0; n < kTilesN; ++n) {
                        w4::mma<kBf16>(acc[i][n], lo.x, hi.x, lo.y, hi.y, x.v[q][n].x, x.v[q][n].y);
                        w4::mma<kBf16>(acc[i][n], lo.z, hi.z, lo.w, hi.w, x.v[q][n].z, x.v[q][n].w);
                    }
                }
        }
        b += kFewDepth * kFewWarps;
#pragma unroll
        for (int i = 0; i < 4; ++i) a_row[i] += kFewDepth * kStep;
#pragma unroll
        for (int n = 0; n < kTilesN; ++n) b_row[n] += kFewDepth * kStep;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                             // every ring is done with

    float *mine = few_smem + warp * 8 * kTilesN * kFewRowFloats;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < kTilesN; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                mine[(8 * n + 2 * t + (r & 1)) * kFewRowFloats + 16 * i + 8 * (r >> 1) + g] = acc[i][n][r];
    __syncthreads();
    for (int32_t i = threadIdx.x; i < 16 * 8 * kTilesN; i += kFewThreads) {
        const int32_t n = i >> 4, m = i & 15;
        if (n >= rows || m0 + m >= p.M) continue;
        float gate = 0.0f, up = 0.0f;
        for (int w = 0; w < kFewWarps; ++w) {
            const float *from = few_smem + (w * 8 * kTilesN + n) * kFewRowFloats + m;
            gate += from[0];
            up += from[16];
        }
        const float y = p.act == kActSilu   ? act_factor<kActSilu>(gate)
                        : p.act == kActGelu ? act_factor<kActGelu>(gate)
                                            : act_factor<kActGeluTanh>(gate);
        const int64_t row = row0 + n;
        p.h[row * p.ldh + m0 + m] = w4::from_float<kBf16>(gate * y * up);
        if (p.pre) {
            p.pre[row * p.pre_ld + m0 + m] = gate;
            p.pre[row * p.pre_ld + p.M + m0 + m] = up;
        }
    }
}

}  // namespace tn
