// The small kernels around the gated projections' and the loss's products: the joins
// of a token's statistics and of a sum's parts, the loss gradient's factors, and the
// gated projections' elementwise backward pass.  All are bound by what they read and
// write.
#pragma once

#include "grouped_sinks.cuh"

namespace tn {

// ------------------------------------------------------------------ loss: joins
// The pieces' pairs of each token, in the order of the classes within a slice and of
// the slices (so results repeat): `lanes` tokens a CTA (a power of two), 512 / lanes
// slices.  Reads 8 bytes per token and 32 classes, kJoinStep pairs a thread at once: one at a
// time the loss of 1021 tokens over 32003 classes of 1024 takes 56.8 us in all, 4 at once
// 56.2, 16 52.1; of 257 over 50021 of 2048 67.3, 65.3 and 64.2.
constexpr int kJoinThreads = 512, kJoinStep = 16;

struct JoinParams {
    const float2 *stats;
    const float *z_target;
    const int64_t *targets;
    float *loss, *lse;
    int64_t N, classes;
    int32_t pieces, lanes;
};

__global__ void __launch_bounds__(kJoinThreads) cross_entropy_join_kernel(const JoinParams p)
{
    __shared__ float2 part[kJoinThreads];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int32_t lane = threadIdx.x & (p.lanes - 1), slice = threadIdx.x / p.lanes, slices = kJoinThreads / p.lanes;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * p.lanes + lane;
    const float none = __int_as_float(0xff800000);
    float m = none, s = 0.0f;
    if (n < p.N) {
        const int32_t per = (p.pieces + slices - 1) / slices;
        const int32_t q0 = slice * per, q1 = min(q0 + per, p.pieces);
        for (int32_t q = q0; q < q1; q += kJoinStep) {       // (their loads all at once)
            float2 x[kJoinStep];
#pragma unroll
            for (int j = 0; j < kJoinStep; ++j)
                x[j] = q + j < q1 ? p.stats[static_cast<int64_t>(q + j) * p.N + n] : make_float2(none, 0.0f);
            float top = m;
#pragma unroll
            for (int j = 0; j < kJoinStep; ++j) top = fmaxf(top, x[j].x);
            const float from = top == none ? 0.0f : top;     // (no logit above -inf: sums of 0, or NaN)
            s *= ex2((m - from) * kLog2e);
#pragma unroll
            for (int j = 0; j < kJoinStep; ++j) s = fmaf(x[j].y, ex2((x[j].x - from) * kLog2e), s);
            m = top;
        }
    }
    part[threadIdx.x] = make_float2(m, s);
    for (int32_t half = slices / 2; half >= 1; half /= 2) {
        __syncthreads();
        if (slice < half) {
            const float2 x = part[threadIdx.x + half * p.lanes];
            Sink<5>::merge(m, s, x.x, x.y);
            part[threadIdx.x] = make_float2(m, s);
        }
    }
    if (slice == 0 && n < p.N) {
        const float above = logf(s);
        p.lse[n] = m + above;
        // (not lse less the logit: where the target is the maximum the lse's rounding is no part of the loss)
        const int64_t t = p.targets[n];
        p.loss[n] = t < 0 ? 0.0f : t < p.classes ? (m - p.z_target[n]) + above : __int_as_float(0x7fffffff);
    }
}

// The loss gradient's factor of each token: the loss's own gradient, 0 where the
// target is negative, NaN where it is no class, as a share of the largest (times 2^13 for
// fp16, whose small numbers end early); `scale` undoes that in the products' FP32 sums.
// Where all tokens weigh alike, as in a mean, the factor is thus a power of two, and the
// rounding of d = factor (p - 1) at the targets does not add the same error to all of
// them (1 / 3900 is 0.2 % off in bf16).  One CTA.
constexpr int kRowsThreads = 1024;

struct LossRowsParams {
    const int64_t *targets;
    const float *lse, *dloss;
    float2 *rows;
    float *scale;
    int64_t N, classes;
    bool half;
};

__global__ void __launch_bounds__(kRowsThreads) cross_entropy_rows_kernel(const LossRowsParams p)
{
    __shared__ float tops[kRowsThreads / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    auto factor = [&p](int64_t n) {
        const int64_t t = p.targets[n];
        const float g = p.dloss[n];
        return t < 0 ? 0.0f : t < p.classes ? g : __int_as_float(0x7fffffff);
    };
    float top = 0.0f;
#pragma unroll 8
    for (int64_t n = threadIdx.x; n < p.N; n += kRowsThreads) {
        const float f = fabsf(factor(n));
        if (f < __int_as_float(0x7f800000)) top = fmaxf(top, f);     // (no infinity and no NaN)
    }
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int i = 0; i < kRowsThreads / 32; ++i) top = fmaxf(top, tops[i]);
    if (top == 0.0f) top = 1.0f;
    const float up = p.half ? 8192.0f : 1.0f;
#pragma unroll 8
    for (int64_t n = threadIdx.x; n < p.N; n += kRowsThreads)
        p.rows[n] = make_float2(-p.lse[n] * kLog2e, __fdiv_rn(factor(n), top) * up);
    if (threadIdx.x == 0) *p.scale = top / up;
}

// ------------------------------------------------------------------ parts of a sum, joined
// out = scale (sum of the parts, in their order), rounded once.  Reads 4 bytes an
// element and part, writes 2.
constexpr int kPartsThreads = 256;

struct PartsParams {
    const float *sum;                // parts of rows x cols, sum_ld floats a row
    int64_t sum_ld, sum_stride;
    uint16_t *out;
    int64_t ld;
    const float *scale;              // one float, or NULL
    int64_t rows;
    int32_t cols, parts;
    bool bf16;
    bool vec;                        // four elements a thread: rows on 16-byte (out: 8-byte) boundaries
};

__global__ void __launch_bounds__(kPartsThreads) parts_join_kernel(const PartsParams p)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const float scale = p.scale ? __ldg(p.scale) : 1.0f;
    const int32_t per = p.vec ? 4 : 1, units = (p.cols + per - 1) / per;
    const int32_t c = static_cast<int32_t>(blockIdx.x) * kPartsThreads + static_cast<int32_t>(threadIdx.x);
    if (c >= units) return;
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const float *from = p.sum + r * p.sum_ld + c * per;
        uint16_t *out = p.out + r * p.ld + c * per;
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int32_t q = 0; q < p.parts; ++q, from += p.sum_stride) {
            if (p.vec) {
                const float4 v = __ldcs(reinterpret_cast<const float4 *>(from));
                x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
            } else {
                x[0] += *from;
            }
        }
        const uint32_t lo = p.bf16 ? ptx::pack_bf16x2(x[0] * scale, x[1] * scale) : ptx::pack_f16x2(x[0] * scale, x[1] * scale);
        const uint32_t hi = p.bf16 ? ptx::pack_bf16x2(x[2] * scale, x[3] * scale) : ptx::pack_f16x2(x[2] * scale, x[3] * scale);
        if (p.vec)
            *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
        else
            *out = static_cast<uint16_t>(lo);
    }
}

// ------------------------------------------------------------------ gated: backward
// d_gate = dH u act'(g) and d_up = dH act(g) from the kept products, rounded to the
// operands' type, as the tensor cores take both operands of a product in one type and a second product with what
// the rounding drops would double the gradients' time (bf16 gradients are 2.3e-3 off so, 1.7e-3 by their own
// rounding alone): 8 bytes of products and 2 of dH read, 4 written an element, nothing
// else.  4096 rows of 14336 take 154 us on GB300 (5.3 TB/s; 171 with loads marked as read once),
// 3001 of 1024 6.4 out of the L2.  kVec: 8 elements a thread (rows on 16-byte boundaries);
// short rows share a CTA (3001 rows of 1024, the whole gradient: 71.3 us with a CTA a row, 69.9
// with half a one).
constexpr int kGatedGradThreads = 256;

// fp16 has gradients to 2^-24 and no more than 65504, so there dP is rounded times a power of
// two that its largest finite number decides, undone in the products' FP32 sums.  dP is not
// there before it is rounded, so: gated_top_kernel takes the largest |dH|, 2 bytes an
// element; the elementwise pass rounds times the factor that puts this at 2^8, and takes the
// largest |dP|; a second one starts over, the factor from |dP| itself, where that came
// out below 2^4 or above 65504, and returns at once where it did not (nearly always: |dP|
// is |dH| times the products' size).  Between the kernels a few numbers stand in a room of the
// workspace, four floats an entry:
//   entry i  [0] the largest |dH| of gated_top_kernel's CTA i
//   entry 0  [1] the largest |dP|, [2] the factor that undoes the final one, [3] the first factor
// (They are read past the L1: an entry's numbers share a line and are written at different times.)
// The gradient of 4096 rows of 14336 x 4096 takes 1267 us so (1206 without a factor; with the second pass
// 1477), of 3001 rows over 8 experts of 1024 x 2048 98 (83).
constexpr int kGatedTopThreads = 512, kGatedTops = 304;      // (its CTAs at most: two an SM)
constexpr int kGatedEntry = 4;

struct GatedGradParams {
    const float *pre;
    int64_t pre_ld;
    const uint16_t *dh;
    int64_t dh_ld;
    uint16_t *dp;                    // T rows of [gate | up], then zeros to dp_units
    int64_t dp_ld, dp_units;
    float *room;                     // fp16: entries, entry_step floats apart
    int64_t entry_step;
    const int32_t *offsets;          // rows before the first and from the last on are left out; or NULL
    int32_t E, T, M;
    int32_t lanes;                   // threads of a row: a power of two from 32 to all
    int32_t tops, top_lanes;         // gated_top_kernel's CTAs, at most T, and its threads of a row (a power of two from 32 on)
    bool top_vec;                    // dH's rows on 16-byte boundaries
    bool again;                      // fp16: the second elementwise pass
};

// The rows [begin, end) that belong to experts, as the products read the offsets (by all
// threads of the CTA; `ends`: an int a warp).
__device__ __forceinline__ void gated_rows(const GatedGradParams &p, int32_t *ends, int32_t &begin, int32_t &end)
{
    begin = 0, end = p.T;
    if (!p.offsets) return;
    auto clamped = [&](int32_t i) {
        const int32_t o = p.offsets[i];
        return o < 0 ? 0 : (o > p.T ? p.T : o);
    };
    int32_t top = 0;
    for (int32_t i = threadIdx.x; i <= p.E; i += blockDim.x) top = max(top, clamped(i));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) ends[threadIdx.x >> 5] = top;
    __syncthreads();
    end = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) end = max(end, ends[i]);
    begin = clamped(0);
}

// The largest of the CTA's numbers (>= 0, as bits), for all its threads; `tops`: a number a warp.
__device__ __forceinline__ uint32_t largest_of_all(uint32_t x, uint32_t *tops)
{
    x = __reduce_max_sync(0xffffffffu, x);
    __syncthreads();                              // (the last call's numbers have been read)
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) x = max(x, tops[i]);
    return x;
}

// 2^k with x 2^k from 2^to to below 2^(to + 1); 1 for x = 0.
__device__ __forceinline__ float factor_for(float x, int to)
{
    if (x == 0.0f) return 1.0f;
    const int k = to + 127 - static_cast<int>(__float_as_uint(x) >> 23);
    return __uint_as_float(static_cast<uint32_t>(127 + max(-100, min(k, 100))) << 23);
}

// fp16: the largest finite |dH| of each CTA's rows.  Bound by the read of dH; short rows share a CTA
// (3001 rows of 1024 6.5 us under ncu, 10.0 with a CTA for each).
__global__ void __launch_bounds__(kGatedTopThreads) gated_top_kernel(const GatedGradParams p)
{
    __shared__ int32_t ends[kGatedTopThreads / 32];
    __shared__ uint32_t tops[kGatedTopThreads / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int32_t begin, end;
    gated_rows(p, ends, begin, end);
    uint32_t top = 0;                             // two halves' bits, which are ordered as their sizes
    auto take = [&top](uint32_t w) {
        w &= 0x7FFF7FFFu;
        top = __vmaxu2(top, w & __vcmpltu2(w, 0x7C007C00u));
    };
    const int32_t units = p.top_vec ? p.M / 8 : 0, lane = threadIdx.x & (p.top_lanes - 1);
    const int64_t rows = gridDim.x * (kGatedTopThreads / p.top_lanes);
    for (int64_t row = begin + threadIdx.x / p.top_lanes * gridDim.x + blockIdx.x; row < end; row += rows) {
        const uint16_t *dh = p.dh + row * p.dh_ld;
#pragma unroll 4
        for (int32_t i = lane; i < units; i += p.top_lanes) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(dh) + i);
            take(v.x), take(v.y), take(v.z), take(v.w);
        }
        for (int32_t i = 8 * units + lane; i < p.M; i += p.top_lanes) take(dh[i]);
    }
    top = largest_of_all(max(top & 0xFFFFu, top >> 16), tops);
    if (threadIdx.x == 0) {
        p.room[blockIdx.x * p.entry_step] = __half2float(__ushort_as_half(static_cast<uint16_t>(top)));
        if (blockIdx.x == 0) p.room[1] = 0.0f;
    }
}

template <int kAct, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kGatedGradThreads) gated_grad_kernel(const GatedGradParams p)
{
    constexpr int kN = kVec ? 8 : 1;
    __shared__ int32_t ends[kGatedGradThreads / 32];
    __shared__ uint32_t tops[kGatedGradThreads / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const float most = 65504.0f;                  // fp16's largest
    float factor = 1.0f;
    if constexpr (!kBf16) {
        const bool first = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
        if (p.again) {
            const float was = __ldcg(p.room + 3), top = __ldcg(p.room + 1), scaled = top * was;
            factor = top == 0.0f || (scaled >= 16.0f && scaled <= most) ? was : factor_for(top, 13);
            if (first) p.room[2] = 1.0f / factor;
            if (factor == was) return;
        } else {
            uint32_t top = 0;
            for (int32_t i = threadIdx.x; i < p.tops; i += kGatedGradThreads) top = max(top, __float_as_uint(__ldcg(p.room + i * p.entry_step)));
            factor = factor_for(__uint_as_float(largest_of_all(top, tops)), 8);
            if (first) p.room[3] = factor;
        }
    }
    int32_t begin, end;
    gated_rows(p, ends, begin, end);
    auto value = [](uint16_t b) {
        return kBf16 ? __uint_as_float(static_cast<uint32_t>(b) << 16) : __half2float(__ushort_as_half(b));
    };
    auto round2 = [factor](float a, float b) {
        return kBf16 ? ptx::pack_bf16x2(a, b) : ptx::pack_f16x2(a * factor, b * factor);
    };
    float top = 0.0f;                             // fp16: the largest finite |dP|
    const int32_t units = (p.M + kN - 1) / kN, rows = kGatedGradThreads / p.lanes;
    const int32_t lane = threadIdx.x & (p.lanes - 1);
    for (int64_t row = begin + blockIdx.y * rows + threadIdx.x / p.lanes; row < end; row += gridDim.y * rows) {
        const float *gate = p.pre + row * p.pre_ld, *up = gate + p.M;
        const uint16_t *dh = p.dh + row * p.dh_ld;
        uint16_t *dp = p.dp + row * p.dp_ld;
        for (int32_t i = blockIdx.x * p.lanes + lane; i < units; i += gridDim.x * p.lanes) {
            float g[kN], u[kN], d[kN], dg[kN], du[kN];
            if constexpr (kVec) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 a = __ldg(reinterpret_cast<const float4 *>(gate) + 2 * i + h);
                    const float4 b = __ldg(reinterpret_cast<const float4 *>(up) + 2 * i + h);
                    g[4 * h] = a.x, g[4 * h + 1] = a.y, g[4 * h + 2] = a.z, g[4 * h + 3] = a.w;
                    u[4 * h] = b.x, u[4 * h + 1] = b.y, u[4 * h + 2] = b.z, u[4 * h + 3] = b.w;
                }
                const uint4 c = __ldg(reinterpret_cast<const uint4 *>(dh) + i);
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    d[2 * q] = value(w[q]);
                    d[2 * q + 1] = value(w[q] >> 16);
                }
            } else {
                g[0] = gate[i];
                u[0] = up[i];
                d[0] = value(dh[i]);
            }
#pragma unroll
            for (int q = 0; q < kN; ++q) {
                const float y = act_factor<kAct>(g[q]);
                dg[q] = d[q] * u[q] * act_slope<kAct>(g[q], y);
                du[q] = d[q] * (g[q] * y);
            }
            if constexpr (!kBf16) {
                const float limit = __int_as_float(0x7F7FFFFF);
                float here = 0.0f;                // (a NaN is no maximum)
#pragma unroll
                for (int q = 0; q < kN; ++q) here = fmaxf(here, fmaxf(fabsf(dg[q]), fabsf(du[q])));
                if (here > limit) {
                    here = 0.0f;
#pragma unroll
                    for (int q = 0; q < kN; ++q) {
                        if (fabsf(dg[q]) <= limit) here = fmaxf(here, fabsf(dg[q]));
                        if (fabsf(du[q]) <= limit) here = fmaxf(here, fabsf(du[q]));
                    }
                }
                top = fmaxf(top, here);
            }
            if constexpr (kVec) {
                reinterpret_cast<uint4 *>(dp)[i] =
                    make_uint4(round2(dg[0], dg[1]), round2(dg[2], dg[3]), round2(dg[4], dg[5]), round2(dg[6], dg[7]));
                reinterpret_cast<uint4 *>(dp + p.M)[i] =
                    make_uint4(round2(du[0], du[1]), round2(du[2], du[3]), round2(du[4], du[5]), round2(du[6], du[7]));
            } else {
                const uint32_t x = round2(dg[0], du[0]);
                dp[i] = static_cast<uint16_t>(x);
                dp[p.M + i] = static_cast<uint16_t>(x >> 16);
            }
        }
        if (blockIdx.x == 0)                      // the products read whole 16-byte units of a row
            for (int64_t c = 2 * static_cast<int64_t>(p.M) + lane; c < p.dp_units; c += p.lanes) dp[c] = 0;
    }
    if constexpr (!kBf16) {
        if (!p.again) {                           // (a maximum: the same in any order)
            const uint32_t all = largest_of_all(__float_as_uint(top), tops);
            if (threadIdx.x == 0 && all != 0) atomicMax(reinterpret_cast<uint32_t *>(p.room + 1), all);
        }
    }
}

}  // namespace tn
