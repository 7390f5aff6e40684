// What the products of a language model's layers do with their accumulators
// (tn_grouped_kernel's operations from kGrGated on).
//
// A sink gets a warp's 32 x 32 piece of the accumulator as the kernel's epilogue
// reads it: register v[q][4 i + 2 h + c] of lane t is column 8 i + 2 (t % 4) + c
// and lane 16 q + 8 h + t / 4 of the piece.  Columns are the result's rows
// (tokens), lanes its contiguous index.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_bf16.h>

#include "grouped_ptx.cuh"

namespace tn {

// (gemm_act_t of the C ABI)
enum Act : int { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2 };

struct SinkParams {
    int32_t act;                     // gated: Act
    float *pre;                      // gated: the products themselves, T rows of [gate | up], or NULL
    int64_t pre_ld;
    const int64_t *targets;          // loss: a class per token; negative: ignored
    float2 *stats;                   // loss: [ceil(classes / 32)][T] maximum, sum of exp(z - maximum)
    float *z_target;                 // loss: [T] the target's logit
    const float2 *rows;              // loss gradient: [T] (-log-sum-exp / log 2, factor)
    const float *lse;                // loss gradient: [T] the log-sum-exps
    int32_t first, classes;          // loss gradient: the piece's first class, and how many
    float *sum;                      // parts added up: FP32 sums, one result for each part
    int64_t sum_ld, sum_stride;
    int32_t add;                     // parts added up: AddPart
    const float *out_scale;          // the result's factor (one float), or NULL
};

enum AddPart : int { kAddOnly = 0, kAddFirst = 1, kAddMore = 2, kAddLast = 3 };

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(x) - 1, for small x by the exponential's series (six terms: below 1/4 the seventh is 2^-24 of it).
__device__ __forceinline__ float exp_less_one(float x)
{
    float y = fmaf(x, 1.0f / 6.0f, 1.0f);
    y = fmaf(x * 0.2f, y, 1.0f);
    y = fmaf(x * 0.25f, y, 1.0f);
    y = fmaf(x * (1.0f / 3.0f), y, 1.0f);
    y = fmaf(x * 0.5f, y, 1.0f);
    return fabsf(x) < 0.25f ? x * y : ex2(x * kLog2e) - 1.0f;
}

// 1 / (1 + exp(-x)) (relative error about 2^-21 and |x| 2^-23, the argument's rounding).  Beyond
// exp(-x) = 2^126 the quotient, less than FP32's smallest normal number, is 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + ex2(-x * kLog2e)); }

// The normal distribution function, erfc(-x / sqrt 2) / 2: for x < 0 t q(t) exp(-x^2 / 2) with t =
// 1 / (1 + 0.3 |x|) (the form of Hastings' approximations, 1955; q's coefficients fitted here
// for the least largest relative error, 1.7e-7), for x > 0 what that leaves of 1.  In FP32 x^2 is rounded before
// the exponential, which adds up to x^2 2^-25: 1.3e-6 in all at -5, 7e-6 at -13, where the function is 6e-39.  The results
// have 16 bits, half a step of 2^-9 or 2^-12, so that is a hundredth of one at most.  Shorter than
// erfcf: 3001 gated rows over 8 experts of 1024 x 2048 31.1 -> 27.4 us, their gradient 69.9 -> 66.0.
__device__ __forceinline__ float normal_below(float x)
{
    const float t = __fdividef(1.0f, fmaf(0.3f, fabsf(x), 1.0f));
    float q = fmaf(0.0354237093f, t, -0.156158348f);
    q = fmaf(q, t, 0.204556627f);
    q = fmaf(q, t, -0.0520338858f);
    q = fmaf(q, t, 0.12769171f);
    q = fmaf(q, t, 0.100175964f);
    q = fmaf(q, t, 0.120712134f);
    q = fmaf(q, t, 0.119632007f);
    const float y = q * t * ex2(-0.5f * kLog2e * x * x);
    return x > 0.0f ? 1.0f - y : y;
}

// y(x) with act(x) = x y(x):
//   silu       sigmoid(x)
//   gelu       the normal distribution function
//   gelu_tanh  (1 + tanh z) / 2 = sigmoid(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3)
template <int kAct>
__device__ __forceinline__ float act_factor(float x)
{
    if constexpr (kAct == kActSilu) return sigmoid(x);
    if constexpr (kAct == kActGelu) return normal_below(x);
    return sigmoid(1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.0f));
}

// act'(x) = y + x y'(x), y = act_factor(x).
template <int kAct>
__device__ __forceinline__ float act_slope(float x, float y)
{
    if constexpr (kAct == kActSilu) return fmaf(x * y, 1.0f - y, y);
    if constexpr (kAct == kActGelu)
        return fmaf(x, 0.3989422804014327f * ex2(-0.5f * kLog2e * x * x), y);
    return fmaf(x * y * (1.0f - y), 1.5957691216057308f * fmaf(0.134145f * x, x, 1.0f), y);
}

template <int kOp>
struct Sink;

// ------------------------------------------------------------------ gated projections
// The L operand's rows alternate, 16 gate rows and the 16 up rows beside them, so
// a thread's v[0] and v[1] hold the gate and the up product of the same 16 results, and
// the products need not go to memory.  On GB300 the activation hides behind the next tile's
// products: 3001 rows over 8 experts of 1024 x 2048 take 26.1 us with silu, 26.6 with gelu_tanh
// and 27.4 with gelu (the plain product of as many rows 25.7); the products' 25 MB in FP32 cost 4
// more.  4096 tokens over 14336 x 4096: 546 to 570 us on different boxes, 0.91 to 0.87 of the
// measured burst rate.
template <>
struct Sink<4 /* kGrGated */> {
    template <int kAct, bool kBf16, class Store>
    static __device__ __forceinline__ void store_h(const SinkParams &k, const Store &store, const uint32_t (&v)[2][16],
                                                   uint16_t *out, int32_t wide, bool vec, int32_t rows)
    {
        const int lane = store.lane;
        uint32_t h[4][2];                         // [8 columns][8 lanes]
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float x[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float g = __uint_as_float(v[0][2 * r + c]), u = __uint_as_float(v[1][2 * r + c]);
                x[c] = g * act_factor<kAct>(g) * u;
            }
            h[r >> 1][r & 1] = kBf16 ? ptx::pack_bf16x2(x[0], x[1]) : ptx::pack_f16x2(x[0], x[1]);
        }
        // Staging rows of 16 results (32 bytes), their two 16-byte pieces exchanged in
        // every other four rows, so that eight rows' pieces meet no bank twice.
        auto piece = [&](int row, int c) { return store.base + row * 32 + ((c ^ ((row >> 2) & 1)) << 4); };
        __syncwarp();                             // the last step's pieces have been read
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            ptx::stmatrix_x4_trans(piece(8 * i + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1), h[i][0], h[i][1],
                                   h[i + 1][0], h[i + 1][1]);
        __syncwarp();
        if (vec) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int32_t r = 16 * q + (lane >> 1);
                if (r < rows)
                    *reinterpret_cast<uint4 *>(out + r * store.ld + 8 * (lane & 1)) = ptx::ld_shared_v4(piece(r, lane & 1));
            }
        } else {
            const int32_t m = lane & 15, n = rows < 32 ? rows : 32;
            if (m < wide)
                for (int32_t r = lane >> 4; r < n; r += 2)
                    out[r * store.ld + m] = ptx::ld_shared_u16(piece(r, m >> 3) + 2 * (m & 7));
        }
    }

    template <class Params, class Store>
    static __device__ __forceinline__ void step(const Params &p, const Store &store, const uint32_t (&v)[2][16],
                                                int32_t l0, int64_t row, int32_t rows, int32_t part)
    {
        const SinkParams &k = p.sink;
        const int lane = store.lane;
        const int32_t wide = p.l_extent - l0 < 16 ? p.l_extent - l0 : 16;
        if (k.pre) {
            // Eight lanes hold eight neighbouring results of a row: whole sectors.
            const int32_t c0 = 2 * (lane & 3), m0 = lane >> 2;
            float *gate = k.pre + (row + c0) * k.pre_ld + l0 + m0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float *at = gate + (8 * i + c) * k.pre_ld;
                    if (8 * i + c0 + c < rows) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (m0 + 8 * h < wide) {
                                at[8 * h] = __uint_as_float(v[0][4 * i + 2 * h + c]);
                                at[p.l_extent + 8 * h] = __uint_as_float(v[1][4 * i + 2 * h + c]);
                            }
                    }
                }
        }
        uint16_t *out = p.out + row * p.out_ld + l0;
        const bool vec = p.out_vec != 0 && wide == 16;
        auto all = [&](auto bf16) {
            constexpr bool kBf16 = decltype(bf16)::value;
            switch (k.act) {
            case kActSilu: return store_h<kActSilu, kBf16>(k, store, v, out, wide, vec, rows);
            case kActGelu: return store_h<kActGelu, kBf16>(k, store, v, out, wide, vec, rows);
            default: return store_h<kActGeluTanh, kBf16>(k, store, v, out, wide, vec, rows);
            }
        };
        if (p.out_fmt != 0)
            all(Flag<true>{});
        else
            all(Flag<false>{});
    }

    template <bool kValue>
    struct Flag {
        static constexpr bool value = kValue;
    };
};

// ------------------------------------------------------------------ loss
// A token's 32 logits of the piece become their maximum and the sum of their
// exponentials above it, both in FP32; cross_entropy_join_kernel adds up the
// pieces.  A column's logits lie in eight lanes, four in each, and a lane has four of
// eight columns.  So the columns' maxima and sums are merged by halving: each turn a
// lane passes on half of its columns, 7 exchanges for 8 columns, and 7 more take the
// maxima back to all lanes before the exponentials.  4096 tokens over 8192 classes of 4096 take
// 153 us on GB300 (0.93 of the measured burst rate); 1021 over 32003 of 1024 52.1, of which the
// products alone would take 35: over short sums the epilogue is longer than a tile's products.
template <>
struct Sink<5 /* kGrLossStats */> {
    static __device__ __forceinline__ void merge(float &m, float &s, float om, float os)
    {
        const float top = fmaxf(m, om);
        // (a piece without a logit above -inf: nothing to scale)
        const float a = m == top ? s : s * ex2((m - top) * kLog2e), b = om == top ? os : os * ex2((om - top) * kLog2e);
        m = top;
        s = a + b;
    }

    // x[j]: the lane's share of column 2 i + c = j; leaves the whole of its own column, 4 b4 +
    // 2 b3 + b2 (bn: bit n of the lane), in x[0].
    template <class Op>
    static __device__ __forceinline__ void halve(float (&x)[8], int lane, Op op)
    {
#pragma unroll
        for (int d = 4, bit = 16; d >= 1; d /= 2, bit /= 2) {
            const bool upper = lane & bit;
#pragma unroll
            for (int j = 0; j < d; ++j) {
                const float other = __shfl_xor_sync(0xffffffffu, upper ? x[j] : x[j + d], bit);
                x[j] = op(upper ? x[j + d] : x[j], other);
            }
        }
    }

    template <class Params, class Store>
    static __device__ __forceinline__ void step(const Params &p, const Store &store, const uint32_t (&v)[2][16],
                                                int32_t l0, int64_t row, int32_t rows, int32_t part)
    {
        if (l0 >= p.l_extent) return;             // (past the last class: no piece)
        const SinkParams &k = p.sink;
        const int lane = store.lane;
        const float none = __int_as_float(0xff800000);
        // (classes past the last are left out)
        const int32_t left = p.l_extent - l0 - (lane >> 2);     // of the lane's classes 0, 8, 16 and 24
        const bool whole = p.l_extent - l0 >= 32;
        auto logit = [&](int j, int q) { return __uint_as_float(v[q >> 1][4 * (j >> 1) + 2 * (q & 1) + (j & 1)]); };
        float x[8], m[8];
        if (whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = fmaxf(fmaxf(logit(j, 0), logit(j, 1)), fmaxf(logit(j, 2), logit(j, 3)));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = none;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (8 * q < left) m[j] = fmaxf(m[j], logit(j, q));
            }
        }
        halve(m, lane, [](float a, float b) { return fmaxf(a, b); });
        const float top = m[0];
#pragma unroll
        for (int d = 1, bit = 4; d <= 4; d *= 2, bit *= 2) {
            const bool upper = lane & bit;
#pragma unroll
            for (int j = 0; j < d; ++j) {
                const float other = __shfl_xor_sync(0xffffffffu, m[j], bit);
                const float mine = m[j];
                m[j] = upper ? other : mine;
                m[j + d] = upper ? mine : other;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // (a maximum of -inf: of logits that all are)
            const float from = m[j] == none ? 0.0f : -m[j] * kLog2e;
            float e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) e[q] = ex2(fmaf(logit(j, q), kLog2e, from));
            if (!whole)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (8 * q >= left) e[q] = 0.0f;
            x[j] = (e[0] + e[1]) + (e[2] + e[3]);
        }
        halve(x, lane, [](float a, float b) { return a + b; });
        const int32_t own = 4 * (lane >> 4 & 1) + 2 * (lane >> 3 & 1) + (lane >> 2 & 1);
        const int32_t col = 8 * (own >> 1) + 2 * (lane & 3) + (own & 1);
        // (top / log 2 was rounded: by 2^-19 at a top of 30, which all of the column's exponentials share)
        if (top != none) x[0] *= fmaf(-kLn2, fmaf(top, kLog2e, -top * kLog2e), 1.0f);
        if (col < rows) k.stats[static_cast<int64_t>(l0 >> 5) * p.T + row + col] = make_float2(top, x[0]);
        // the target's logit, where this piece has it
        int64_t at = -1;
        if (lane < rows) at = __ldg(k.targets + row + lane) - l0;
        uint32_t hits = __ballot_sync(0xffffffffu, at >= 0 && at < 32 && l0 + at < p.l_extent);
        while (hits) {
            const int32_t c = __ffs(hits) - 1;
            hits &= hits - 1;
            const int32_t q = __shfl_sync(0xffffffffu, static_cast<int32_t>(at), c);
            if ((lane & 3) == ((c & 7) >> 1) && lane >> 2 == (q & 7)) {
                const int32_t want = 16 * (q >> 4) + 4 * (c >> 3) + 2 * (q >> 3 & 1) + (c & 1);
#pragma unroll
                for (int r = 0; r < 32; ++r)
                    if (r == want) k.z_target[row + c] = __uint_as_float(v[r >> 4][r & 15]);
            }
        }
    }
};

// d = (exp(z - lse) - [m = target]) factor, rounded to the operands' type: what the
// tensor cores multiply in both gradients.  At the target exp(x) - 1 is taken as such, which keeps what is left of
// a probability near one.  (The factors are shares of the largest, in
// fp16 times 2^13, see cross_entropy_rows_kernel; d then keeps its relative precision
// down to 2^-27 of it.)  Classes past the piece's end are zeros: the
// products over the piece read them.  A piece of 16384 classes of 4096 for 4096 tokens
// takes 336 us on GB300, 0.85 of the measured burst rate (306 as one sum a logit).
template <>
struct Sink<6 /* kGrLossGrad */> {
    template <class Params, class Store>
    static __device__ __forceinline__ void step(const Params &p, const Store &store, const uint32_t (&v)[2][16],
                                                int32_t l0, int64_t row, int32_t rows, int32_t part)
    {
        const SinkParams &k = p.sink;
        const int lane = store.lane;
        float d[2][16];
        int64_t at = -1;
        if (lane < rows) at = __ldg(k.targets + row + lane) - k.first - l0;
        const bool hits = __any_sync(0xffffffffu, at >= 0 && at < 32);
        float2 r[8];                              // of the lane's columns: -lse / log 2, factor
        bool some = false;                        // a token that is ignored among them
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t col = 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
            r[j] = col < rows ? __ldg(k.rows + row + col) : make_float2(0.0f, 1.0f);
            some |= r[j].y == 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int b = 4 * (j >> 1) + 2 * (q & 1) + (j & 1);
                d[q >> 1][b] = ex2(fmaf(__uint_as_float(v[q >> 1][b]), kLog2e, r[j].x));
            }
        if (hits) {                               // targets among these classes: all at once
            const int32_t own = at >= 0 && at < 32 ? static_cast<int32_t>(at) : -1;
            const float own_lse = lane < rows ? __ldg(k.lse + row + lane) : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int32_t col = 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
                const int32_t m = __shfl_sync(0xffffffffu, own, col) - (lane >> 2);       // 8 q: the lane's class q
                const float lse = __shfl_sync(0xffffffffu, own_lse, col);
                float z = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (m == 8 * q) z = __uint_as_float(v[q >> 1][4 * (j >> 1) + 2 * (q & 1) + (j & 1)]);
                const float left = exp_less_one(z - lse);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (m == 8 * q) d[q >> 1][4 * (j >> 1) + 2 * (q & 1) + (j & 1)] = left;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q >> 1][4 * (j >> 1) + 2 * (q & 1) + (j & 1)] *= r[j].y;
        const int32_t left = k.classes - l0 - (lane >> 2);
        if (__any_sync(0xffffffffu, some || left < 25)) {
            // an ignored token's logits may be anything; and what the classes leave of the last 32
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (r[j].y == 0.0f || 8 * q >= left) d[q >> 1][4 * (j >> 1) + 2 * (q & 1) + (j & 1)] = 0.0f;
        }
        uint32_t bits[2][16];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 16; ++i) bits[q][i] = __float_as_uint(d[q][i]);
        uint16_t *out = p.out + row * p.out_ld + l0;
        if (p.out_fmt != 0)
            store.template step<true, false>(bits, out, rows, nullptr);
        else
            store.template step<false, false>(bits, out, rows, nullptr);
    }
};

template <>
struct Sink<11 /* kGrLossGradLong */> : Sink<6> {};

// ------------------------------------------------------------------ sums in parts
// A token gradient's sum may be cut twice.  Pieces of the vocabulary are launches: the
// first leaves FP32 sums, the next ones add theirs (each element once a launch, so the
// order is the launches'), and the last one's result is rounded once.  And where a
// launch's tiles are few, parts of its sum are tiles of their own, each part with
// sums of its own; parts_join_kernel adds them up in their order.  A piece of 16384 classes
// for 4096 tokens of 4096: 347 us on GB300, of which the FP32 sums (64 MiB, read and written
// once) take some 30.
template <>
struct Sink<7 /* kGrGradBAdd */> {
    template <class Params, class Store>
    static __device__ __forceinline__ void step(const Params &p, const Store &store, const uint32_t (&v)[2][16],
                                                int32_t l0, int64_t row, int32_t rows, int32_t part)
    {
        const SinkParams &k = p.sink;
        const int lane = store.lane;
        const int32_t c0 = 2 * (lane & 3), m0 = lane >> 2;
        float *sum = k.sum + part * k.sum_stride + (row + c0) * k.sum_ld + l0 + m0;
        uint32_t x[2][16];
        const float scale = k.out_scale ? __ldg(k.out_scale) : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float *at = sum + (8 * i + c) * k.sum_ld;
                const bool inside = k.add != kAddOnly && 8 * i + c0 + c < rows;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int b = 4 * i + 2 * (q & 1) + c;
                    float y = __uint_as_float(v[q >> 1][b]);
                    if (inside && m0 + 8 * q < store.wide) {
                        if (k.add == kAddFirst)
                            at[8 * q] = y;
                        else if (k.add == kAddMore)
                            asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(at + 8 * q), "f"(y) : "memory");
                        else
                            y += at[8 * q];
                    }
                    x[q >> 1][b] = __float_as_uint(y * scale);
                }
            }
        if (k.add == kAddFirst || k.add == kAddMore) return;
        uint16_t *out = p.out + row * p.out_ld + l0;
        if (p.out_fmt != 0)
            store.template step<true, false>(x, out, rows, nullptr);
        else
            store.template step<false, false>(x, out, rows, nullptr);
    }
};

// Gradients whose sums carry a scale: the loss gradient's (one group), or that of fp16's
// gated dP.  Nothing else is added to the plain ones: 16384 classes of 4096, 4096 tokens, 316 us
// on GB300 (0.90 of the burst rate).
struct ScaledSink {
    template <class Params, class Store>
    static __device__ __forceinline__ void step(const Params &p, const Store &store, const uint32_t (&v)[2][16],
                                                int32_t l0, int64_t row, int32_t rows, int32_t group)
    {
        const float scale = p.sink.out_scale ? __ldg(p.sink.out_scale) : 1.0f;
        uint32_t x[2][16];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int b = 0; b < 16; ++b) x[q][b] = __float_as_uint(__uint_as_float(v[q][b]) * scale);
        uint16_t *out = p.out + group * p.out_stride + row * p.out_ld + l0;
        if (p.out_fmt != 0)
            store.template step<true, false>(x, out, rows, nullptr);
        else
            store.template step<false, false>(x, out, rows, nullptr);
    }
};
template <>
struct Sink<8 /* kGrGradAOne */> : ScaledSink {};
template <>
struct Sink<9 /* kGrGradBScaled */> : ScaledSink {};
template <>
struct Sink<10 /* kGrGradAScaled */> : ScaledSink {};

}  // namespace tn
