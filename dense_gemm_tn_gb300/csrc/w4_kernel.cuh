// Products with 4-bit weights and a scale per group of terms, for few tokens, and
// the quantiser that makes such weights.
//
//     C[n, m] = sum_g scale[m, g] (sum over k in g of q[m, k] B[n, k])
//
// q: signed 4-bit integers, two to a byte, the even term in the low half.  What
// bounds the product is the read of the codes, so the kernel is built around wide
// loads of them, many in flight: each warp takes kTilesM tiles of 16 rows m and
// every so many-th block of 128 terms (64 bytes of a row, 16 a lane), all tokens at
// once; a CTA's warps share the rows and split the sum, joined in shared memory in
// the order of the warps.
//
// Integers are exact in both 16-bit types, so they are multiplied as such by
// mma.m16n8k16 (a warp's own instruction: at up to 64 tokens its rate is not what
// bounds, and it takes its operands from registers, where the codes arrive), a
// group's sum is FP32, and the scale multiplies that sum, in FP32.
//
// Which terms an MMA step pairs does not matter as long as both operands agree.  A
// lane's word of eight codes, masked where it stands, gives the terms (0, 4), (1, 5),
// (2, 6) and (3, 7) in 16-bit halves with one shift each; the tokens' halves are put
// in that order by byte permutations, once for all of a warp's rows.
//   groups of 128 terms or more: word j of lane t are the terms 32 t + 8 j .. + 7
//   smaller ones: the four lanes of a row exchange their words first, so that an MMA
//   step's terms lie in 32 consecutive ones: word j of lane t are 32 j + 8 t .. + 7
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm103_ptx.cuh"

namespace w4 {

namespace ptx = tn::ptx;

constexpr int kBlock = 128;                      // terms of a warp's step

struct ProductParams {
    const uint8_t *a;                // codes, M rows of lda bytes
    int64_t lda;
    const uint16_t *scale;           // M rows of lds scales
    int64_t lds;
    const uint16_t *b;               // tokens, N rows
    int64_t ldb;
    uint16_t *c;                     // N rows of M
    int64_t ldc;
    int32_t M, N, K;
    int32_t group;                   // terms per scale: 32, 64, 128 or 256
    int32_t groups;                  // scales of a row
    int32_t token_tiles;             // tiles of 8 kTilesN tokens
    bool words;                      // (rows not on 16-byte boundaries) the operands start on 4-byte ones
};

// 16 bytes from p on, which all count, wherever p is: four aligned words cut, or
// five; those that hold none of them are not read.
__device__ __forceinline__ uint4 load_words(const uint8_t *p)
{
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3u;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p - s);
    uint32_t x[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(w + i);
    x[4] = s ? __ldg(w + 4) : 0u;
    return make_uint4(__funnelshift_r(x[0], x[1], 8 * s), __funnelshift_r(x[1], x[2], 8 * s),
                      __funnelshift_r(x[2], x[3], 8 * s), __funnelshift_r(x[3], x[4], 8 * s));
}

// 16 bytes from p on, of which the first `valid` count, the rest zeros; nothing else
// is read.
__device__ __noinline__ uint4 load_part(const uint8_t *p, int32_t valid)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (4 * i + q < valid) r[i] |= static_cast<uint32_t>(__ldg(p + 4 * i + q)) << (8 * q);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The eight codes of a word as four pairs of 16-bit floats: (0, 4), (1, 5), (2, 6), (3, 7).
// A code's four bits, the top one flipped, are q + 8 in the low bits of 1024 (fp16)
// or 128 (bf16), whose steps are 1 there.
template <bool kBf16>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4])
{
    constexpr uint32_t kMagic = kBf16 ? 0x43084308u : 0x64086408u;      // (xor 8: the flip)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t x;
        asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(x) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(kMagic));
        if constexpr (kBf16)
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(x), "r"(0x43084308u));
        else
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(x), "r"(0x64086408u));
    }
}

template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool kBf16>
__device__ __forceinline__ float to_float(uint16_t x)
{
    return kBf16 ? __uint_as_float(static_cast<uint32_t>(x) << 16) : __half2float(__ushort_as_half(x));
}

template <bool kBf16>
__device__ __forceinline__ uint16_t from_float(float x)
{
    return kBf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// The words of four neighbouring lanes transposed: lane t's word j becomes lane j's word t.
__device__ __forceinline__ void exchange(uint4 &v, int t)
{
    uint32_t x[4] = {v.x, v.y, v.z, v.w};
    const bool odd = t & 1, high = t & 2;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {             // words i, i + 1 with the lane beside
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? x[i] : x[i + 1], 1);
        if (odd) x[i] = got;
        else x[i + 1] = got;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {                // words i, i + 2 with the lane two on
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? x[i] : x[i + 2], 2);
        if (high) x[i] = got;
        else x[i + 2] = got;
    }
    v = make_uint4(x[0], x[1], x[2], x[3]);
}

// Floats of shared memory that one warp leaves its sums in: 8 kTilesN tokens of
// 16 kTilesM rows, four apart so that a fragment's stores meet no bank twice.
__host__ __device__ constexpr int part_floats(int tiles_m, int tiles_n) { return 8 * tiles_n * (16 * tiles_m + 4); }

template <bool kBf16, int kTilesM, int kTilesN, bool kWhole, bool kAligned>
__global__ void __launch_bounds__(512) product_kernel(const __grid_constant__ ProductParams p)
{
    extern __shared__ float parts[];
    constexpr int kRows = 16 * kTilesM, kTokens = 8 * kTilesN, kLd = kRows + 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int32_t tile = static_cast<int32_t>(blockIdx.x) / p.token_tiles;
    const int32_t n0 = (static_cast<int32_t>(blockIdx.x) - tile * p.token_tiles) * kTokens;
    const int32_t m0 = tile * kRows;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int32_t blocks = (p.K + kBlock - 1) / kBlock, row_bytes = (p.K + 1) / 2;
    const uint8_t *a_row[kTilesM][2];
    const uint16_t *s_row[kTilesM][2];
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {            // (rows past the last are the last again, and not stored)
            const int32_t m = min(m0 + 16 * i + 8 * h + g, p.M - 1);
            a_row[i][h] = p.a + m * p.lda + 16 * t;
            s_row[i][h] = p.scale + m * p.lds;
        }
    const uint16_t *b_row[kTilesN];
    bool held[kTilesN];
#pragma unroll
    for (int i = 0; i < kTilesN; ++i) {
        const int32_t n = n0 + 8 * i + g;
        held[i] = n < p.N;
        b_row[i] = p.b + (held[i] ? n : 0) * p.ldb + (kWhole ? 32 : 8) * t;
    }

    struct Step {
        uint4 code[kTilesM][2];
        uint16_t scale[kTilesM][2];
    };
    // A block that can be read without a look at its ends: the whole of it is there, and
    // where words are cut, the bytes that the last one takes along are (the next block's,
    // or the next row's).
    const bool last_tile = m0 + kRows >= p.M;
    auto plain = [&](int32_t b) {
        if (kAligned) return (b + 1) * kBlock <= p.K;
        return p.words && b + (last_tile ? 2 : 1) < blocks;
    };
    auto load = [&](int32_t b, Step &s) {
        const bool whole = plain(b);
        const int32_t off = b * (kBlock / 2), valid = row_bytes - off - 16 * t;
        const int32_t grp = (b * kBlock + 32 * t) / p.group;
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *at = a_row[i][h] + off;
                if (whole)
                    s.code[i][h] = kAligned ? __ldg(reinterpret_cast<const uint4 *>(at)) : load_words(at);
                else
                    s.code[i][h] = load_part(at, valid);
                s.scale[i][h] = grp < p.groups ? __ldg(s_row[i][h] + grp) : uint16_t(0);
            }
    };
    float acc[kTilesM][kTilesN][4] = {};

    auto compute = [&](int32_t b, Step &s) {
        const bool whole = plain(b);
        if constexpr (!kWhole) {
#pragma unroll
            for (int i = 0; i < kTilesM; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) exchange(s.code[i][h], t);
        }
        float part[kTilesM][kTilesN][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // the tokens' eight terms of this word
            uint32_t x[kTilesN][4];
            const int32_t k = b * kBlock + (kWhole ? 32 * t + 8 * j : 32 * j + 8 * t);
#pragma unroll
            for (int i = 0; i < kTilesN; ++i) {
                const uint16_t *at = b_row[i] + b * kBlock + (kWhole ? 8 : 32) * j;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (held[i]) {
                    if (whole)
                        v = kAligned ? __ldg(reinterpret_cast<const uint4 *>(at))
                                     : load_words(reinterpret_cast<const uint8_t *>(at));
                    else
                        v = load_part(reinterpret_cast<const uint8_t *>(at), 2 * min(p.K - k, 8));
                }
                x[i][0] = __byte_perm(v.x, v.z, 0x5410);
                x[i][1] = __byte_perm(v.x, v.z, 0x7632);
                x[i][2] = __byte_perm(v.y, v.w, 0x5410);
                x[i][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < kTilesM; ++i) {
                const uint4 lo = s.code[i][0], hi = s.code[i][1];
                uint32_t u[4], v[4];
                widen<kBf16>(j == 0 ? lo.x : j == 1 ? lo.y : j == 2 ? lo.z : lo.w, u);
                widen<kBf16>(j == 0 ? hi.x : j == 1 ? hi.y : j == 2 ? hi.z : hi.w, v);
                const bool begin = !kWhole || j == 0, end = !kWhole || j == 3;
#pragma unroll
                for (int n = 0; n < kTilesN; ++n) {
                    float(&d)[4] = part[i][n];
                    if (begin) d[0] = d[1] = d[2] = d[3] = 0.0f;
                    mma<kBf16>(d, u[0], v[0], u[1], v[1], x[n][0], x[n][1]);
                    mma<kBf16>(d, u[2], v[2], u[3], v[3], x[n][2], x[n][3]);
                }
                if (end) {
                    float s0 = to_float<kBf16>(s.scale[i][0]), s1 = to_float<kBf16>(s.scale[i][1]);
                    if constexpr (!kWhole) {     // lane j of the four has the scales of these 32 terms
                        s0 = __shfl_sync(0xffffffffu, s0, (lane & ~3) | j);
                        s1 = __shfl_sync(0xffffffffu, s1, (lane & ~3) | j);
                    }
#pragma unroll
                    for (int n = 0; n < kTilesN; ++n) {
                        acc[i][n][0] = fmaf(s0, part[i][n][0], acc[i][n][0]);
                        acc[i][n][1] = fmaf(s0, part[i][n][1], acc[i][n][1]);
                        acc[i][n][2] = fmaf(s1, part[i][n][2], acc[i][n][2]);
                        acc[i][n][3] = fmaf(s1, part[i][n][3], acc[i][n][3]);
                    }
                }
            }
        }
    };

    // one block's codes on their way while another's are multiplied
    Step s0, s1;
    int32_t b = warp;
    if (b < blocks) load(b, s0);
    while (b < blocks) {
        if (b + warps < blocks) load(b + warps, s1);
        compute(b, s0);
        b += warps;
        if (b >= blocks) break;
        if (b + warps < blocks) load(b + warps, s0);
        compute(b, s1);
        b += warps;
    }

    float *mine = parts + warp * part_floats(kTilesM, kTilesN);
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int n = 0; n < kTilesN; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) mine[(8 * n + 2 * t + (r & 1)) * kLd + 16 * i + 8 * (r >> 1) + g] = acc[i][n][r];
    __syncthreads();
    for (int32_t i = threadIdx.x; i < kRows * kTokens; i += blockDim.x) {
        const int32_t n = i / kRows, m = i - n * kRows;
        if (n0 + n >= p.N || m0 + m >= p.M) continue;
        float sum = 0.0f;
        for (int w = 0; w < warps; ++w) sum += parts[w * part_floats(kTilesM, kTilesN) + n * kLd + m];
        p.c[(n0 + n) * p.ldc + m0 + m] = from_float<kBf16>(sum);
    }
}

// ------------------------------------------------------------------ quantiser
//     scale[r, g] = amax times the float next to 1 / 7, in FP32, rounded to 16 bits
//     q[r, c]     = round(x / scale) of the exact quotient, ties to even, within -8 .. 7
// A warp takes 256 terms of a row at a time, eight a lane, so a group's maximum is
// one of up to 32 neighbouring lanes.  Bound by the read of x.
constexpr int kQuantThreads = 256, kQuantSeg = 256;

struct QuantParams {
    const void *x;
    int64_t ldx;
    uint8_t *q;
    int64_t ldq;
    uint16_t *scale;
    int64_t lds;
    int64_t rows;
    int32_t cols, group;
    int32_t segs;                    // of a row
    bool bf16;                       // the scales' type
    bool vec;                        // x's rows on 16-byte boundaries, q's on 4-byte ones
};

enum In : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

// round(x / s) for s > 0: the quotient by a reciprocal, put right by the exact rest
// x - q s (q s has at most 15 bits, and the rest is below s: no bit is lost).
__device__ __forceinline__ int32_t code(float x, float s, float inverse)
{
    float q = rintf(x * inverse);
    q = fminf(fmaxf(q, -16.0f), 16.0f);
    const float rest2 = 2.0f * fmaf(-q, s, x);
    const bool odd = static_cast<int32_t>(q) & 1;
    if (rest2 > s || (rest2 == s && odd)) q += 1.0f;
    if (rest2 < -s || (rest2 == -s && odd)) q -= 1.0f;
    const int32_t i = static_cast<int32_t>(q);
    return i < -8 ? -8 : i > 7 ? 7 : i;
}

template <int kIn>
__global__ void __launch_bounds__(kQuantThreads) quant_kernel(const QuantParams p)
{
    constexpr int kElem = kIn == kF32 ? 4 : 2;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t units = p.rows * p.segs, step = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const int64_t r = u / p.segs;
        const int32_t c = static_cast<int32_t>(u - r * p.segs) * kQuantSeg + 8 * lane;
        const uint8_t *src = static_cast<const uint8_t *>(p.x) + (r * p.ldx + c) * kElem;
        float x[8];
        if (p.vec && c + 8 <= p.cols) {
            if constexpr (kIn == kF32) {
                const float4 a = __ldcs(reinterpret_cast<const float4 *>(src));
                const float4 b = __ldcs(reinterpret_cast<const float4 *>(src) + 1);
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
                x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            } else {
                const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(src));
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = to_float<kIn == kBF16>(static_cast<uint16_t>(w[i]));
                    x[2 * i + 1] = to_float<kIn == kBF16>(static_cast<uint16_t>(w[i] >> 16));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = 0.0f;
                if (c + i < p.cols) {
                    if constexpr (kIn == kF32)
                        x[i] = reinterpret_cast<const float *>(src)[i];
                    else
                        x[i] = to_float<kIn == kBF16>(reinterpret_cast<const uint16_t *>(src)[i]);
                }
            }
        }
        uint32_t top = 0;                        // as bits: a NaN is above all others
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        for (int d = p.group / 16; d >= 1; d /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        float s = __fmul_rn(__uint_as_float(top), 1.0f / 7.0f);
        const uint16_t s16 = p.bf16 ? from_float<true>(s) : from_float<false>(s);
        s = p.bf16 ? to_float<true>(s16) : to_float<false>(s16);
        const bool finite = s < __int_as_float(0x7f800000);
        uint32_t word = 0;
        if (finite && s > 0.0f) {
            // (a scale whose reciprocal is no normal number: both times 2^96)
            const float up = s < 0x1p-96f ? 0x1p96f : 1.0f;
            const float su = s * up, inverse = __fdividef(1.0f, su);
#pragma unroll
            for (int i = 0; i < 8; ++i) word |= (static_cast<uint32_t>(code(x[i] * up, su, inverse)) & 15u) << (4 * i);
        }
        if (c < p.cols) {
            uint8_t *dst = p.q + r * p.ldq + c / 2;
            if (p.vec && c + 7 <= p.cols) {
                *reinterpret_cast<uint32_t *>(dst) = word;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + 2 * i < p.cols) dst[i] = static_cast<uint8_t>(word >> (8 * i));
            }
            if (c % p.group == 0) p.scale[r * p.lds + c / p.group] = finite ? s16 : uint16_t(0x7FFF);
        }
    }
}

}  // namespace w4
