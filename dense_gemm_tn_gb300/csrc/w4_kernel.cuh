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
// 8192 x 8192 in groups of 128 and one token take 11.1 us on GB300 (3.1 TB/s), 28672 x 4096
// 19.0: neither memory (30 % busy) nor an arithmetic pipe (27 %) bounds them but the
// warps' waits for tokens and scales, at 16 warps an SM, whose registers hold them a block ahead.
// (Three CTAs an SM with tokens read late: 8192 x 8192 15.1 us, with the registers cut 19.5; tokens and
// codes shared as in wide_kernel 13.5 to 18.8.)
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
    int32_t group_shift;             // terms per scale: 32, 64, 128 or 256, as a power of two
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
[[maybe_unused]] static __device__ __noinline__ uint4 load_part(const uint8_t *p, int32_t valid)
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
// (Integers widened by their place in a half's mantissa: Kim, Henry, Fahim and Awadalla, 2022.)
// A code's four bits, the top one flipped, are q + 8 in the low bits of 1024 (fp16)
// or 128 (bf16), whose steps are 1 there.  fp16 has room for them four bits further up
// as well, as 1024 + 16 (q + 8), which a sixteenth of takes back exactly; bf16 takes a
// shift for that.
template <bool kBf16>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4])
{
    auto pick = [](uint32_t v, uint32_t mask, uint32_t magic) {        // (v & mask) ^ magic
        uint32_t x;
        asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(x) : "r"(v), "r"(mask), "r"(magic));
        return x;
    };
    if constexpr (kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(pick(w >> (4 * i), 0x000F000Fu, 0x43084308u)), "r"(0x43084308u));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = w >> (8 * i);
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * i]) : "r"(pick(v, 0x000F000Fu, 0x64086408u)), "r"(0x64086408u));
            asm("fma.rn.f16x2 %0, %1, %2, %3;"
                : "=r"(h[2 * i + 1])
                : "r"(pick(v, 0x00F000F0u, 0x64806480u)), "r"(0x2C002C00u), "r"(0xD480D480u));     // / 16 - 72
        }
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

// The first of a sum's.
template <bool kBf16>
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kDepth = 4;                        // blocks of a warp's ring
__host__ __device__ constexpr int ring_floats(int tiles_m) { return kDepth * tiles_m * 2 * 32 * 4; }

__device__ __forceinline__ uint4 ld_shared(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

template <bool kBf16, int kTilesM, int kTilesN, bool kWhole, bool kAligned>
__global__ void __launch_bounds__(kThreads) product_kernel(const __grid_constant__ ProductParams p)
{
    extern __shared__ float parts[];
    constexpr int kRows = 16 * kTilesM, kTokens = 8 * kTilesN, kLd = kRows + 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int32_t tile = static_cast<int32_t>(blockIdx.x) / p.token_tiles;
    const int32_t n0 = (static_cast<int32_t>(blockIdx.x) - tile * p.token_tiles) * kTokens;
    const int32_t m0 = tile * kRows;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int32_t blocks = (p.K + kBlock - 1) / kBlock, row_bytes = (p.K + 1) / 2;
    // Blocks that are read without a look at their ends: all of one is there, and where
    // words are cut, so are the bytes that the last one takes along (the next block's,
    // or the next row's).
    const int32_t plain = kAligned ? p.K / kBlock : p.words ? max(blocks - (m0 + kRows >= p.M ? 2 : 1), 0) : 0;
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

    float acc[kTilesM][kTilesN][4] = {};

    // What a block's multiplication needs beside its codes: the scales, and the tokens where
    // there are few enough to be held.
    constexpr bool kAhead = kTilesN <= 2;
    struct Beside {
        uint16_t scale[kTilesM][2];
        uint4 tokens[kAhead ? 4 : 1][kTilesN];
    };
    auto load = [&](Beside &s, int32_t b, bool whole, auto token) {
        const int32_t grp = kWhole ? b >> (p.group_shift - 7) : (b * kBlock + 32 * t) >> p.group_shift;
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) s.scale[i][h] = whole || grp < p.groups ? __ldg(s_row[i][h] + grp) : uint16_t(0);
        if constexpr (kAhead)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < kTilesN; ++i) s.tokens[j][i] = token(j, i);
    };
    // The multiplication.  token(j, i): the tokens' terms of word j, tile i; codes(v): the
    // block's codes, as soon as they are there.
    auto compute = [&](const Beside &s, auto token, auto codes) {
        uint4 code[kTilesM][2];
        codes(code);
        if constexpr (!kWhole) {
#pragma unroll
            for (int i = 0; i < kTilesM; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) exchange(code[i][h], t);
        }
        float part[kTilesM][kTilesN][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t x[kTilesN][4];              // the tokens' eight terms of this word
#pragma unroll
            for (int i = 0; i < kTilesN; ++i) {
                const uint4 v = kAhead ? s.tokens[kAhead ? j : 0][i] : token(j, i);
                x[i][0] = __byte_perm(v.x, v.z, 0x5410);
                x[i][1] = __byte_perm(v.x, v.z, 0x7632);
                x[i][2] = __byte_perm(v.y, v.w, 0x5410);
                x[i][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < kTilesM; ++i) {
                const uint4 lo = code[i][0], hi = code[i][1];
                uint32_t u[4], v[4];
                widen<kBf16>(j == 0 ? lo.x : j == 1 ? lo.y : j == 2 ? lo.z : lo.w, u);
                widen<kBf16>(j == 0 ? hi.x : j == 1 ? hi.y : j == 2 ? hi.z : hi.w, v);
#pragma unroll
                for (int n = 0; n < kTilesN; ++n) {
                    if (!kWhole || j == 0)
                        mma_first<kBf16>(part[i][n], u[0], v[0], u[1], v[1], x[n][0], x[n][1]);
                    else
                        mma<kBf16>(part[i][n], u[0], v[0], u[1], v[1], x[n][0], x[n][1]);
                    mma<kBf16>(part[i][n], u[2], v[2], u[3], v[3], x[n][2], x[n][3]);
                }
                if (!kWhole || j == 3) {
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

    // The blocks warp, warp + kWarps, ...: the plain ones kDepth at a time, so that all
    // addresses are a pointer and a constant.
    constexpr int kCodeStep = kWarps * kBlock / 2, kTokenStep = kWarps * kBlock;
    int32_t b = warp;
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) a_row[i][h] += warp * (kBlock / 2);
#pragma unroll
    for (int i = 0; i < kTilesN; ++i) b_row[i] += warp * kBlock;
    // Aligned: each lane copies its own pieces kDepth - 1 blocks ahead into a ring of its
    // own in shared memory: many bytes in flight, few registers, nothing to synchronise.
    const uint32_t ring = ptx::smem_addr(parts) + (warp * kDepth * kTilesM * 2 * 32 + lane) * 16;
    auto copy = [&](int32_t left, int ahead, int stage) {        // the block `ahead` turns on, if there is one
        if (left > ahead * kWarps) {
#pragma unroll
            for (int i = 0; i < kTilesM; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(
                                     ring + ((stage * kTilesM + i) * 2 + h) * 512),
                                 "l"(a_row[i][h] + ahead * kCodeStep)
                                 : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (kAligned)
#pragma unroll
        for (int s = 0; s < kDepth - 1; ++s) copy(plain - b, s, s);
    auto token_at = [&](int turn) {
        return [&, turn](int j, int i) {
            const uint16_t *at = b_row[i] + turn * kTokenStep + (kWhole ? 8 : 32) * j;
            if (!held[i]) return make_uint4(0, 0, 0, 0);
            if constexpr (kAligned) return __ldg(reinterpret_cast<const uint4 *>(at));
            return load_words(reinterpret_cast<const uint8_t *>(at));
        };
    };
    Beside beside[2];                            // this turn's and the next one's
    static_assert(kDepth % 2 == 0, "which is which does not depend on the round");
    if (b < plain) load(beside[0], b, true, token_at(0));
#pragma unroll 1
    while (b < plain) {
        const int32_t left = plain - b;
#pragma unroll
        for (int s = 0; s < kDepth; ++s) {
            if (s > 0 && left <= s * kWarps) break;
            if constexpr (kAligned) copy(left, s + kDepth - 1, (s + kDepth - 1) % kDepth);
            if (left > (s + 1) * kWarps) load(beside[(s + 1) & 1], b + (s + 1) * kWarps, true, token_at(s + 1));
            compute(beside[s & 1], token_at(s), [&](uint4(&code)[kTilesM][2]) {
                if constexpr (kAligned) asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
#pragma unroll
                for (int i = 0; i < kTilesM; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        code[i][h] = kAligned ? ld_shared(ring + ((s * kTilesM + i) * 2 + h) * 512)
                                              : load_words(a_row[i][h] + s * kCodeStep);
            });
        }
        const int32_t turns = min((left + kWarps - 1) / kWarps, kDepth);
        b += turns * kWarps;
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a_row[i][h] += turns * kCodeStep;
#pragma unroll
        for (int i = 0; i < kTilesN; ++i) b_row[i] += turns * kTokenStep;
    }
#pragma unroll 1
    for (; b < blocks; b += kWarps) {            // what is left is read byte by byte
        auto token = [&](int j, int i) {
            const int32_t k = (kWhole ? 32 * t + 8 * j : 32 * j + 8 * t);
            return load_part(reinterpret_cast<const uint8_t *>(b_row[i] + (kWhole ? 8 : 32) * j),
                             held[i] ? 2 * min(p.K - b * kBlock - k, 8) : 0);
        };
        load(beside[0], b, false, token);
        compute(beside[0], token, [&](uint4(&code)[kTilesM][2]) {
#pragma unroll
            for (int i = 0; i < kTilesM; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) code[i][h] = load_part(a_row[i][h], row_bytes - b * (kBlock / 2) - 16 * t);
        });
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a_row[i][h] += kCodeStep;
#pragma unroll
        for (int i = 0; i < kTilesN; ++i) b_row[i] += kTokenStep;
    }
    if constexpr (kAligned) asm volatile("cp.async.wait_all;" ::: "memory");

    __syncthreads();                             // every ring is done with
    float *mine = parts + warp * part_floats(kTilesM, kTilesN);
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int n = 0; n < kTilesN; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) mine[(8 * n + 2 * t + (r & 1)) * kLd + 16 * i + 8 * (r >> 1) + g] = acc[i][n][r];
    __syncthreads();
    for (int32_t i = threadIdx.x; i < kRows * kTokens; i += kThreads) {
        const int32_t n = i / kRows, m = i - n * kRows;
        if (n0 + n >= p.N || m0 + m >= p.M) continue;
        float sum = 0.0f;
        for (int w = 0; w < kWarps; ++w) sum += parts[w * part_floats(kTilesM, kTilesN) + n * kLd + m];
        p.c[(n0 + n) * p.ldc + m0 + m] = from_float<kBf16>(sum);
    }
}

// ------------------------------------------------------------------ more than 8 tokens
// Tokens weigh as much as codes from here on, so warps share them: a CTA's warps are
// kWideRows (rows of 16 kTilesM each) by kWideSums (parts of the sum), and step
// through the sum together, kWideSums blocks of 128 terms a stage, codes and tokens copied
// to shared memory kDepth - 1 stages ahead.  Aligned rows only; what a row or the tokens
// lack of the last block arrives as zeros.  28672 x 4096 in groups of 64 and 16 tokens take 24.5
// us: the issue slots are half full, the units that widen codes 42 %, memory 29 %.
// (Sums in four, 64 rows to a CTA of two tiles a warp: 28.1 to 28.8 in groups of 128, against 24.1.)
constexpr int kWideRows = 4, kWideSums = 2;
static_assert(kWideRows * kWideSums == kWarps, "all of them");

template <int kTilesM, int kTilesN, bool kWhole>
struct WideCfg {
    static constexpr int kRows = 16 * kTilesM * kWideRows, kTokens = 8 * kTilesN;
    // A token's block of 16 pieces (16 bytes).  kWhole: lane t reads piece 4 t + j, which the
    // swizzle and a pitch of 9 banks of 32 bytes keep from meeting; else piece 4 j + t.
    static constexpr int kTokenPitch = kWhole ? 256 + 32 : 256 + 64;
    static constexpr int kCodeBytes = kRows * kWideSums * 64, kTokenBytes = kTokens * kWideSums * kTokenPitch;
    static constexpr int kStageBytes = kCodeBytes + kTokenBytes;
    static constexpr int kDepth = kTilesN <= 2 ? 4 : kTilesN <= 4 ? 3 : 2;
    static constexpr int kSumFloats = kTokens * (kRows + 4);
    static constexpr int kBytes = kDepth * kStageBytes > 4 * kWideSums * kSumFloats ? kDepth * kStageBytes
                                                                                      : 4 * kWideSums * kSumFloats;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int32_t bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <bool kBf16, int kTilesM, int kTilesN, bool kWhole>
__global__ void __launch_bounds__(kThreads) wide_kernel(const __grid_constant__ ProductParams p)
{
    using Cfg = WideCfg<kTilesM, kTilesN, kWhole>;
    extern __shared__ __align__(16) float wide_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int part = warp % kWideSums, row0 = warp / kWideSums * 16 * kTilesM;    // this warp's share of the sum, its rows
    const int32_t tile = static_cast<int32_t>(blockIdx.x) / p.token_tiles;
    const int32_t n0 = (static_cast<int32_t>(blockIdx.x) - tile * p.token_tiles) * Cfg::kTokens;
    const int32_t m0 = tile * Cfg::kRows;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    constexpr int kStep = kWideSums * kBlock;                // terms of a stage
    const int32_t stages = (p.K + kStep - 1) / kStep, row_bytes = (p.K + 1) / 2;
    const uint32_t smem = ptx::smem_addr(wide_smem);

    // What this thread copies of every stage: codes, 16 bytes of a row each (4 kWideSums to a
    // row), then tokens (16 kWideSums to a token).
    constexpr int kCodePieces = Cfg::kCodeBytes / 16, kTokenPieces = Cfg::kTokens * kWideSums * 16;
    constexpr int kCodeTurns = (kCodePieces + kThreads - 1) / kThreads, kTokenTurns = (kTokenPieces + kThreads - 1) / kThreads;
    const uint8_t *code_src[kCodeTurns];
    const uint16_t *token_src[kTokenTurns];
    uint32_t code_dst[kCodeTurns], token_dst[kTokenTurns];
    int32_t code_at[kCodeTurns], token_at[kTokenTurns], token_bytes[kTokenTurns];      // first byte, first term
#pragma unroll
    for (int i = 0; i < kCodeTurns; ++i) {
        const int x = threadIdx.x + i * kThreads, r = x / (4 * kWideSums), c = x % (4 * kWideSums);
        code_at[i] = 16 * c;
        code_src[i] = p.a + min(m0 + r, p.M - 1) * p.lda + 16 * c;
        // (not kWhole: the four lanes of a row read a word each of the same piece)
        const int piece = kWhole ? c & 3 : (c & 3) ^ (r >> 1 & 3);
        code_dst[i] = ((c >> 2) * Cfg::kRows + r) * 64 + 16 * piece;
    }
#pragma unroll
    for (int i = 0; i < kTokenTurns; ++i) {
        const int x = threadIdx.x + i * kThreads, n = x / (16 * kWideSums), c = x % (16 * kWideSums);
        token_at[i] = 8 * c;
        token_bytes[i] = n0 + n < p.N && n < Cfg::kTokens ? 16 : 0;      // (no such token: zeros)
        token_src[i] = p.b + min(n0 + n, p.N - 1) * p.ldb + 8 * c;
        const int piece = kWhole ? (c & 15) ^ (c >> 3 & 1) : c & 15;
        token_dst[i] = Cfg::kCodeBytes + ((c >> 4) * Cfg::kTokens + n) * Cfg::kTokenPitch + 16 * piece;
    }
    // The copies of a stage into ring slot `slot`, the pointers on to the next one's.  A whole
    // stage's are all 16 bytes; of the last one's what the rows and tokens lack arrives as zeros.
    const int32_t whole = p.K / kStep;
    auto copy = [&](int32_t stage, int slot) {
        if (stage < stages) {
            const uint32_t to = smem + slot * Cfg::kStageBytes;
            const int32_t k0 = stage * kStep;
#pragma unroll
            for (int i = 0; i < kCodeTurns; ++i) {
                if (kCodePieces % kThreads && static_cast<int>(threadIdx.x) + i * kThreads >= kCodePieces) break;
                int32_t bytes = 16;
                if (stage >= whole) bytes = max(min(row_bytes - k0 / 2 - code_at[i], 16), 0);
                copy16(to + code_dst[i], bytes ? code_src[i] : p.a, bytes);
                code_src[i] += kStep / 2;
            }
#pragma unroll
            for (int i = 0; i < kTokenTurns; ++i) {
                if (kTokenPieces % kThreads && static_cast<int>(threadIdx.x) + i * kThreads >= kTokenPieces) break;
                int32_t bytes = token_bytes[i];
                if (stage >= whole) bytes = max(min(2 * min(p.K - k0 - token_at[i], 8), bytes), 0);
                copy16(to + token_dst[i], bytes ? token_src[i] : p.b, bytes);
                token_src[i] += kStep;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const uint16_t *s_row[kTilesM][2];
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) s_row[i][h] = p.scale + min(m0 + row0 + 16 * i + 8 * h + g, p.M - 1) * p.lds;
    struct Scales {
        uint16_t v[kTilesM][2];
    };
    auto load_scales = [&](int32_t stage, Scales &s) {
        const int32_t grp = (stage * kStep + part * kBlock + (kWhole ? 0 : 32 * t)) >> p.group_shift;
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) s.v[i][h] = grp < p.groups ? __ldg(s_row[i][h] + grp) : uint16_t(0);
    };

    float acc[kTilesM][kTilesN][4] = {};
#pragma unroll
    for (int s = 0; s < Cfg::kDepth - 1; ++s) copy(s, s);
    Scales next;
    load_scales(0, next);
#pragma unroll 1
    for (int32_t first = 0; first < stages; first += Cfg::kDepth) {
#pragma unroll
    for (int slot = 0; slot < Cfg::kDepth; ++slot) {
        const int32_t stage = first + slot;
        if (slot > 0 && stage >= stages) break;
        asm volatile("cp.async.wait_group %0;" ::"n"(Cfg::kDepth - 2) : "memory");
        __syncthreads();                         // the stage is whole, and the one before it done with
        copy(stage + Cfg::kDepth - 1, (slot + Cfg::kDepth - 1) % Cfg::kDepth);
        const Scales now = next;
        load_scales(stage + 1, next);
        const uint32_t from = smem + slot * Cfg::kStageBytes;
        const uint32_t codes = from + (part * Cfg::kRows + row0 + g) * 64;
        const uint32_t tokens = from + Cfg::kCodeBytes + (part * Cfg::kTokens + g) * Cfg::kTokenPitch;
        uint4 code[kTilesM][2];
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = codes + (16 * i + 8 * h) * 64;
                if constexpr (kWhole) {
                    code[i][h] = ld_shared(at + 16 * t);
                } else {
                    const uint32_t x = g >> 1 & 3;           // (row0, 16 i and 8 h leave these bits of the row)
                    code[i][h] = make_uint4(ld_shared_u32(at + 16 * x + 4 * t), ld_shared_u32(at + 16 * (1 ^ x) + 4 * t),
                                            ld_shared_u32(at + 16 * (2 ^ x) + 4 * t), ld_shared_u32(at + 16 * (3 ^ x) + 4 * t));
                }
            }
        float sum[kTilesM][kTilesN][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t x[kTilesN][4];
#pragma unroll
            for (int n = 0; n < kTilesN; ++n) {
                const int piece = kWhole ? (4 * t + j) ^ (t >> 1) : 4 * j + t;
                const uint4 v = ld_shared(tokens + 8 * n * Cfg::kTokenPitch + 16 * piece);
                x[n][0] = __byte_perm(v.x, v.z, 0x5410);
                x[n][1] = __byte_perm(v.x, v.z, 0x7632);
                x[n][2] = __byte_perm(v.y, v.w, 0x5410);
                x[n][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < kTilesM; ++i) {
                const uint4 lo = code[i][0], hi = code[i][1];
                uint32_t u[4], v[4];
                widen<kBf16>(j == 0 ? lo.x : j == 1 ? lo.y : j == 2 ? lo.z : lo.w, u);
                widen<kBf16>(j == 0 ? hi.x : j == 1 ? hi.y : j == 2 ? hi.z : hi.w, v);
#pragma unroll
                for (int n = 0; n < kTilesN; ++n) {
                    if (!kWhole || j == 0)
                        mma_first<kBf16>(sum[i][n], u[0], v[0], u[1], v[1], x[n][0], x[n][1]);
                    else
                        mma<kBf16>(sum[i][n], u[0], v[0], u[1], v[1], x[n][0], x[n][1]);
                    mma<kBf16>(sum[i][n], u[2], v[2], u[3], v[3], x[n][2], x[n][3]);
                }
                if (!kWhole || j == 3) {
                    float s0 = to_float<kBf16>(now.v[i][0]), s1 = to_float<kBf16>(now.v[i][1]);
                    if constexpr (!kWhole) {     // lane j of the four has the scales of these 32 terms
                        s0 = __shfl_sync(0xffffffffu, s0, (lane & ~3) | j);
                        s1 = __shfl_sync(0xffffffffu, s1, (lane & ~3) | j);
                    }
#pragma unroll
                    for (int n = 0; n < kTilesN; ++n) {
                        acc[i][n][0] = fmaf(s0, sum[i][n][0], acc[i][n][0]);
                        acc[i][n][1] = fmaf(s0, sum[i][n][1], acc[i][n][1]);
                        acc[i][n][2] = fmaf(s1, sum[i][n][2], acc[i][n][2]);
                        acc[i][n][3] = fmaf(s1, sum[i][n][3], acc[i][n][3]);
                    }
                }
            }
        }
    }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    constexpr int kLd = Cfg::kRows + 4;
    float *mine = wide_smem + part * Cfg::kSumFloats + row0;
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
        for (int n = 0; n < kTilesN; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) mine[(8 * n + 2 * t + (r & 1)) * kLd + 16 * i + 8 * (r >> 1) + g] = acc[i][n][r];
    __syncthreads();
    for (int32_t i = threadIdx.x; i < Cfg::kRows * Cfg::kTokens; i += kThreads) {
        const int32_t n = i / Cfg::kRows, m = i - n * Cfg::kRows;
        if (n0 + n >= p.N || m0 + m >= p.M) continue;
        float all = 0.0f;
#pragma unroll
        for (int w = 0; w < kWideSums; ++w) all += wide_smem[w * Cfg::kSumFloats + n * kLd + m];
        p.c[(n0 + n) * p.ldc + m0 + m] = from_float<kBf16>(all);
    }
}

// ------------------------------------------------------------------ quantiser
//     scale[r, g] = amax / 7, divided in FP32 and rounded to 16 bits
//     q[r, c]     = round(x / scale) of the exact quotient, ties to even, within -8 .. 7
// A warp takes 512 terms of a row at a time (FP32: 256), 16 a lane (8), so a group's
// maximum is one of up to 32 neighbouring lanes.  8192 x 8192 in bf16 take 43.6 us (3.9
// TB/s): the conversions and roundings of 16 terms a lane between a row's load and its store.
constexpr int kQuantThreads = 256;

struct QuantParams {
    const void *x;
    int64_t ldx;
    uint8_t *q;
    int64_t ldq;
    uint16_t *scale;
    int64_t lds;
    int64_t rows;
    int32_t cols, group;
    bool bf16;                       // the scales' type
    bool vec;                        // x's rows on 16-byte boundaries, q's on 8-byte ones
};

enum In : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

// round(x / s) for s > 0 and any x: the quotient by a reciprocal, put right by the
// exact rest x - q s (q s has at most 15 bits, and the rest is below s: no bit is lost).
__device__ __forceinline__ uint32_t code(float x, float s, float inverse)
{
    float q = rintf(x * inverse);
    q = fminf(fmaxf(q, -16.0f), 16.0f);
    const float rest2 = 2.0f * fmaf(-q, s, x);
    const bool odd = static_cast<int32_t>(q) & 1;
    if (rest2 > s || (rest2 == s && odd)) q += 1.0f;
    if (rest2 < -s || (rest2 == -s && odd)) q -= 1.0f;
    return static_cast<uint32_t>(static_cast<int32_t>(fminf(fmaxf(q, -8.0f), 7.0f))) & 15u;
}

// A lane's terms at a time: 16 of a 16-bit type, 8 of FP32; a warp's are kSeg.
template <int kIn>
struct QuantCfg {
    static constexpr int kTerms = kIn == kF32 ? 8 : 16, kSeg = 32 * kTerms;
};

template <int kIn>
__global__ void __launch_bounds__(kQuantThreads) quant_kernel(const QuantParams p)
{
    constexpr int kTerms = QuantCfg<kIn>::kTerms, kSeg = QuantCfg<kIn>::kSeg, kElem = kIn == kF32 ? 4 : 2;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row_step = static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32);
    const int32_t c = static_cast<int32_t>(blockIdx.y) * kSeg + kTerms * lane;
    // A row's terms as they are read, one row ahead of the one that is worked on.
    constexpr int kWords = kTerms * kElem / 16;
    const bool whole = p.vec && c + kTerms <= p.cols;
    auto read = [&](int64_t r, uint4 (&w)[kWords]) {
        const uint8_t *src = static_cast<const uint8_t *>(p.x) + (r * p.ldx + c) * kElem;
        if (whole) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
        } else {
            union {
                uint4 v[kWords];
                uint32_t f[kTerms];
                uint16_t h[kTerms];
            } part;
#pragma unroll
            for (int i = 0; i < kWords; ++i) part.v[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kTerms; ++i)
                if (c + i < p.cols) {
                    if constexpr (kIn == kF32)
                        part.f[i] = reinterpret_cast<const uint32_t *>(src)[i];
                    else
                        part.h[i] = reinterpret_cast<const uint16_t *>(src)[i];
                }
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = part.v[i];
        }
    };
    int64_t r = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
    uint4 next[kWords];
    if (r < p.rows) read(r, next);
#pragma unroll 1
    for (; r < p.rows; r += row_step) {
        float x[kTerms];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t w[4] = {next[i].x, next[i].y, next[i].z, next[i].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (kIn == kF32) {
                    x[4 * i + q] = __uint_as_float(w[q]);
                } else {
                    x[8 * i + 2 * q] = to_float<kIn == kBF16>(static_cast<uint16_t>(w[q]));
                    x[8 * i + 2 * q + 1] = to_float<kIn == kBF16>(static_cast<uint16_t>(w[q] >> 16));
                }
            }
        }
        if (r + row_step < p.rows) read(r + row_step, next);
        float top = 0.0f;                        // (a NaN stays)
#pragma unroll
        for (int i = 0; i < kTerms; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
        for (int d = p.group / (2 * kTerms); d >= 1; d /= 2)
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(__shfl_xor_sync(0xffffffffu, top, d)));
        // (The FP32 quotient is never on a tie of 16 bits that amax / 7 is not on: off a tie t, amax - 7 t
        // is a step of amax at least, so the quotient is a seventh of one away, and it is rounded by an
        // eighth at most.  So the scale is the exact quotient's nearest, down to FP32's normal numbers.)
        const float s32 = __fdiv_rn(top, 7.0f);
        const uint16_t s16 = p.bf16 ? from_float<true>(s32) : from_float<false>(s32);
        const float s = p.bf16 ? to_float<true>(s16) : to_float<false>(s16);
        const bool finite = s < __int_as_float(0x7f800000);
        uint32_t word[kTerms / 8];
        // The usual way: a 16-bit x's quotient is a tie or at least 2^-12 off every tie
        // (x and s have 11 bits at most, and x is not below s / 2 there), so x / s rounded to
        // 2^-14 is on the tie or on its own side of it, and rounding that to a whole number is
        // rounding the exact quotient.  The sums' last bits are the code, one step 2^-14 and
        // then 1.  A scale below the type's normal numbers has less than 11 bits of precision and may
        // leave codes beyond 7: the other way.
        bool usual = s >= (p.bf16 ? 0x1p-96f : 0x1p-14f) && finite;
        if constexpr (kIn == kF32) {
            // FP32 x has 24 bits, and its quotients come as near to a tie as they like: the other way
            // for a lane with one within 2^-13 of a tie (one lane in some 500).  8192 x 8192: 121 us
            // with that way for all, 69 to 73 with this check.
            const float inverse = __fdividef(1.0f, s);
            float off = 0.0f;                    // the largest distance from a whole number
#pragma unroll
            for (int i = 0; i < kTerms; ++i) {
                const float y = x[i] * inverse, n = (y + 12582912.0f) - 12582912.0f;
                off = fmaxf(off, fabsf(y - n));
            }
            usual = usual && off < 0.5f - 0x1p-13f;
        }
        if (usual) {
            const float inverse = __fdividef(1.0f, s);
#pragma unroll
            for (int i = 0; i < kTerms / 8; ++i) {
                // 0x4B400000 is 1.5 2^23 as bits; the codes' top bits come out flipped
                uint32_t w = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float fine = fmaf(x[8 * i + q], inverse, 768.0f) - 768.0f;
                    w += __float_as_uint(fine + (12582912.0f + 8.0f)) << (4 * q);
                }
                word[i] = w ^ 0x88888888u;
            }
        } else {
            // (a scale whose reciprocal is no normal number: both times 2^96)
            const float up = s < 0x1p-96f ? 0x1p96f : 1.0f;
            const float su = s * up, inverse = __fdividef(1.0f, su);
#pragma unroll
            for (int i = 0; i < kTerms / 8; ++i) {
                word[i] = 0;
                if (finite && s > 0.0f)
#pragma unroll
                    for (int q = 0; q < 8; ++q) word[i] |= code(x[8 * i + q] * up, su, inverse) << (4 * q);
            }
        }
        if (c < p.cols) {
            uint8_t *dst = p.q + r * p.ldq + c / 2;
            if (p.vec && c + kTerms - 1 <= p.cols) {
                if constexpr (kTerms == 16)
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(word[0], word[1]);
                else
                    *reinterpret_cast<uint32_t *>(dst) = word[0];
            } else {
#pragma unroll
                for (int i = 0; i < kTerms / 2; ++i)
                    if (c + 2 * i < p.cols) dst[i] = static_cast<uint8_t>(word[i / 4] >> (8 * (i % 4)));
            }
            if (c % p.group == 0) p.scale[r * p.lds + c / p.group] = finite ? s16 : uint16_t(0x7FFF);
        }
    }
}

}  // namespace w4
