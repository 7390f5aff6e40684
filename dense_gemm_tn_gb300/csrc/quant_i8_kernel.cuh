// quant_i8_kernel.cuh -- 8-bit integer quantisation with one scale per row:
//     amax_r  = max_c |x[r, c]|
//     scale_r = amax_r / 127                       (fp32)
//     q[r, c] = round(127 x[r, c] / amax_r)        (ties to even, the quotient exact)
// A row of zeros (or of no elements) has scale 0 and codes 0.  A row that holds
// an infinity or a NaN has scale NaN and codes 0, so that a product with it is
// NaN in that row and in no other.
//
// The code is the exact quotient's, whatever the rounding of 127 / amax: the
// fp32 product x * (127 / amax) is off by less than 2^-16, so only where it lies
// within 2^-15 of a border n + 1/2 can the code be another than its rounding,
// and there 254 |x| is compared with (2 n + 1) amax exactly (border_code).
//
// Bound by memory.  x is read once, kept in registers while the row's maximum is
// found, and the codes written from there.  Measured on GB300: 16384 x 8192 bf16 73.2 us
// (5.5 TB/s, 0.81 of the copy bandwidth; what is left is the pause between a row's
// loads and its stores, which five or six CTAs an SM cover only in part), 16384 x 8191
// 99 us.  Few rows are bound by the launch: 16 x 2048 1.4 us replayed from a graph.
#pragma once

#include <cstdint>

#include "quant_e4m3_kernel.cuh"
#include "sm103_ptx.cuh"

namespace qz {

constexpr int kRowThreads = 256;
constexpr int kLongThreads = 512;
// Shared memory that a launch has without asking for more, less the row kernels'
// own (the largest team's 32 maxima): what is left to stage a row's codes in.
constexpr int kMaxStaging = 49152 - 32 * 4;

struct QuantRowsParams {
    const void *x;            // rows x cols, row stride ldx elements
    int8_t *q;                // rows x cols codes, row stride ldq
    float *scale;             // rows
    int64_t ldx, ldq, rows, cols;
    int32_t staging_bytes;    // shared memory for one row's codes
};

// The code of an fp32 x next to the border n + 1/2 of two codes, n = floor(127 |x| / a):
// 254 |x| against (2 n + 1) a.  Either side of the difference is taken as an
// fp32 product and its exact remainder (24 + 8 bits: the remainder has 8); the
// products are within an ulp or two of each other, so their difference is
// exact too, and so is the remainders'.
__device__ __forceinline__ float border_code(float x, float a, float n)
{
    const float ax = fabsf(x), m = 2.0f * n + 1.0f;
    const float p = 254.0f * ax, q = m * a;
    const float d = (p - q) + (fmaf(254.0f, ax, -p) - fmaf(m, a, -q));
    const float r = d < 0.0f || (d == 0.0f && (static_cast<int32_t>(n) & 1) == 0) ? n : n + 1.0f;
    return copysignf(r, x);
}

// How near to a border 127 x / a, as x times the rounded 127 / a, may be on the
// wrong side of it: 127 * 2^-24 < 2^-17 from the rounding of 127 / a (the
// products below are fused or allowed another 2^-17).
constexpr float kNearBorder = 0x1p-15f;

// Rows whose largest value is below 2^-100 are scaled by 2^100 (exactly, and
// also out of the subnormals) so that 127 / amax stays finite, and those above
// 2^100 by 2^-100 so that 254 x does (what that takes into the subnormals has
// code 0 either way).
__device__ __forceinline__ float row_lift(float amax)
{
    return amax < 0x1p-100f ? 0x1p100f : (amax > 0x1p100f ? 0x1p-100f : 1.0f);
}

// 1.5 * 2^23: added to a value of at most 2^22, it leaves the value rounded to
// an integer (ties to even) in the low bits.
constexpr float kRoundMagic = 12582912.0f;

// The codes of one 16-byte window of x (kVec elements), packed.
template <int kIn>
__device__ __forceinline__ uint2 window_codes(const uint4 &w, float lift, float a, float inv)
{
    constexpr int kVec = In<kIn>::kVec;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    float x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if constexpr (kIn == kInF32)
            x[i] = __uint_as_float(words[i]);
        else if constexpr (kIn == kInBF16)
            x[i] = __uint_as_float(i & 1 ? words[i >> 1] & 0xFFFF0000u : words[i >> 1] << 16);
        else
            x[i] = f16_bits_to_f32(words[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
    }
    if (kIn != kInF16 && lift != 1.0f) {                 // (a half is never that small or large)
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] *= lift;
    }
    float z[kVec], worst = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        z[i] = fmaf(x[i], inv, kRoundMagic);
        worst = fmaxf(worst, fabsf(fmaf(x[i], inv, kRoundMagic - z[i])));
    }
    if (worst > 0.5f - kNearBorder) {                    // a value next to a border: one window in thousands
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if constexpr (kIn == kInF32) {
                if (fabsf(fmaf(x[i], inv, kRoundMagic - z[i])) > 0.5f - kNearBorder)
                    z[i] = kRoundMagic + border_code(x[i], a, floorf(fabsf(x[i]) * inv));
            } else {
                // 16-bit types have ties in earnest (x = amax / 2 is one), so this is
                // for the whole window without a branch: the remainder 127 x - k amax
                // is exact (18 bits), and k is one off where it is past amax / 2, or
                // is amax / 2 with an odd k
                const float k = z[i] - kRoundMagic;
                const float rem = fmaf(-k, a, 127.0f * x[i]);
                const float half = (__float_as_uint(z[i]) & 1u) ? 0.49999997f * a : 0.5f * a;
                if (fabsf(rem) > half) z[i] += copysignf(1.0f, rem);
            }
        }
    }
    uint32_t packed[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < kVec; i += 4) {
        const uint32_t lo = __byte_perm(__float_as_uint(z[i]), __float_as_uint(z[i + 1]), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(z[i + 2]), __float_as_uint(z[i + 3]), 0x0040);
        packed[i / 4] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(packed[0], packed[1]);
}

// The 16 bytes of x from column c on, the columns outside the row 0 (and not
// read): a window that reaches past an end of the row.
template <int kIn>
__device__ __noinline__ uint4 part_window(const uint8_t *row, int32_t c, int32_t cols)
{
    constexpr int kVec = In<kIn>::kVec, kElem = elem_bytes(kIn);
    union {
        uint16_t h[8];
        uint32_t f[4];
        uint4 u;
    } part;
    part.u = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (c + j >= 0 && c + j < cols) {
            if constexpr (kElem == 4)
                part.f[j] = reinterpret_cast<const uint32_t *>(row)[c + j];
            else
                part.h[j] = reinterpret_cast<const uint16_t *>(row)[c + j];
        }
    return part.u;
}

// What a row's codes are made with, from the maximum of its bit patterns.
struct RowScale {
    float lift, a, inv;
    bool codes;               // some code is not 0
    __device__ __forceinline__ RowScale(uint32_t top, float *scale)
    {
        const bool finite = top < 0x7F800000u;
        const float amax = __uint_as_float(top);
        if (scale) *scale = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FFFFFFFu);
        lift = row_lift(amax);
        a = amax * lift;
        codes = finite && top != 0u;
        inv = codes ? __fdiv_rn(127.0f, a) : 0.0f;
    }
};

template <int kIn>
__device__ __forceinline__ uint32_t window_top(uint32_t acc)
{
    // the maxima of 16-bit types are two halfwords; both orders are the magnitudes'
    return __float_as_uint(In<kIn>::amax(acc)) & 0x7FFFFFFFu;
}

// CTAs per SM that the registers leave room for: what hides the loads' latency
// and the steps of a row is other rows.
__host__ __device__ constexpr int quant_min_blocks(int team, int windows)
{
    return windows == 2 ? 6 : team <= 256 ? (windows <= 5 ? 5 : 4) : team == 512 ? 2 : 1;
}

// kTeam threads per row (a warp, or a whole CTA), which keep the row's 16-byte
// windows in registers, kWindows each: one read of x, one write of q.  kAligned:
// rows of x start on 16-byte boundaries and rows of q where a window's codes
// can be stored at once.  Otherwise the windows are those of the aligned
// addresses that the row lies in; the first and last are read element by
// element, and the codes are staged in a row of shared memory, from where they
// are written in aligned words (with byte stores at the row's own misalignment
// 16384 x 8191 bf16 took 136 us).
template <int kIn, int kTeam, int kWindows, bool kAligned>
__global__ void __launch_bounds__(kTeam == 32 ? kRowThreads : kTeam, quant_min_blocks(kTeam, kWindows)) quant_rows_kernel(const QuantRowsParams p)
{
    constexpr int kVec = In<kIn>::kVec, kElem = elem_bytes(kIn);
    constexpr int kTeams = kTeam == 32 ? kRowThreads / 32 : 1, kTeamWarps = kTeam / 32;
    __shared__ uint32_t warp_top[kTeamWarps];
    extern __shared__ __align__(16) uint8_t staged[];        // !kAligned: staging_bytes a team
    tn::ptx::griddep_wait();
    const int t = kTeam == 32 ? threadIdx.x & 31 : threadIdx.x, team = kTeam == 32 ? threadIdx.x >> 5 : 0;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kTeams + team;
    const bool in = r < p.rows;                // (a team past the last row does nothing)
    const int32_t cols = static_cast<int32_t>(p.cols);
    const uint8_t *row = static_cast<const uint8_t *>(p.x) + (in ? r : 0) * p.ldx * kElem;
    const int32_t skew = kAligned ? 0 : static_cast<int32_t>((reinterpret_cast<uintptr_t>(row) & 15u) / kElem);
    uint4 w[kWindows];
    uint32_t top = 0;
    // whole windows first, all of their loads in flight; then the row's ends
#pragma unroll
    for (int i = 0; i < kWindows; ++i) {
        const int32_t c = (t + i * kTeam) * kVec - skew;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (in && c >= 0 && c + kVec <= cols) w[i] = __ldcs(reinterpret_cast<const uint4 *>(row + c * kElem));
    }
#pragma unroll
    for (int i = 0; i < kWindows; ++i) {
        const int32_t c = (t + i * kTeam) * kVec - skew;
        if (in && c < cols && (c < 0 || c + kVec > cols)) w[i] = part_window<kIn>(row, c, cols);
    }
#pragma unroll
    for (int i = 0; i < kWindows; ++i) top = In<kIn>::acc_chunk(top, w[i]);
    top = __reduce_max_sync(0xffffffffu, window_top<kIn>(top));
    if constexpr (kTeam > 32) {
        if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, warp_top[(threadIdx.x & 31) % kTeamWarps]);
    }
    const RowScale rs(top, in && t == 0 ? p.scale + r : nullptr);
    int8_t *q = p.q + (in ? r : 0) * p.ldq;
    uint8_t *mine = staged + team * p.staging_bytes;
#pragma unroll
    for (int i = 0; i < kWindows; ++i) {
        const int32_t c = (t + i * kTeam) * kVec - skew;
        if (!in || c >= cols) continue;
        const uint2 k = rs.codes ? window_codes<kIn>(w[i], rs.lift, rs.a, rs.inv) : make_uint2(0u, 0u);
        if (!kAligned || c + kVec <= cols) {
            // (staged: column c at byte skew + c)
            void *to = kAligned ? static_cast<void *>(q + c) : static_cast<void *>(mine + (t + i * kTeam) * kVec);
            if constexpr (kVec == 8)
                *static_cast<uint2 *>(to) = k;
            else
                *static_cast<uint32_t *>(to) = k.x;
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (c + j < cols) q[c + j] = static_cast<int8_t>((j < 4 ? k.x : k.y) >> (8 * (j & 3)));
        }
    }
    if constexpr (!kAligned) {
        if constexpr (kTeam == 32)
            __syncwarp();
        else
            __syncthreads();
        if (!in) return;
        // aligned words of q, each cut out of two staged ones
        const int32_t q_skew = static_cast<int32_t>(reinterpret_cast<uintptr_t>(q) & 3u);
        for (int32_t b = t * 4 - q_skew; b < cols; b += kTeam * 4) {
            const int32_t at = b + skew;
            if (b >= 0 && b + 4 <= cols) {
                const uint32_t *words = reinterpret_cast<const uint32_t *>(mine) + (at >> 2);
                *reinterpret_cast<uint32_t *>(q + b) = __funnelshift_r(words[0], words[1], 8u * (at & 3));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (b + j >= 0 && b + j < cols) q[b + j] = static_cast<int8_t>(mine[at + j]);
            }
        }
    }
}

// Rows of more than the largest team's windows: one CTA per row at a time, x
// read twice (the second time in part from L2).
template <int kIn>
__global__ void __launch_bounds__(kLongThreads) quant_long_rows_kernel(const QuantRowsParams p)
{
    constexpr int kVec = In<kIn>::kVec, kElem = elem_bytes(kIn);
    __shared__ uint32_t warp_top[kLongThreads / 32];
    tn::ptx::griddep_wait();
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const uint8_t *row = static_cast<const uint8_t *>(p.x) + r * p.ldx * kElem;
        const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(row) & 15u) / kElem);
        // columns are counted in 64 bits here: a row may have more than 2^31
        const int64_t windows = (p.cols + skew + kVec - 1) / kVec;
        auto window = [&](int64_t i) {
            // (a part window is read from its own start, so that 32 bits count its columns)
            const int64_t c = i * kVec - skew;
            const uint8_t *from = row + c * kElem;
            if (c >= 0 && c + kVec <= p.cols) return __ldcs(reinterpret_cast<const uint4 *>(from));
            if (c < 0) return part_window<kIn>(row, -skew, static_cast<int32_t>(p.cols < kVec ? p.cols : kVec));
            return part_window<kIn>(from, 0, static_cast<int32_t>(p.cols - c));
        };
        uint32_t acc = 0;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < windows; i += kLongThreads) acc = In<kIn>::acc_chunk(acc, window(i));
        uint32_t top = __reduce_max_sync(0xffffffffu, window_top<kIn>(acc));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, warp_top[(threadIdx.x & 31) % (kLongThreads / 32)]);
        const RowScale rs(top, threadIdx.x == 0 ? p.scale + r : nullptr);
        int8_t *q = p.q + r * p.ldq - skew;          // the code of window i's element j: q[i * kVec + j]
        const bool vec = reinterpret_cast<uintptr_t>(q) % kVec == 0;
#pragma unroll 2
        for (int64_t i = threadIdx.x; i < windows; i += kLongThreads) {
            const uint2 k = rs.codes ? window_codes<kIn>(window(i), rs.lift, rs.a, rs.inv) : make_uint2(0u, 0u);
            if (vec && i > 0 && (i + 1) * kVec <= p.cols + skew) {
                if constexpr (kVec == 8)
                    *reinterpret_cast<uint2 *>(q + i * kVec) = k;
                else
                    *reinterpret_cast<uint32_t *>(q + i * kVec) = k.x;
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (i * kVec + j >= skew && i * kVec + j < p.cols + skew)
                        q[i * kVec + j] = static_cast<int8_t>((j < 4 ? k.x : k.y) >> (8 * (j & 3)));
            }
        }
    }
}

}  // namespace qz
