// quant_i8_kernel.cuh -- 8-bit integer quantisation with one scale per row:
//     amax_r  = max_c |x[r, c]|
//     scale_r = amax_r / 127                       (fp32)
//     q[r, c] = round(127 x[r, c] / amax_r)        (ties to even, the quotient exact)
// A row of zeros (or of no elements) has scale 0 and codes 0.  A row that holds
// an infinity or a NaN has scale NaN and codes 0, so that a product with it is
// NaN in that row and in no other.
//
// The code is the exact quotient's, whatever the rounding of 127 / amax: the
// fp32 product x * (127 / amax) is off by less than 2^-15 (127 * 2^-22), so
// only where it lies within 2^-13 of a border n + 1/2 can the code be another
// than its rounding, and there 254 |x| is compared with (2 n + 1) amax, both
// exact in fp64 (24 + 8 bits).
#pragma once

#include <cstdint>

#include "quant_e4m3_kernel.cuh"
#include "sm103_ptx.cuh"

namespace qz {

constexpr int kRowThreads = 256;

struct QuantRowsParams {
    const void *x;            // rows x cols, row stride ldx elements
    int8_t *q;                // rows x cols codes, row stride ldq
    float *scale;             // rows
    int64_t ldx, ldq, rows, cols;
};

template <int kIn>
__device__ __forceinline__ float load_one(const void *x, int64_t i)
{
    if constexpr (kIn == kInF32)
        return static_cast<const float *>(x)[i];
    else if constexpr (kIn == kInF16)
        return f16_bits_to_f32(static_cast<const uint16_t *>(x)[i]);
    else
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(x)[i]) << 16);
}

// x, amax and inv = 127 / amax all of the row's (scaled) values, amax > 0.
__device__ __forceinline__ int32_t row_code(float x, float amax, float inv)
{
    const float y = x * inv;
    float k = rintf(y);
    if (fabsf(fabsf(y - k) - 0.5f) < 0x1p-13f) {
        const float n = floorf(fabsf(y));
        const double a = 254.0 * fabs(static_cast<double>(x)), b = (2.0 * n + 1.0) * static_cast<double>(amax);
        const float up = n + 1.0f;
        const float r = a < b ? n : (a > b ? up : (fmodf(n, 2.0f) == 0.0f ? n : up));
        k = copysignf(r, x);
    }
    return static_cast<int32_t>(k);
}

// Rows whose largest value is below 2^-100 are scaled by 2^100 (exactly, and
// also out of the subnormals) so that 127 / amax stays finite.
__device__ __forceinline__ float row_lift(float amax) { return amax < 0x1p-100f ? 0x1p100f : 1.0f; }

// One CTA per row.
template <int kIn>
__global__ void __launch_bounds__(kRowThreads) quant_rows_kernel(const QuantRowsParams p)
{
    __shared__ uint32_t warp_top[kRowThreads / 32];
    tn::ptx::griddep_wait();
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const int64_t base = r * p.ldx;
        uint32_t top = 0;
        for (int64_t c = threadIdx.x; c < p.cols; c += kRowThreads)
            top = max(top, __float_as_uint(load_one<kIn>(p.x, base + c)) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xffffffffu, top);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int i = 0; i < kRowThreads / 32; ++i) top = max(top, warp_top[i]);
        const bool finite = top < 0x7F800000u;
        const float amax = __uint_as_float(top);
        if (threadIdx.x == 0) p.scale[r] = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FFFFFFFu);
        const float lift = row_lift(amax), a = amax * lift;
        const float inv = finite && top != 0u ? __fdiv_rn(127.0f, a) : 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += kRowThreads)
            p.q[r * p.ldq + c] = inv != 0.0f ? static_cast<int8_t>(row_code(load_one<kIn>(p.x, base + c) * lift, a, inv)) : 0;
    }
}

}  // namespace qz
