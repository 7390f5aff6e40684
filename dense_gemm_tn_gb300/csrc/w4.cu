// w4.cu -- the C ABI's products with 4-bit weights and their quantiser
// (include/tn_gemm.h).
#include "host_common.cuh"
#include "w4_kernel.cuh"

namespace {

#include "w4_host.cuh"

}  // namespace

extern "C" {

gemm_status_t gemm_w4_tn(int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *scale_a,
                         int64_t ld_scale, int64_t group, const void *B, int64_t ldb, void *C, int64_t ldc, void *stream)
{
    clear_error();
    return run_w4(type, M, N, K, A, lda, scale_a, ld_scale, group, B, ldb, C, ldc, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_quantize_w4_rows(const void *x, int x_type, int64_t rows, int64_t cols, int64_t ldx, int64_t group, void *q,
                                    int64_t ldq, int scale_type, void *scale, int64_t ld_scale, void *stream)
{
    clear_error();
    return run_quant_w4(x, x_type, rows, cols, ldx, group, q, ldq, scale_type, scale, ld_scale,
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
