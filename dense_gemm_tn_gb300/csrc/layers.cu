// layers.cu -- the C ABI's gated projections and vocabulary loss, with their
// gradients (include/tn_gemm.h).
#include "host_common.cuh"
#include "gated_few_kernel.cuh"
#include "grouped_kernel.cuh"
#include "layers_kernels.cuh"

namespace {

#include "grouped_host.cuh"
#include "sinks_host.cuh"

}  // namespace

namespace tn_host {

cudaError_t take_layers_status(int *value)
{
    const cudaError_t e = cudaMemcpyFromSymbol(value, tn::g_tn_status, sizeof(int));
    const int zero = 0;
    return e != cudaSuccess || *value == 0 ? e : cudaMemcpyToSymbol(tn::g_tn_status, &zero, sizeof(int));
}

}  // namespace tn_host

extern "C" {

int64_t gemm_gated_workspace(int grad, int dense, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                             int64_t stride_a, const void *B, int64_t ldb)
{
    return gated_workspace(grad, dense, E, M, K, T, A, lda, stride_a, B, ldb);
}

gemm_status_t gemm_tn_gated(int type, int act, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                            int64_t stride_a, const void *B, int64_t ldb, const int32_t *offsets, void *H, int64_t ldh,
                            float *P, int64_t ldp, void *workspace, int64_t workspace_bytes, void *stream)
{
    clear_error();
    return run_gated(type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, H, ldh, P, ldp, workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_tn_gated_grad(int type, int act, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                                 int64_t stride_a, const void *B, int64_t ldb, const int32_t *offsets, const float *P,
                                 int64_t ldp, const void *dH, int64_t lddh, void *dA, int64_t ldda, int64_t stride_da,
                                 void *dB, int64_t lddb, void *workspace, int64_t workspace_bytes, void *stream)
{
    clear_error();
    return run_gated_grad(type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, P, ldp, dH, lddh, dA, ldda, stride_da, dB,
                          lddb, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int64_t gemm_cross_entropy_workspace(int grad, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B,
                                     int64_t ldb)
{
    return loss_workspace(grad, M, N, K, A, lda, B, ldb);
}

gemm_status_t gemm_tn_cross_entropy(int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B,
                                    int64_t ldb, const int64_t *targets, float *loss, float *lse, void *workspace,
                                    int64_t workspace_bytes, void *stream)
{
    clear_error();
    return run_loss(type, M, N, K, A, lda, B, ldb, targets, loss, lse, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_tn_cross_entropy_grad(int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B,
                                         int64_t ldb, const int64_t *targets, const float *lse, const float *dloss, void *dA,
                                         int64_t ldda, void *dB, int64_t lddb, void *workspace, int64_t workspace_bytes,
                                         void *stream)
{
    clear_error();
    return run_loss_grad(type, M, N, K, A, lda, B, ldb, targets, lse, dloss, dA, ldda, dB, lddb, workspace, workspace_bytes,
                         static_cast<cudaStream_t>(stream));
}

}  // extern "C"
