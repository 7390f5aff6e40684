/*
 * tn_gemm.h -- C ABI of the GB300 (sm_103a) dense TN GEMM library
 *              (libdense_gemm_tn.so).
 *
 * The operation, for every 0 <= m < M and 0 <= n < N:
 *
 *     C[m,n] = sum_{k=0}^{K-1} A[m,k] * B[k,n]
 *
 * is the plain matrix product of hello-gpu ch.11 "GEMM-Like", section 11.1
 * (no alpha, no beta: C is overwritten), in the "TN" storage of the AMD ROCm
 * blog "FP16 GEMM optimization on AMD RDNA 3 and RDNA 4", section "What we
 * compute":
 *
 *   A  row-major M x K:     element (m,k) at A[m*lda + k],  lda >= max(1,K)
 *   B  column-major K x N:  element (k,n) at B[k + n*ldb],  ldb >= max(1,K)
 *   C  column-major M x N:  element (m,n) at C[m + n*ldc],  ldc >= max(1,M)
 *
 * so A and B are both contiguous along K.  (A PyTorch caller holds B as an
 * (N, K) row-major tensor and C as an (N, M) row-major tensor.)  Products
 * are accumulated in FP32 on the tensor cores and rounded once to the output
 * type with round-to-nearest-even.  M, N and K need not be multiples of any
 * tile size (the same section requires non-divisible shapes to work).
 *
 * Conventions shared by every entry point below:
 *   - Pointers A, B, C are DEVICE pointers (or managed memory) on the
 *     current CUDA device.  The caller owns all of them; the library keeps
 *     no reference after the call returns.
 *   - `stream` is a cudaStream_t passed as void*; NULL means the legacy
 *     default stream.  Calls are asynchronous: they return after enqueueing
 *     work; errors found inside a kernel (a bounded wait that ran out) are
 *     reported later by gemm_poll_device_status().
 *   - M == 0 or N == 0: nothing is launched, GEMM_OK.  K == 0: C is filled
 *     with +0.
 *   - C must not overlap A or B (undefined result).
 *   - Operands whose row stride (ld * element size) or base address is not
 *     a multiple of 16 bytes are first copied into a library-owned, lazily
 *     grown device workspace with a padded stride, one per (device,
 *     stream), so calls on different streams may take this path at once.
 *   - When the tiles of a launch end in a partly filled wave, each leftover
 *     tile is computed as two halves of its k range whose FP32 partial sums
 *     meet in a library-owned buffer kept per (device, stream), allocated on
 *     first need (about 0.5 MiB per leftover tile).  The sum is taken in a
 *     fixed way, so results do not depend on timing.  cudaStreamPerThread
 *     counts as one stream per host thread.  Problems with at most 64
 *     columns n and a short K run a kernel of their own whose k ranges meet
 *     in the same buffer (at most 128 KiB per 128 rows m), also in a fixed
 *     order.
 *   - CUDA graphs: once a call has run on a stream (the first call may
 *     allocate that stream's buffers and set kernel attributes), later calls
 *     with the same sizes on that stream enqueue kernel launches only and can
 *     be captured and replayed; the kernels leave their buffers ready for the
 *     next launch.
 *   - Thread safety: every entry point may be called from several host
 *     threads, also on one stream (the legacy default stream included); the
 *     per-device state is guarded internally.  A call may enqueue several
 *     kernels (a row copy, the GEMM, a reduce pass) that share the stream's
 *     buffers; the calls on one stream hold a lock of that stream from their
 *     first buffer lookup through their last launch, so two threads' calls
 *     never interleave their kernels on it.  gemm_release_workspace() waits
 *     for calls in progress on other threads.  On a thread's first call for
 *     a device, the library makes that device's primary context current on
 *     the thread (cudaSetDevice), so a thread that has made no CUDA call of
 *     its own can call it.
 */
#ifndef DENSE_GEMM_TN_H
#define DENSE_GEMM_TN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,   /* negative size, ld too small, NULL or misaligned pointer */
    GEMM_ERR_UNSUPPORTED = 2,   /* device is not sm_103, or a size beyond 2^31 - 256 */
    GEMM_ERR_CUDA = 3,          /* a CUDA runtime / driver call failed (see gemm_last_error) */
    GEMM_ERR_TIMEOUT = 4        /* a kernel's bounded wait ran out (reported by poll) */
} gemm_status_t;

/*
 * FP16 TN GEMM.  A, B: IEEE binary16 (__half); C: binary16.
 * Errors: GEMM_ERR_INVALID_ARG for M, N or K < 0, lda/ldb < max(1,K),
 * ldc < max(1,M), a NULL pointer with work to do, or a pointer not 2-byte
 * aligned; GEMM_ERR_UNSUPPORTED off sm_103; GEMM_ERR_CUDA on a failed launch.
 */
gemm_status_t gemm_f16_tn(int64_t M, int64_t N, int64_t K,
                          const void *A, int64_t lda,
                          const void *B, int64_t ldb,
                          void *C, int64_t ldc,
                          void *stream);

/*
 * FP8 TN GEMM.  A, B: OCP E4M3 ("e4m3fn") codes, one byte each; C: bfloat16.
 * scale_a and scale_b are per-tensor DEQUANTISATION factors: the FP32
 * accumulator is multiplied by (scale_a * scale_b) in FP32 and rounded once
 * to bfloat16, i.e. C[m,n] = bf16(acc[m,n] * scale_a * scale_b).  (The FP8
 * variant with per-tensor scales and bf16 output has no printed counterpart
 * on the pages; the blog above announces the FP8 port as its part 2.)
 * Errors as for gemm_f16_tn (pointers need 1-byte alignment, C 2-byte).
 */
gemm_status_t gemm_f8e4m3_tn(int64_t M, int64_t N, int64_t K,
                             const void *A, int64_t lda,
                             const void *B, int64_t ldb,
                             void *C, int64_t ldc,
                             float scale_a, float scale_b,
                             void *stream);

/*
 * FP8 TN GEMM with device-resident per-tensor scales: gemm_f8e4m3_tn with
 * scale_a and scale_b passed as DEVICE pointers to one fp32 value each.  The
 * kernel reads them when it runs, so an earlier kernel on the same stream
 * (gemm_quantize_e4m3) may produce them without a round trip to the host.
 * C[m,n] = bf16(acc[m,n] * ((*scale_a) * (*scale_b))), the product of the two
 * scales taken in FP32 -- the same arithmetic as gemm_f8e4m3_tn, so both
 * entry points give bit-identical C for the same scale values.  The caller
 * owns the scale buffers.  Errors as for gemm_f8e4m3_tn, plus
 * GEMM_ERR_INVALID_ARG for a NULL or not 4-byte aligned scale pointer.
 */
gemm_status_t gemm_f8e4m3_tn_dscale(int64_t M, int64_t N, int64_t K,
                                    const void *A, int64_t lda,
                                    const void *B, int64_t ldb,
                                    void *C, int64_t ldc,
                                    const float *scale_a, const float *scale_b,
                                    void *stream);

/*
 * Attention scores with the softmax's row statistics, fused into the GEMM's
 * epilogue: the QK^T step of hello-gpu ch.11's closing note (the next chapter
 * joins the GEMM and the softmax so that less of the intermediate goes back to
 * memory) and of the TileLang attention article (its QK^T block, M = N = 1024,
 * K = 128, with the softmax fused into the same kernel).  A holds Q (M x K,
 * row-major), B holds K (its column n = key n, i.e. an N x K row-major array).
 * With acc = the FP32 sum over k:
 *
 *     C[m,n]     = fp16(fp32(acc[m,n] * scale))           column-major, ldc, as gemm_f16_tn
 *     row_max[m] = max over n of fp32(acc[m,n] * scale)
 *     row_sum[m] = sum over n of exp(fp32(acc[m,n] * scale) - row_max[m])
 *
 * i.e. the softmax of row m of the scores is exp(s - row_max[m]) / row_sum[m]
 * (the pages do not fix the statistics; these are the two reductions that
 * normalise a softmax, from the FP32 scores before their rounding).  The sum
 * is formed in FP32 (each exp as 2^(x log2 e) with the hardware ex2, relative
 * error about 2^-22) in a fixed order, so results repeat exactly.
 * row_max and row_sum: DEVICE arrays of M floats owned by the caller.
 * scale: any finite float (typically 1/sqrt(K)).  M or N == 0: nothing is
 * written.  K == 0: C = scale * 0, row_max = 0, row_sum = N.
 * Uses a library-owned buffer per (device, stream) for the partial
 * statistics, allocated on first use.  Tiles are never split along K here.
 * Errors as for gemm_f16_tn, plus GEMM_ERR_INVALID_ARG for NULL or misaligned
 * row_max / row_sum or a non-finite scale.
 */
gemm_status_t gemm_f16_tn_softmax_stats(int64_t M, int64_t N, int64_t K,
                                        const void *A, int64_t lda,
                                        const void *B, int64_t ldb,
                                        void *C, int64_t ldc, float scale,
                                        float *row_max, float *row_sum,
                                        void *stream);

/* Element types of the quantisers' inputs, and of the grouped products. */
typedef enum {
    GEMM_IN_F32 = 0,    /* IEEE binary32 */
    GEMM_IN_F16 = 1,    /* IEEE binary16 */
    GEMM_IN_BF16 = 2    /* bfloat16 */
} gemm_quant_in_t;

/*
 * Per-tensor E4M3 quantisation of one operand, the amax taken on the device:
 *
 *     amax  = max |x[r,c]|                       over the whole tensor
 *     s_q   = 448 / amax                         fp32 (0 if amax = 0; FLT_MAX if it overflows)
 *     q[r,c] = E4M3(fp32(x[r,c] * s_q))          round to nearest even, saturating to +-448
 *     *scale = amax / 448                        fp32: the dequantisation factor
 *
 * so that gemm_f8e4m3_tn_dscale(..., scale_a, scale_b) on two quantised
 * operands approximates the GEMM of the originals.  (The pages print no FP8
 * rule; the ROCm blog above only announces an FP8 port.  This is the plain
 * per-tensor scaling to the E4M3 maximum, 448.)
 *
 * x: rows x cols, row-major, element (r,c) at x[r*ldx + c], x_type one of
 *    gemm_quant_in_t, aligned to its element size; ldx >= max(1, cols).
 *    For the GEMM's operands: A is M x K with ldx = lda, B (column-major
 *    K x N) is N x K with ldx = ldb.
 * q: rows x cols OCP E4M3 ("e4m3fn") codes, q[r*ldq + c], ldq >= max(1, cols).
 * scale: one fp32 in device memory.
 * All three are DEVICE pointers owned by the caller; q and scale must not
 * overlap x.  rows or cols == 0 writes *scale = 0 and nothing else.
 * Inputs must be finite (an Inf or NaN gives unspecified codes and scale).
 *
 * Two kernel launches per call on `stream`: the first finds each CTA's
 * maximum and leaves it in a small library-owned array kept per (device,
 * stream) and allocated on first use; the second reads them and quantises.
 * No CTA waits on another.  Calls on one stream may share the array; calls on
 * different streams use different arrays.
 * Errors: GEMM_ERR_INVALID_ARG for an unknown x_type, negative sizes, an ld
 * below its minimum, NULL pointers with work to do, a misaligned x or scale;
 * GEMM_ERR_UNSUPPORTED off sm_103 or above 2^40 elements; GEMM_ERR_CUDA on a
 * failed allocation or launch.
 */
gemm_status_t gemm_quantize_e4m3(const void *x, int x_type, int64_t rows, int64_t cols, int64_t ldx,
                                 void *q, int64_t ldq, float *scale, void *stream);

/*
 * gemm_f16_tn without any device allocation by the library.
 *
 * The paper has no counterpart to this entry point; it exists for callers
 * that cannot let a library call cudaMalloc: programs that hand out all
 * device memory from their own pool or fixed budget, and latency-critical
 * paths where the implicit device synchronisation of cudaMalloc / cudaFree
 * is not acceptable.  Arguments, layouts and results are those of
 * gemm_f16_tn; the caller still passes (and owns) A, B and C.
 *
 * Where gemm_f16_tn would copy an operand into its lazily grown workspace
 * (base, row stride or K not a multiple of 16 bytes), this call copies it
 * into a fixed 32 MiB array that is part of the library's device image
 * instead (every GPU that loads the library holds it until the process
 * exits).  If the padded copies need more than 32 MiB
 * (2 * roundup(K, 8) * (rows of each operand that needs the copy), each
 * operand rounded up to 256 bytes), the call returns GEMM_ERR_INVALID_ARG
 * and launches nothing.  Aligned operands need no copy and no scratch.
 *
 * The array is shared by every call on a device and keeps the last call's
 * contents (each call overwrites all of the part it reads).  Calls that
 * overlap on the GPU -- on different streams, without ordering -- race on it.
 * Calls on one stream do not, whatever host threads make them: each call
 * enqueues its copy and its GEMM with no other call's launches between.
 * The call never takes the paths that need the library's per-stream buffers
 * (split-K partial sums in memory); small grids with a long K add up their
 * k ranges inside a cluster of CTAs instead, which needs no buffer.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.
 */
gemm_status_t gemm_f16_tn_noalloc(int64_t M, int64_t N, int64_t K,
                                  const void *A, int64_t lda,
                                  const void *B, int64_t ldb,
                                  void *C, int64_t ldc,
                                  void *stream);

/* ---------------------------------------------------------------------------
 * Products grouped by expert.
 *
 * E experts hold one M x K matrix A_e each; T rows of B (T x K, row-major: the
 * columns of the TN product's B, one per token) are sorted by expert.  Expert
 * e's rows are those with offsets[e] <= t < offsets[e+1], offsets being E + 1
 * ascending 32-bit row numbers in DEVICE memory (read when the kernels run, so
 * an earlier kernel on the stream may write them):
 *
 *     gemm_tn_grouped         C[t,m]    = sum_k A_e[m,k] B[t,k]        (t of e)
 *     gemm_tn_grouped_grad_b  dB[t,k]   = sum_m dC[t,m] A_e[m,k]       (t of e)
 *     gemm_tn_grouped_grad_a  dA_e[m,k] = sum_{t of e} dC[t,m] B[t,k]
 *
 * A_e's element (m,k) is at A[e*stride_a + m*lda + k]; B, C and dC are T rows
 * with leading dimensions ldb, ldc and lddc (C row t is column t of the
 * column-major product, as in gemm_f16_tn).  `type` is GEMM_IN_F16 or
 * GEMM_IN_BF16, the type of every operand and of the result.  Sums are FP32
 * (their order does not depend on timing) and rounded once.  Where tiles are
 * few and the sum long, parts of it are summed on several SMs and then added up
 * in a fixed order.
 *
 * An expert may have no rows: its dA is written as zeros.  Rows before
 * offsets[0] and from offsets[E] on belong to no expert: they are not read, and
 * their rows of C and dB are left as they were.  Values of one expert's rows
 * never reach another's results, infinities and NaNs included.  Offsets that
 * descend, are negative or pass T are read as if each were at least the ones
 * before it and at most T.  K == 0 (M == 0 for grad_b) writes zeros to the
 * experts' rows.  At most 1024 experts.
 *
 * Workspace: an operand that the TMA cannot address in place (base, row stride
 * or expert stride not a multiple of 16 bytes, or a row along the sum whose
 * length is not one) is first copied into the workspace, and grad_a keeps two
 * tensor maps per expert there.  gemm_grouped_workspace returns the bytes a
 * call with the same arguments needs (often 0: NULL will do).  The caller owns
 * the workspace (256-byte aligned); it may be used again, or freed in stream
 * order, once the call's kernels have run.  These calls keep no buffer of the
 * library's: calls and captured graphs that overlap need workspaces of their
 * own and nothing else.  A workspace with tensor maps (grad_a's, and by expert that of
 * gemm_tn_gated_grad) is best followed by 64 KiB of mapped memory: on a GB300 a call
 * whose maps lay nearer to unmapped memory was seen to fail with an illegal address.
 *
 * Errors: GEMM_ERR_INVALID_ARG for an unknown type, a negative size or stride,
 * a leading dimension below its row's length, overlapping dA_e, NULL or
 * misaligned pointers with work to do, or a workspace that is too small;
 * GEMM_ERR_UNSUPPORTED off sm_103, for more than 1024 experts, sizes beyond
 * 2^31 - 256 or 2^30 result tiles; GEMM_ERR_CUDA on a failed launch.
 */
typedef enum {
    GEMM_GROUPED_PRODUCT = 0,   /* X = A,  Y = B */
    GEMM_GROUPED_GRAD_B = 1,    /* X = A,  Y = dC */
    GEMM_GROUPED_GRAD_A = 2,    /* X = dC, Y = B (stride_x is not used) */
    GEMM_GROUPED_I8 = 3         /* X = A,  Y = B; gemm_i8_tn has E = 1 */
} gemm_grouped_op_t;

/* Workspace bytes of a call, -1 for an op, size, stride or leading dimension that
 * it would refuse.  X and Y are looked at for their alignment alone. */
int64_t gemm_grouped_workspace(int op, int64_t E, int64_t M, int64_t K, int64_t T,
                               const void *X, int64_t ldx, int64_t stride_x,
                               const void *Y, int64_t ldy);

gemm_status_t gemm_tn_grouped(int type, int64_t E, int64_t M, int64_t K, int64_t T,
                              const void *A, int64_t lda, int64_t stride_a,
                              const void *B, int64_t ldb, const int32_t *offsets,
                              void *C, int64_t ldc,
                              void *workspace, int64_t workspace_bytes, void *stream);

gemm_status_t gemm_tn_grouped_grad_b(int type, int64_t E, int64_t M, int64_t K, int64_t T,
                                     const void *A, int64_t lda, int64_t stride_a,
                                     const void *dC, int64_t lddc, const int32_t *offsets,
                                     void *dB, int64_t lddb,
                                     void *workspace, int64_t workspace_bytes, void *stream);

gemm_status_t gemm_tn_grouped_grad_a(int type, int64_t E, int64_t M, int64_t K, int64_t T,
                                     const void *dC, int64_t lddc,
                                     const void *B, int64_t ldb, const int32_t *offsets,
                                     void *dA, int64_t ldda, int64_t stride_da,
                                     void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Products of 8-bit integers with a scale for each channel m and each token:
 *
 *     gemm_i8_tn          C[n,m] = out((S * scale_a[m]) * scale_b[n]),     S = sum_k A[m,k] B[n,k]
 *     gemm_i8_tn_grouped  the same for every expert's rows, scale_a being E x M
 *
 * A, B: signed 8-bit integers, all 256 values; C: N (or T) rows of M, out_type
 * GEMM_IN_F16 or GEMM_IN_BF16.  scale_a, scale_b: fp32 in device memory, 4-byte
 * aligned.  GB300's tensor cores multiply 8-bit integers far below their FP16
 * rate, so the integers are widened to FP16, which holds each of them exactly, and
 * FP32 sums of 1024 products, which are exact too, are added up as integers.  S is
 * the exact sum, rounded once to FP32, for K up to 131071; beyond, every 1024 terms
 * are first rounded to a multiple of a power of two below K / 32768.  The two
 * scalings are FP32 products, in the order above, and the last is rounded to out_type.
 * The workspace (op GEMM_GROUPED_I8) also holds
 * the tokens widened to FP16 where there are many rows per expert and tiles; an
 * operand that the TMA cannot address is copied into it as it is.  Everything
 * else (offsets, rows of no expert, errors) is as for gemm_tn_grouped.
 */
gemm_status_t gemm_i8_tn(int out_type, int64_t M, int64_t N, int64_t K,
                         const int8_t *A, int64_t lda, const float *scale_a,
                         const int8_t *B, int64_t ldb, const float *scale_b,
                         void *C, int64_t ldc,
                         void *workspace, int64_t workspace_bytes, void *stream);

gemm_status_t gemm_i8_tn_grouped(int out_type, int64_t E, int64_t M, int64_t K, int64_t T,
                                 const int8_t *A, int64_t lda, int64_t stride_a, const float *scale_a,
                                 const int8_t *B, int64_t ldb, const float *scale_b, const int32_t *offsets,
                                 void *C, int64_t ldc,
                                 void *workspace, int64_t workspace_bytes, void *stream);

/*
 * 8-bit integer quantisation with one scale per row (a token of activations, or
 * a channel of weights):
 *
 *     amax     = max_c |x[r,c]|
 *     scale[r] = amax / 127                        fp32
 *     q[r,c]   = round(127 x[r,c] / amax)          of the exact quotient, ties to even
 *
 * x, x_type, ldx as for gemm_quantize_e4m3; q: rows x cols, q[r*ldq + c]; scale:
 * `rows` floats.  A row of zeros, or cols == 0, has scale 0 (and codes 0).  A
 * row with an infinity or a NaN has scale NaN and codes 0: a product with it is
 * NaN in that row only.  rows == 0 writes nothing.  One launch, no buffer.
 * Errors as for gemm_quantize_e4m3.
 */
gemm_status_t gemm_quantize_i8_rows(const void *x, int x_type, int64_t rows, int64_t cols, int64_t ldx,
                                    int8_t *q, int64_t ldq, float *scale, void *stream);

/* ---------------------------------------------------------------------------
 * Gated projections: the first half of a gated feed-forward block, and its
 * backward pass.
 *
 * A_e holds 2 M rows of K: M gate rows, then M up rows (element (m,k) of the gate
 * at A[e*stride_a + m*lda + k], of the up rows at A[e*stride_a + (M+m)*lda + k]).
 * For every row t of expert e:
 *
 *     P[t,j] = sum_k A_e[j,k] B[t,k]                 0 <= j < 2 M
 *     H[t,m] = act(P[t,m]) * P[t,M+m]                0 <= m < M
 *
 * and, with dH the gradient of H:
 *
 *     dP[t,m]   = dH[t,m] P[t,M+m] act'(P[t,m])
 *     dP[t,M+m] = dH[t,m] act(P[t,m])
 *     dB[t,k]   = sum_j dP[t,j] A_e[j,k]             dA_e[j,k] = sum_{t of e} dP[t,j] B[t,k]
 *
 * Operands and results are of `type` (GEMM_IN_F16 or GEMM_IN_BF16); P is FP32.  Its sums
 * are the tensor cores', as all products' here, which cut what is below a running sum's last
 * bit: short by some 8e-10 of themselves a term (3.3e-6 at K = 4096).  act is within 2^-19
 * of itself for gates from -4 on, within 2^-14 further out (and 0 below 2^-126).
 * gemm_tn_gated is one kernel: P goes to memory only where the caller passes it
 * (T rows of 2 M with leading dimension ldp), to be kept for the backward pass.
 * gemm_tn_gated_grad rounds dP to `type` before the two products; in fp16 times a power of
 * two that the largest finite number of dP decides (over all experts), which the products'
 * FP32 sums take back: of numbers below 2^-18 of the largest bits are lost, and those below
 * 2^-29 are 0.  dA or dB may be NULL: that gradient is not computed.
 *
 * offsets as for gemm_tn_grouped (rows of no expert are neither read nor written,
 * an expert without rows has a dA of zeros); or NULL with E == 1: all T rows.
 *
 * Workspace: gemm_gated_workspace returns the bytes that a call needs (grad: 0 for
 * gemm_tn_gated, else 1; dense: not 0 where offsets is NULL), -1 for sizes it would
 * refuse.  The forward call needs none where the TMA reads the operands in place
 * (base, lda, ldb, stride_a and K multiples of 16 bytes); the backward call holds dP
 * there (4 M T bytes, and up to 4864 for its factor) and, without offsets, up to 16 FP32
 * sums of dB (64 K T bytes).
 * Ownership and alignment as for gemm_tn_grouped.
 *
 * H, P, dA, dB and the workspace share no byte with one another or with what the call
 * reads, except: dA and dB may lie in P and dH, which are read first; dA may be A itself; and
 * dB may lie in B where dA is NULL.  Such calls are refused.  (Of two operands both of whose
 * rows have gaps, of different pitches, the call cannot tell: it does not refuse them.)
 *
 * Errors: as for gemm_tn_grouped, and GEMM_ERR_INVALID_ARG for an unknown
 * activation, offsets NULL with E != 1, or results that overlap as above.
 */
typedef enum {
    GEMM_ACT_SILU = 0,       /* x / (1 + exp(-x)) */
    GEMM_ACT_GELU = 1,       /* x (1 + erf(x / sqrt 2)) / 2 */
    GEMM_ACT_GELU_TANH = 2   /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2 */
} gemm_act_t;

int64_t gemm_gated_workspace(int grad, int dense, int64_t E, int64_t M, int64_t K, int64_t T,
                             const void *A, int64_t lda, int64_t stride_a,
                             const void *B, int64_t ldb);

gemm_status_t gemm_tn_gated(int type, int act, int64_t E, int64_t M, int64_t K, int64_t T,
                            const void *A, int64_t lda, int64_t stride_a,
                            const void *B, int64_t ldb, const int32_t *offsets,
                            void *H, int64_t ldh, float *P, int64_t ldp,
                            void *workspace, int64_t workspace_bytes, void *stream);

gemm_status_t gemm_tn_gated_grad(int type, int act, int64_t E, int64_t M, int64_t K, int64_t T,
                                 const void *A, int64_t lda, int64_t stride_a,
                                 const void *B, int64_t ldb, const int32_t *offsets,
                                 const float *P, int64_t ldp, const void *dH, int64_t lddh,
                                 void *dA, int64_t ldda, int64_t stride_da,
                                 void *dB, int64_t lddb,
                                 void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Softmax cross entropy of a projection onto M classes (a vocabulary), and its
 * gradients, without the N x M logits ever being held:
 *
 *     Z[n,m]  = sum_k A[m,k] B[n,k]
 *     lse[n]  = log sum_m exp(Z[n,m])
 *     loss[n] = lse[n] - Z[n,targets[n]]
 *     d[n,m]  = dloss[n] (exp(Z[n,m] - lse[n]) - (m == targets[n] ? 1 : 0))
 *     dB[n,k] = sum_m d[n,m] A[m,k]                  dA[m,k] = sum_n d[n,m] B[n,k]
 *
 * A (M x K), B (N x K) and the gradients are of `type` (GEMM_IN_F16 or
 * GEMM_IN_BF16); targets are 64-bit integers, loss, lse and dloss N floats, all in
 * device memory.  A token whose target is negative is ignored: its loss is 0 and its
 * d is 0 (its lse is written; its row of B still takes part in dA as 0 * B, so it
 * must be finite).  A target of M or more has a loss of NaN, and NaN gradients.
 * Logits and statistics are FP32.
 *
 * gemm_tn_cross_entropy_grad takes the lse that the forward call left.  It computes
 * the logits again, a piece of the vocabulary at a time.  There d, as a share of the
 * largest finite |dloss|, is rounded to `type` (in fp16 a share below 2^-27 loses bits,
 * and one below 2^-38 is 0); the products' FP32 sums are scaled back before they are
 * rounded.  dB is summed over the pieces in FP32, in a fixed order.  dA or dB may be
 * NULL: that gradient is not computed.  N == 0 writes zeros to dA.
 *
 * The logits of both calls are summed alike, 1024 terms at a time, the parts in FP32, so that
 * what is left of a probability near one, exp(Z - lse) - 1, is theirs and not their sums'
 * difference; the loss does not go through the rounded lse.
 *
 * Workspace: gemm_cross_entropy_workspace returns the bytes that a call needs (grad:
 * 0 for gemm_tn_cross_entropy, else 1), -1 for sizes it would refuse: forward N M / 4
 * + 4 N, gradient about 256 MiB (2048 N beyond 131072 tokens; 2 N M where that is
 * less) + up to 64 N K, and copies of operands that the TMA cannot read in place (as for
 * gemm_tn_grouped).  Ownership and alignment as there.
 *
 * loss, lse, dA, dB and the workspace share no byte with one another, with targets or, in
 * the gradient, with lse and dloss; dA none with A (unless it is A itself) and B, dB none
 * with A, nor with B unless dA is NULL; the workspace none with A and B.  Such calls are
 * refused, as far as gemm_tn_gated's.
 *
 * Errors: GEMM_ERR_INVALID_ARG for such an overlap, an unknown type, a negative size, M == 0 with
 * N > 0, a leading dimension below its row's length, NULL or misaligned pointers
 * with work to do (targets: 8 bytes), or a workspace that is too small;
 * GEMM_ERR_UNSUPPORTED and GEMM_ERR_CUDA as for gemm_tn_grouped.
 */
int64_t gemm_cross_entropy_workspace(int grad, int64_t M, int64_t N, int64_t K,
                                     const void *A, int64_t lda, const void *B, int64_t ldb);

gemm_status_t gemm_tn_cross_entropy(int type, int64_t M, int64_t N, int64_t K,
                                    const void *A, int64_t lda, const void *B, int64_t ldb,
                                    const int64_t *targets, float *loss, float *lse,
                                    void *workspace, int64_t workspace_bytes, void *stream);

gemm_status_t gemm_tn_cross_entropy_grad(int type, int64_t M, int64_t N, int64_t K,
                                         const void *A, int64_t lda, const void *B, int64_t ldb,
                                         const int64_t *targets, const float *lse, const float *dloss,
                                         void *dA, int64_t ldda, void *dB, int64_t lddb,
                                         void *workspace, int64_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Products with 4-bit weights and a scale per group of terms, for the few tokens of
 * a decode step:
 *
 *     C[n,m] = sum_g scale_a[m,g] (sum_{k in group g} q[m,k] B[n,k])
 *
 * q: signed 4-bit integers (-8 .. 7, two's complement), row m at A + m*lda bytes, term
 * k in byte k / 2: the low four bits for even k, the high four for odd k (lda >=
 * (K + 1) / 2; the last half of an odd row is not used).  Group g holds the terms
 * g*group .. g*group + group - 1, the last one what is left; group is 32, 64, 128 or
 * 256.  scale_a[m,g] at scale_a[m*ld_scale + g], ld_scale >= ceil(K / group).  B
 * (N x K), C (N rows of M) and the scales are of `type` (GEMM_IN_F16 or GEMM_IN_BF16).
 * A group's sum is FP32 of exact products, the scale is applied to it in FP32, and the
 * result is rounded once.  Any N is accepted; the codes are read and widened once for
 * every 32 to 64 tokens, so for hundreds of them a product of widened weights is
 * faster.  One launch, no buffer.
 *
 * gemm_quantize_w4_rows makes such weights of x (rows x cols; x_type and ldx as for
 * gemm_quantize_e4m3):
 *
 *     scale[r,g] = max_{c in g} |x[r,c]| / 7       in fp32, rounded to scale_type
 *     q[r,c]     = round(x[r,c] / scale[r,g])      of the exact quotient, ties to even, within -8 .. 7
 *
 * A group of zeros, or whose scale rounds to 0, has codes 0; one with an infinity or a
 * NaN, or whose scale is beyond the type, has scale NaN and codes 0.  The unused half
 * of an odd row's last byte is 0.  rows == 0 or cols == 0 writes nothing.  One launch.
 *
 * C, q and scale share no byte with what the call reads, nor q with scale; such calls are
 * refused, as far as gemm_tn_gated's.
 *
 * Errors of both: GEMM_ERR_INVALID_ARG for such an overlap, an unknown type or group, a negative size,
 * a leading dimension below its row's length, or NULL or misaligned pointers with work
 * to do (codes need no alignment; rows on 16-byte boundaries are fastest);
 * GEMM_ERR_UNSUPPORTED off sm_103 or for sizes beyond 2^31 - 256 (the quantiser: 2^40
 * elements, 16776960 columns of FP32, twice that of 16 bits); GEMM_ERR_CUDA on a
 * failed launch.
 */
gemm_status_t gemm_w4_tn(int type, int64_t M, int64_t N, int64_t K,
                         const void *A, int64_t lda, const void *scale_a, int64_t ld_scale, int64_t group,
                         const void *B, int64_t ldb, void *C, int64_t ldc, void *stream);

gemm_status_t gemm_quantize_w4_rows(const void *x, int x_type, int64_t rows, int64_t cols, int64_t ldx, int64_t group,
                                    void *q, int64_t ldq, int scale_type, void *scale, int64_t ld_scale, void *stream);

/* Human-readable name of a status code (static storage). */
const char *gemm_status_string(gemm_status_t status);

/* Detail of the last error returned on the calling host thread (static,
 * thread-local storage; "" when none). */
const char *gemm_last_error(void);

/*
 * Synchronises `stream`, then reads and clears the current device's status
 * word.  Returns GEMM_ERR_TIMEOUT if a kernel gave up on a bounded wait since
 * the last poll (its C is then incomplete), GEMM_ERR_CUDA if the stream
 * reported an error, GEMM_OK otherwise.
 */
gemm_status_t gemm_poll_device_status(void *stream);

/* Frees the current device's workspaces, all kept per stream: the row
 * copies of unaligned operands, the split-K partial sums, the quantiser's
 * arrays and the softmax-statistics buffers, and the smaller buffers that
 * growth replaced.  It first waits for calls in progress on other host
 * threads to have enqueued their kernels, then synchronises the device
 * (cudaFree).  The next call that needs a buffer allocates it again. */
void gemm_release_workspace(void);

/*
 * Output-tile order of the persistent scheduler, exported so the host can
 * check it.  Tile `id` of a tiles_m x tiles_n grid maps to (*tile_m, *tile_n)
 * by the grouped raster of hello-gpu ch.11 section 11.3.4 (GROUP_M) and of the
 * ROCm blog's "Step 6" (blocks grouped into tall regions of `group` tile rows,
 * the last group short): consecutive ids walk down `group` rows of one tile
 * column before moving to the next column.  Returns 0, or -1 if an argument
 * is out of range (a grid of more than 2^31 - 1 tiles included).
 */
int gemm_tile_coord(int64_t tiles_m, int64_t tiles_n, int64_t group, int64_t id,
                    int64_t *tile_m, int64_t *tile_n);

/*
 * Limit, in nanoseconds, of every device-side wait of kernels launched after
 * this call on any device (default 2e9).  0 restores the default.  A wait that
 * exceeds it makes the kernel record GEMM_ERR_TIMEOUT, drain its in-flight
 * copies, free its tensor memory and return.
 */
void gemm_set_wait_limit_ns(uint64_t limit_ns);

/*
 * Test hook: while `mode` is non-zero, launched GEMM kernels make one thread
 * wait first on a barrier nothing arrives on, so its bounded wait runs out and
 * the kernel leaves through its timeout path (no fault, no hang):
 *   1  the MMA-issuing thread;
 *   2  the TMA producer of the even CTA of each pair (or of each CTA);
 *   3  the TMA producer of the odd CTA of each pair.
 * Where a grouped or 8-bit product splits its sums over clusters, 2 means the
 * first CTA of each and 3 all the others.
 * 0 turns the hook off.
 */
void gemm_debug_inject_stall(int mode);

/*
 * Test hook: 0 (default) lets the library choose the tile shape per call;
 * 1 forces one CTA per 128 x 256 tile, 2 a CTA pair per 256 x 256 tile in
 * 2-CTA clusters.  Returns 0, or -1 for other values.
 */
int gemm_debug_force_cta_group(int group);

/*
 * Test hook: whether CTA pairs compute 256 x 512 tiles (two N = 256 halves
 * sharing the n-side rows, a 512-column accumulator) instead of 256 x 256.
 * 0 (default): an estimate of the launch's length in tile times decides;
 * 1: always, wherever CTA pairs run without the softmax statistics; -1:
 * never.  Returns 0, or -1 for
 * other values.
 */
int gemm_debug_force_wide_tiles(int mode);

/*
 * Test hook: the height, in tile rows, of the scheduler's raster groups
 * (see gemm_tile_coord); 0 restores the default (8).  Even values only, so
 * that raster ids 2j and 2j + 1 stay neighbouring m tiles of one n tile.
 * Returns 0, or -1 for odd values or values outside 0 .. 64.
 */
int gemm_debug_set_raster_group(int rows);

/*
 * Test hook: the order in which whole tiles walk their k blocks.  0
 * (default): the library's choice; 1: every tile from the first k block to
 * the last; 2: tiles of odd waves (tile id / co-resident slots odd) from the
 * last to the first, so that a wave starts on the k slices that the wave
 * before it, which shares its A panels, read last.  Only the order of the
 * FP32 partial sums changes (results on integer inputs are identical).
 * Returns 0, or -1 for other values.
 */
int gemm_debug_set_k_order(int mode);

/*
 * Test hook: how a grid of at most half the co-resident slots with a long K
 * (at least 32 k blocks) is cut into k ranges.  0 (default): the library's
 * choice; 1: always the split-reduce (FP32 partials in a per-stream buffer,
 * summed by a second kernel); 2: wherever the tiles are single-CTA tiles,
 * a cluster of 2 to 4 CTAs per tile that add their partials through
 * distributed shared memory (no buffer, no second kernel).  Returns 0, or
 * -1 for other values.
 */
int gemm_debug_set_long_k_mode(int mode);

/*
 * Test hook: the configuration of launches whose units are all m-part units
 * of single CTAs (grids of at most half the co-resident slots' tiles with a
 * short K, each tile cut into four 64-row or two 128-row ranges of m).  The
 * lean configuration has a ring sized for such a unit (three stages of 24 KiB
 * for quarters, two of 32 KiB for halves), 128 or 256 TMEM columns, and runs
 * two CTAs per SM; the full one has four stages of 48 KiB, 512 columns and
 * one CTA per SM.  0 (default): the library's choice (lean for launches of
 * more units than half the co-resident slots with at most 8 k blocks, 4 for
 * halves); 1: always the full one; 2: lean wherever the units are quarters
 * or halves.  The arithmetic, and so every result, is the same.  Returns 0,
 * or -1 for other values.
 */
int gemm_debug_set_lean_mode(int mode);

/*
 * Test hook: problems with N <= 64 (no softmax statistics) may run a kernel
 * with the operands on the other sides of the MMA (128 rows m of A by the N
 * columns n), whose k ranges meet in a small per-stream workspace.  0
 * (default): the library's choice (where K holds at most 64 blocks of 128
 * bytes); 1: never; 2: always where N <= 64.
 * Returns 0, or -1 for other values.
 */
int gemm_debug_set_skinny_mode(int mode);

/*
 * Measurement hook: while `counters` (a DEVICE pointer to 3 zeroed unsigned
 * 64-bit words) is set, every launch of the general GEMM kernel (not the
 * kernel for at most 64 columns) afterwards adds, from the first thread of
 * its first CTA, the SM cycles (%clock64) and nanoseconds
 * (%globaltimer) from its start to its end to counters[0] and counters[1],
 * and 1 to counters[2] (three atomic adds per launch, nothing else).
 * counters[0] / counters[1] is then the average SM clock, in GHz, that those
 * launches ran at.  NULL turns it off (the default).  The caller owns the
 * buffer and keeps it alive while launches that use it may run.
 */
void gemm_debug_set_clock_probe(unsigned long long *counters);

/* Description of the last GEMM kernel launch on the calling host thread
 * (tile shape, grid, co-resident cluster slots), for logs and tests
 * (thread-local storage; "" before the first launch). */
const char *gemm_debug_last_launch(void);

/* Tile configuration and build string, e.g. for logs (static storage). */
const char *gemm_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_TN_H */
