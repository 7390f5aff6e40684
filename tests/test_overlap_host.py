"""Results in memory that the call still reads: refused on the CPU, before any CUDA call; layouts that share a buffer but no byte,
and the overlaps that are harmless, are not."""
import pytest
import torch

g = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

BINDINGS = [b for b in (g.lib, g.fast) if b is not None]
P = 0x100000        # stands for device pointers, never followed here
WS = 0x10000000


def gated(lib, E=2, M=16, K=8, T=40, A=P, lda=8, stride_a=256, B=2 * P, ldb=8, offsets=3 * P, H=4 * P, ldh=16, kept=5 * P, ldp=32,
          ws=None, n=0):
    return lib.gemm_tn_gated(g.GEMM_IN_F16, g.GEMM_ACT_SILU, E, M, K, T, A, lda, stride_a, B, ldb, offsets, H, ldh, kept, ldp, ws, n, None)


def gated_grad(lib, E=2, M=16, K=8, T=40, A=P, lda=8, stride_a=256, B=2 * P, ldb=8, offsets=3 * P, kept=5 * P, ldp=32, dH=4 * P, lddh=16,
               dA=6 * P, ldda=8, stride_da=256, dB=7 * P, lddb=8, ws=WS, n=1 << 20):
    return lib.gemm_tn_gated_grad(g.GEMM_IN_BF16, g.GEMM_ACT_GELU, E, M, K, T, A, lda, stride_a, B, ldb, offsets, kept, ldp, dH, lddh,
                                  dA, ldda, stride_da, dB, lddb, ws, n, None)


def loss(lib, M=100, N=40, K=8, A=P, B=2 * P, targets=3 * P, out=4 * P, lse=5 * P, ws=WS, n=1 << 20):
    return lib.gemm_tn_cross_entropy(g.GEMM_IN_F16, M, N, K, A, K, B, K, targets, out, lse, ws, n, None)


def loss_grad(lib, M=100, N=40, K=8, A=P, lda=8, B=2 * P, ldb=8, targets=3 * P, lse=4 * P, dloss=5 * P, dA=6 * P, ldda=8, dB=7 * P, lddb=8,
              ws=WS, n=1 << 20):
    return lib.gemm_tn_cross_entropy_grad(g.GEMM_IN_BF16, M, N, K, A, lda, B, ldb, targets, lse, dloss, dA, ldda, dB, lddb, ws, n, None)


def w4(lib, M=16, N=4, K=64, A=P, lda=32, scale=2 * P, B=3 * P, ldb=64, C=4 * P, ldc=16):
    return lib.gemm_w4_tn(g.GEMM_IN_F16, M, N, K, A, lda, scale, 2, 32, B, ldb, C, ldc, None)


def quant(lib, rows=4, cols=64, x=P, ldx=64, q=2 * P, ldq=32, scale=3 * P):
    return lib.gemm_quantize_w4_rows(x, g.GEMM_IN_F32, rows, cols, ldx, 32, q, ldq, g.GEMM_IN_F16, scale, 2, None)


REFUSED = [
    (gated, dict(H=P)), (gated, dict(H=2 * P)), (gated, dict(H=P + 1000)), (gated, dict(H=3 * P)), (gated, dict(H=5 * P)),
    (gated, dict(kept=4 * P + 1276)), (gated, dict(kept=2 * P + 8)), (gated, dict(kept=P + 1020)), (gated, dict(H=2 * P - 1278)),
    (gated, dict(lda=9, stride_a=288, ws=2 * P, n=1 << 19)), (gated, dict(lda=9, stride_a=288, ws=WS, n=1 << 19, H=WS + 256)),
    (gated_grad, dict(dB=2 * P)), (gated_grad, dict(dB=P)), (gated_grad, dict(dB=P + 1022, dA=None)), (gated_grad, dict(dB=3 * P)),
    (gated_grad, dict(dB=2 * P + 638)), (gated_grad, dict(dB=2 * P - 638)), (gated_grad, dict(dA=2 * P)), (gated_grad, dict(dA=P + 16)),
    (gated_grad, dict(dA=P, ldda=16, stride_da=512)), (gated_grad, dict(dA=7 * P)), (gated_grad, dict(dA=3 * P, dB=None)),
    (gated_grad, dict(dA=WS)), (gated_grad, dict(dB=WS + 256)), (gated_grad, dict(dH=WS)), (gated_grad, dict(kept=WS)), (gated_grad, dict(B=WS)),
    (gated_grad, dict(A=WS)), (gated_grad, dict(E=1, offsets=None, dB=2 * P)),
    (loss, dict(out=5 * P)), (loss, dict(out=3 * P + 300)), (loss, dict(lse=3 * P)), (loss, dict(lse=4 * P + 156)), (loss, dict(out=WS)),
    (loss, dict(lse=WS + 1000)), (loss, dict(targets=WS)), (loss, dict(A=WS)), (loss, dict(B=WS)),
    (loss_grad, dict(dB=2 * P)), (loss_grad, dict(dB=P)), (loss_grad, dict(dA=2 * P)), (loss_grad, dict(dA=P + 16)), (loss_grad, dict(dA=7 * P)),
    (loss_grad, dict(dA=3 * P)), (loss_grad, dict(dB=4 * P)), (loss_grad, dict(dA=5 * P)), (loss_grad, dict(dA=P, ldda=16)),
    (loss_grad, dict(dB=WS)), (loss_grad, dict(lse=WS)), (loss_grad, dict(dloss=WS)), (loss_grad, dict(A=WS + 512)),
    (w4, dict(C=P)), (w4, dict(C=2 * P)), (w4, dict(C=3 * P + 100)), (w4, dict(C=3 * P - 126)),
    (quant, dict(q=P)), (quant, dict(scale=P + 16)), (quant, dict(q=3 * P)), (quant, dict(q=P + 1023)),
]

TAKEN = [
    (gated, dict(H=2 * P - 1280)), (gated, dict(kept=None, H=5 * P)),
    # x and H, and A and dA, beside each other in the rows of one buffer; experts' A and dA one after the other in turn
    (gated, dict(B=2 * P, ldb=24, H=2 * P + 16, ldh=24)), (gated_grad, dict(A=P, lda=16, stride_a=512, dA=P + 16, ldda=16, stride_da=512)),
    (gated_grad, dict(A=P, stride_a=512, dA=P + 512, stride_da=512)),
    (gated_grad, dict(dB=4 * P)), (gated_grad, dict(dA=5 * P)), (gated_grad, dict(dA=P)), (gated_grad, dict(dB=2 * P, dA=None)),
    (gated_grad, dict(dA=P + 16, dB=None)), (gated_grad, dict(dA=WS + (1 << 19))),
    (loss, dict(out=P)), (loss, dict(out=5 * P - 160)), (loss_grad, dict(dA=P)), (loss_grad, dict(dB=2 * P, dA=None)),
    (loss_grad, dict(B=2 * P, ldb=16, dB=2 * P + 16, lddb=16)),
    (w4, dict(B=3 * P, ldb=80, C=3 * P + 128, ldc=80)), (quant, dict(x=P, ldx=80, q=P + 256, ldq=320)),
]


@pytest.mark.parametrize("lib", BINDINGS, ids=lambda b: getattr(b, "__name__", "ctypes"))
@pytest.mark.parametrize("call,bad", REFUSED)
def test_overlaps_are_refused(lib, call, bad):
    assert call(lib, **bad) == g.GEMM_ERR_INVALID_ARG
    assert "overlaps" in g.last_error()


@pytest.mark.parametrize("call,good", [*((c, {}) for c in (gated, gated_grad, loss, loss_grad, w4, quant)), *TAKEN])
def test_what_shares_no_byte_is_taken(call, good):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these pointers are not to reach it")
    assert call(g.lib, **good) == g.GEMM_ERR_CUDA


def test_empty_results_overlap_nothing():
    assert gated(g.lib, T=0, H=P) == g.GEMM_OK
    assert gated_grad(g.lib, K=0, dA=P, dB=2 * P) == g.GEMM_OK
    assert loss(g.lib, N=0, out=P, lse=P) == g.GEMM_OK
    assert w4(g.lib, N=0, C=P) == g.GEMM_OK
    assert quant(g.lib, rows=0, q=P) == g.GEMM_OK
