"""Refusals and the workspace queries of the gated projections, the vocabulary's loss and the
4-bit products, on the CPU: arguments are checked before any CUDA call.  And the 64-bit
forms that the GPU tests compare with, against differences."""
import pytest
import torch

from tests.sink_helpers import act64, gated64, gated_grad64, loss64, loss_grad64

g = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

BINDINGS = [b for b in (g.lib, g.fast) if b is not None]
P = 0x10000        # stands for device pointers, never followed here
BIG = 1 << 40


def gated(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, act=g.GEMM_ACT_SILU, E=2, M=16, K=8, T=4, A=P, lda=8, stride_a=256, B=2 * P, ldb=8, offsets=3 * P,
             H=4 * P, ldh=16, P=5 * P, ldp=32, ws=None, n=0)
    a.update(kw)
    return lib.gemm_tn_gated(*(a[k] for k in ("type", "act", "E", "M", "K", "T", "A", "lda", "stride_a", "B", "ldb", "offsets", "H",
                                              "ldh", "P", "ldp", "ws", "n")), None)


def gated_grad(lib, **kw):
    a = dict(type=g.GEMM_IN_BF16, act=g.GEMM_ACT_GELU, E=2, M=16, K=8, T=4, A=P, lda=8, stride_a=256, B=2 * P, ldb=8, offsets=3 * P,
             P=5 * P, ldp=32, dH=4 * P, lddh=16, dA=6 * P, ldda=8, stride_da=256, dB=7 * P, lddb=8, ws=8 * P, n=1 << 20)
    a.update(kw)
    return lib.gemm_tn_gated_grad(*(a[k] for k in ("type", "act", "E", "M", "K", "T", "A", "lda", "stride_a", "B", "ldb", "offsets",
                                                   "P", "ldp", "dH", "lddh", "dA", "ldda", "stride_da", "dB", "lddb", "ws", "n")), None)


def loss(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, M=100, N=4, K=8, A=P, lda=8, B=2 * P, ldb=8, targets=3 * P, loss=4 * P, lse=5 * P, ws=6 * P, n=1 << 20)
    a.update(kw)
    return lib.gemm_tn_cross_entropy(*(a[k] for k in ("type", "M", "N", "K", "A", "lda", "B", "ldb", "targets", "loss", "lse", "ws",
                                                      "n")), None)


def loss_grad(lib, **kw):
    a = dict(type=g.GEMM_IN_BF16, M=100, N=4, K=8, A=P, lda=8, B=2 * P, ldb=8, targets=3 * P, lse=4 * P, dloss=5 * P, dA=6 * P, ldda=8,
             dB=7 * P, lddb=8, ws=8 * P, n=1 << 20)
    a.update(kw)
    return lib.gemm_tn_cross_entropy_grad(*(a[k] for k in ("type", "M", "N", "K", "A", "lda", "B", "ldb", "targets", "lse", "dloss",
                                                           "dA", "ldda", "dB", "lddb", "ws", "n")), None)


def w4(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, M=16, N=4, K=70, A=P, lda=35, scale=2 * P, lds=3, group=32, B=3 * P, ldb=70, C=4 * P, ldc=16)
    a.update(kw)
    return lib.gemm_w4_tn(*(a[k] for k in ("type", "M", "N", "K", "A", "lda", "scale", "lds", "group", "B", "ldb", "C", "ldc")), None)


def quant(lib, **kw):
    a = dict(x=P, type=g.GEMM_IN_F32, rows=4, cols=70, ldx=70, group=32, q=2 * P, ldq=35, stype=g.GEMM_IN_F16, scale=3 * P, lds=3)
    a.update(kw)
    return lib.gemm_quantize_w4_rows(*(a[k] for k in ("x", "type", "rows", "cols", "ldx", "group", "q", "ldq", "stype", "scale",
                                                      "lds")), None)


INVALID = [
    *((c, bad) for c in (gated, gated_grad) for bad in (
        dict(type=g.GEMM_IN_F32), dict(type=-1), dict(act=3), dict(act=-1), dict(E=-1), dict(M=-1), dict(K=-1), dict(T=-1), dict(lda=7),
        dict(ldb=7), dict(stride_a=-8), dict(offsets=None), dict(offsets=P + 2), dict(A=None), dict(B=None), dict(A=P + 1),
        dict(B=2 * P + 1), dict(ldp=31), dict(P=5 * P + 2))),
    (gated, dict(H=None)), (gated, dict(H=4 * P + 1)), (gated, dict(ldh=15)), (gated, dict(lda=9, stride_a=288)),
    (gated, dict(K=9, lda=16, ldb=16, stride_a=512)), (gated, dict(lda=9, stride_a=288, ws=5 * P, n=16)),
    (gated, dict(lda=9, stride_a=288, ws=5 * P + 64, n=1 << 20)),
    (gated_grad, dict(P=None)), (gated_grad, dict(dH=None)), (gated_grad, dict(dH=4 * P + 1)), (gated_grad, dict(lddh=15)),
    (gated_grad, dict(ldda=7)), (gated_grad, dict(lddb=7)), (gated_grad, dict(stride_da=-1)), (gated_grad, dict(stride_da=8)),
    (gated_grad, dict(dA=6 * P + 1)), (gated_grad, dict(dB=7 * P + 1)), (gated_grad, dict(ws=None)), (gated_grad, dict(n=64)),
    (gated_grad, dict(ws=8 * P + 128)),
    *((c, bad) for c in (loss, loss_grad) for bad in (
        dict(type=g.GEMM_IN_F32), dict(M=-1), dict(N=-1), dict(K=-1), dict(M=0), dict(lda=7), dict(ldb=7), dict(targets=None),
        dict(targets=3 * P + 4), dict(A=None), dict(B=None), dict(A=P + 1), dict(ws=None), dict(n=64), dict(ws=6 * P + 64))),
    (loss, dict(loss=None)), (loss, dict(lse=None)), (loss, dict(loss=4 * P + 2)), (loss, dict(lse=5 * P + 1)),
    (loss_grad, dict(lse=None)), (loss_grad, dict(dloss=None)), (loss_grad, dict(lse=4 * P + 2)), (loss_grad, dict(dloss=5 * P + 2)),
    (loss_grad, dict(ldda=7)), (loss_grad, dict(lddb=7)), (loss_grad, dict(dA=6 * P + 1)), (loss_grad, dict(dB=7 * P + 1)),
    (w4, dict(type=g.GEMM_IN_F32)), (w4, dict(M=-1)), (w4, dict(N=-1)), (w4, dict(K=-1)), (w4, dict(group=0)), (w4, dict(group=48)),
    (w4, dict(group=512)), (w4, dict(lda=34)), (w4, dict(lds=2)), (w4, dict(ldb=69)), (w4, dict(ldc=15)), (w4, dict(A=None)),
    (w4, dict(scale=None)), (w4, dict(B=None)), (w4, dict(C=None)), (w4, dict(scale=2 * P + 1)), (w4, dict(B=3 * P + 1)),
    (w4, dict(C=4 * P + 1)),
    (quant, dict(type=9)), (quant, dict(type=-1)), (quant, dict(stype=g.GEMM_IN_F32)), (quant, dict(rows=-1)), (quant, dict(cols=-1)),
    (quant, dict(group=16)), (quant, dict(ldx=69)), (quant, dict(ldq=34)), (quant, dict(lds=2)), (quant, dict(x=None)),
    (quant, dict(q=None)), (quant, dict(scale=None)), (quant, dict(x=P + 2)), (quant, dict(scale=3 * P + 1)),
]


@pytest.mark.parametrize("lib", BINDINGS, ids=lambda b: getattr(b, "__name__", "ctypes"))
@pytest.mark.parametrize("call,bad", INVALID)
def test_refused_before_any_cuda_call(lib, call, bad):
    assert call(lib, **bad) == g.GEMM_ERR_INVALID_ARG
    assert g.last_error() != ""


@pytest.mark.parametrize("call,bad", [
    (gated, dict(E=1025)), (gated, dict(M=1 << 30)), (gated, dict(T=1 << 31)), (gated, dict(stride_a=BIG)), (gated, dict(ldh=BIG)),
    (gated, dict(ldp=BIG)), (gated_grad, dict(E=1025)), (gated_grad, dict(stride_da=BIG)), (gated_grad, dict(lddh=BIG)),
    (loss, dict(M=1 << 31)), (loss, dict(N=1 << 31)), (loss_grad, dict(ldda=BIG)), (loss_grad, dict(K=1 << 31, lda=1 << 31, ldb=1 << 31, ldda=1 << 31, lddb=1 << 31)),
    (w4, dict(M=1 << 31, ldc=1 << 31)), (w4, dict(lda=BIG)), (quant, dict(rows=1 << 41)), (quant, dict(cols=1 << 25, ldx=1 << 25, ldq=1 << 25, lds=1 << 25)),
])
def test_too_large_unsupported(call, bad):
    assert call(g.lib, **bad) == g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,none", [
    (gated, dict(E=0)), (gated, dict(T=0)), (gated, dict(M=0, ldh=1)), (gated_grad, dict(E=0)), (gated_grad, dict(K=0)),
    (gated_grad, dict(dA=None, dB=None)), (gated_grad, dict(M=0, dB=None)), (gated_grad, dict(T=0, dA=None)), (loss, dict(N=0)),
    (loss, dict(N=0, M=0)), (loss_grad, dict(K=0)), (loss_grad, dict(dA=None, dB=None)), (loss_grad, dict(N=0, dA=None)),
    (w4, dict(M=0)), (w4, dict(N=0)), (quant, dict(rows=0)), (quant, dict(cols=0)),
])
def test_empty_results_need_nothing(call, none):
    assert call(g.lib, **none) == g.GEMM_OK


def test_no_device_reports_cuda_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (gated, gated_grad, loss, loss_grad, w4, quant):
        assert call(g.lib) == g.GEMM_ERR_CUDA


def up(n):
    return (n + 255) // 256 * 256


def test_workspace_queries():
    ws = g.gemm_gated_workspace
    assert ws(0, 0, 3, 64, 32, 100, P, 32, 64 * 64, 2 * P, 32) == 0
    # an odd K: 2 M rows of each expert and the tokens copied, rows padded to 64 elements
    assert ws(0, 0, 3, 64, 33, 100, P, 33, 64 * 66, 2 * P, 33) == up(3 * 128 * 64 * 2) + up(100 * 64 * 2)
    # the gradients of both products, and two tensor maps per expert
    assert ws(1, 0, 3, 50, 32, 100, P, 32, 100 * 32, 2 * P, 32) == up(100 * 128 * 2) + 3 * 2 * 128
    dense = ws(1, 1, 1, 50, 32, 100, P, 32, 0, 2 * P, 32)
    assert dense == up(100 * 128 * 2)                      # a short sum: not in parts
    assert ws(1, 1, 1, 8000, 32, 100, P, 32, 0, 2 * P, 32) > up(100 * 16000 * 2)
    for bad in (dict(E=-1), dict(dense=1), dict(lda=31), dict(M=1 << 30), dict(stride=-1)):
        a = dict(dense=0, E=2, M=16, lda=32, stride=2048)
        a.update(bad)
        with pytest.raises(ValueError):
            ws(1, a["dense"], a["E"], a["M"], 32, 10, P, a["lda"], a["stride"], P, 32)
    ws = g.gemm_cross_entropy_workspace
    assert ws(0, 1000, 300, 64, P, 64, 2 * P, 64) == up(300 * 32 * 8) + up(300 * 4)
    assert ws(1, 1000, 300, 64, P, 64, 2 * P, 64) == up(300 * 1024 * 2) + up(300 * 8) + 256
    for N in (1, 1000, 4096, 100000, 1 << 20):             # it does not grow with the vocabulary
        most = max(1 << 28, 2048 * N) + 64 * N * 512 + 16 * N + 4096
        assert ws(1, 262144, N, 512, P, 512, 2 * P, 512) <= most
    with pytest.raises(ValueError):
        ws(0, 1000, 300, 64, P, 63, 2 * P, 64)


def test_helpers_refuse_wrong_tensors():
    h = torch.zeros(8, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    off = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(8, 8, dtype=torch.uint8)
    s = torch.zeros(8, 1, dtype=torch.bfloat16)
    for call in (lambda: g.tn_gated(h, h), lambda: g.tn_gated(h.view(2, 4, 16), h, off), lambda: g.tn_cross_entropy(h, h[:4], t),
                 lambda: g.tn_cross_entropy_grad(h, h[:4], t, f, f), lambda: g.w4_tn(q, h, s, 32),
                 lambda: g.quantize_w4_rows(h, 32), lambda: g.tn_gated_grad(h, h, torch.zeros(8, 8), h[:, :4])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call, word in (
            (lambda: g.tn_gated(h[:7], h), "even number"), (lambda: g.tn_gated(h, h, act="relu"), "act must"),
            (lambda: g.tn_gated(h.float(), h), "float16"), (lambda: g.tn_gated(h, h.half()), "bfloat16"),
            (lambda: g.tn_gated(h, h[:, :8]), "columns"), (lambda: g.tn_gated(h, h, off), "3-D"),
            (lambda: g.tn_gated(h.view(2, 4, 16), h, off.long()), "int32"), (lambda: g.tn_gated(h.view(2, 4, 16), h, off[:2]), "shape"),
            (lambda: g.tn_gated(h.t(), h), "unit stride"), (lambda: g.tn_gated(3, h), "tensors"),
            (lambda: g.tn_gated_grad(h, h, torch.zeros(8, 7), h[:, :4]), "shape"), (lambda: g.tn_gated_grad(h, h, h, h[:, :4]), "float32"),
            (lambda: g.tn_gated_grad(h, h, torch.zeros(8, 8), h), "shape"),
            (lambda: g.tn_cross_entropy(h, h, t), "shape"), (lambda: g.tn_cross_entropy(h, h[:4], t.int()), "int64"),
            (lambda: g.tn_cross_entropy(h, h[:4].half(), t), "bfloat16"), (lambda: g.tn_cross_entropy(h.float(), h[:4], t), "float16"),
            (lambda: g.tn_cross_entropy(h, h[:4, :8], t), "second dimensions"), (lambda: g.tn_cross_entropy(h[:0], h[:4], t), "classes|CUDA"),
            (lambda: g.tn_cross_entropy_grad(h, h[:4], t, f.double(), f), "float32|CUDA"),
            (lambda: g.w4_tn(q, h, s, 31), "group"), (lambda: g.w4_tn(q[:, :7], h, s, 32), "bytes"), (lambda: g.w4_tn(q, h, s.half(), 32), "bfloat16"),
            (lambda: g.w4_tn(q.char(), h, s, 32), "uint8"), (lambda: g.w4_tn(q, h, s.repeat(1, 2), 32), "shape"),
            (lambda: g.quantize_w4_rows(h, 33), "group"), (lambda: g.quantize_w4_rows(h.float(), 32), "dtype"),
            (lambda: g.quantize_w4_rows(h.double(), 32), "float32"), (lambda: g.quantize_w4_rows(h[0], 32), "2-D"),
            (lambda: g.quantize_w4_rows(h, 32, dtype=torch.float32), "float16")):
        with pytest.raises(ValueError, match=word):
            call()


def differences(f, x, step=1e-6):
    """df/dx by central differences."""
    grad = torch.zeros_like(x)
    flat, out = x.reshape(-1), grad.reshape(-1)
    for i in range(flat.numel()):
        was = flat[i].item()
        flat[i] = was + step
        hi = f()
        flat[i] = was - step
        lo = f()
        flat[i] = was
        out[i] = (hi - lo) / (2 * step)
    return grad


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradients_are_the_differences(act):
    gen = torch.Generator().manual_seed(3)
    A, Bt, dH = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((2, 6, 5), (7, 5), (7, 3)))
    bounds = [0, 4, 7]

    def value():
        return float((gated64(A, Bt, bounds, act)[0] * dH).sum())
    _, P64, _ = gated64(A, Bt, bounds, act)
    dA, dB, _, _ = gated_grad64(A, Bt, P64, dH, bounds, act, torch.bfloat16)
    assert float((dA - differences(value, A)).abs().max()) < 1e-7
    assert float((dB - differences(value, Bt)).abs().max()) < 1e-7
    x = torch.linspace(-6, 6, 101, dtype=torch.float64)
    slope = (act64(x + 1e-6, act)[0] - act64(x - 1e-6, act)[0]) / 2e-6
    assert float((slope - act64(x, act)[1]).abs().max()) < 1e-8


def test_loss_gradients_are_the_differences():
    gen = torch.Generator().manual_seed(4)
    A, Bt = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((9, 5), (6, 5)))
    dloss = torch.rand(6, generator=gen, dtype=torch.float64)
    targets = torch.tensor([3, 0, -100, 8, 3, -1])

    def value():
        return float((loss64(A, Bt, targets)[0] * dloss).sum())
    lse = loss64(A, Bt, targets)[1]
    dA, dB, _, _ = loss_grad64(A, Bt, targets, dloss, torch.bfloat16, lse)
    assert float((dA - differences(value, A)).abs().max()) < 1e-7
    assert float((dB - differences(value, Bt)).abs().max()) < 1e-7
    ref = torch.nn.functional.cross_entropy(Bt @ A.t(), targets.where(targets >= 0, torch.tensor(-100)), reduction="none")
    assert float((loss64(A, Bt, targets)[0] - ref).abs().max()) < 1e-12
