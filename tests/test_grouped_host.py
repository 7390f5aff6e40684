"""Refusals and the workspace query of the grouped and 8-bit products and the row
quantiser, on the CPU: arguments are checked before any CUDA call."""
import pytest
import torch

g = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

BINDINGS = [b for b in (g.lib, g.fast) if b is not None]
P = 0x10000        # stands for device pointers, never followed here


def product(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, E=2, M=16, K=8, T=4, A=P, lda=8, stride_a=128, B=2 * P, ldb=8, offsets=3 * P, C=4 * P,
             ldc=16, ws=None, n=0)
    a.update(kw)
    return lib.gemm_tn_grouped(a["type"], a["E"], a["M"], a["K"], a["T"], a["A"], a["lda"], a["stride_a"], a["B"],
                               a["ldb"], a["offsets"], a["C"], a["ldc"], a["ws"], a["n"], None)


def grad_b(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, E=2, M=16, K=8, T=4, A=P, lda=8, stride_a=128, dC=2 * P, lddc=16, offsets=3 * P,
             dB=4 * P, lddb=8, ws=None, n=0)
    a.update(kw)
    return lib.gemm_tn_grouped_grad_b(a["type"], a["E"], a["M"], a["K"], a["T"], a["A"], a["lda"], a["stride_a"],
                                      a["dC"], a["lddc"], a["offsets"], a["dB"], a["lddb"], a["ws"], a["n"], None)


def grad_a(lib, **kw):
    a = dict(type=g.GEMM_IN_BF16, E=2, M=16, K=8, T=4, dC=P, lddc=16, B=2 * P, ldb=8, offsets=3 * P, dA=4 * P, ldda=8,
             stride_da=128, ws=5 * P, n=4096)
    a.update(kw)
    return lib.gemm_tn_grouped_grad_a(a["type"], a["E"], a["M"], a["K"], a["T"], a["dC"], a["lddc"], a["B"], a["ldb"],
                                      a["offsets"], a["dA"], a["ldda"], a["stride_da"], a["ws"], a["n"], None)


def i8(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, M=16, N=4, K=16, A=P, lda=16, sa=2 * P, B=3 * P, ldb=16, sb=4 * P, C=5 * P, ldc=16,
             ws=6 * P, n=1 << 20)
    a.update(kw)
    return lib.gemm_i8_tn(a["type"], a["M"], a["N"], a["K"], a["A"], a["lda"], a["sa"], a["B"], a["ldb"], a["sb"],
                          a["C"], a["ldc"], a["ws"], a["n"], None)


def i8_grouped(lib, **kw):
    a = dict(type=g.GEMM_IN_F16, E=2, M=16, K=16, T=4, A=P, lda=16, stride_a=256, sa=2 * P, B=3 * P, ldb=16, sb=4 * P,
             offsets=7 * P, C=5 * P, ldc=16, ws=6 * P, n=1 << 20)
    a.update(kw)
    return lib.gemm_i8_tn_grouped(a["type"], a["E"], a["M"], a["K"], a["T"], a["A"], a["lda"], a["stride_a"], a["sa"],
                                  a["B"], a["ldb"], a["sb"], a["offsets"], a["C"], a["ldc"], a["ws"], a["n"], None)


def quant(lib, **kw):
    a = dict(x=P, type=g.GEMM_IN_F16, rows=4, cols=8, ldx=8, q=2 * P, ldq=8, scale=3 * P)
    a.update(kw)
    return lib.gemm_quantize_i8_rows(a["x"], a["type"], a["rows"], a["cols"], a["ldx"], a["q"], a["ldq"], a["scale"], None)


INVALID = [
    (product, dict(type=g.GEMM_IN_F32)), (product, dict(type=7)), (product, dict(E=-1)), (product, dict(M=-1)),
    (product, dict(K=-1)), (product, dict(T=-1)), (product, dict(lda=7)), (product, dict(ldb=7)), (product, dict(ldc=15)),
    (product, dict(stride_a=-8)), (product, dict(A=None)), (product, dict(B=None)), (product, dict(C=None)),
    (product, dict(offsets=None)), (product, dict(offsets=P + 2)), (product, dict(A=P + 1)), (product, dict(C=P + 1)),
    (product, dict(lda=9, stride_a=144)),                                  # a copy without a workspace
    (product, dict(lda=9, stride_a=144, ws=5 * P, n=16)),                  # ... with too small a one
    (product, dict(lda=9, stride_a=144, ws=5 * P + 64, n=1 << 20)),        # ... with a misaligned one
    (grad_b, dict(lddc=15)), (grad_b, dict(lddb=7)), (grad_b, dict(dC=None)), (grad_b, dict(dB=None)),
    (grad_b, dict(offsets=None)), (grad_b, dict(dC=2 * P + 2)),
    (grad_a, dict(ws=None)), (grad_a, dict(n=256)), (grad_a, dict(stride_da=8, ldda=8)), (grad_a, dict(stride_da=-1)),
    (grad_a, dict(dA=None)), (grad_a, dict(type=g.GEMM_IN_F32)), (grad_a, dict(ldda=7)), (grad_a, dict(lddc=15)),
    (i8, dict(type=g.GEMM_IN_F32)), (i8, dict(sa=None)), (i8, dict(sb=None)), (i8, dict(sa=P + 2)), (i8, dict(lda=15)),
    (i8, dict(ldc=15)), (i8, dict(N=-1)), (i8, dict(C=5 * P + 1)), (i8, dict(lda=17, n=0)), (i8, dict(lda=17, ws=None)), (i8, dict(N=20000, n=0)),
    (i8_grouped, dict(offsets=None)), (i8_grouped, dict(sb=None)), (i8_grouped, dict(ldb=15)), (i8_grouped, dict(T=-1)),
    (quant, dict(type=9)), (quant, dict(rows=-1)), (quant, dict(cols=-1)), (quant, dict(ldx=7)), (quant, dict(ldq=7)),
    (quant, dict(x=None)), (quant, dict(q=None)), (quant, dict(scale=None)), (quant, dict(scale=P + 2)),
    (quant, dict(x=P + 1)),
]


@pytest.mark.parametrize("lib", BINDINGS, ids=lambda b: getattr(b, "__name__", "ctypes"))
@pytest.mark.parametrize("call,bad", INVALID)
def test_refused_before_any_cuda_call(lib, call, bad):
    assert call(lib, **bad) == g.GEMM_ERR_INVALID_ARG
    assert g.last_error() != ""


@pytest.mark.parametrize("call,bad", [
    (product, dict(E=1025)), (product, dict(K=1 << 31, lda=1 << 31, ldb=1 << 31)), (product, dict(stride_a=1 << 40)),
    (product, dict(T=1 << 31)), (grad_a, dict(E=1025)), (quant, dict(rows=1 << 41)),
])
def test_too_large_unsupported(call, bad):
    assert call(g.lib, **bad) == g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,none", [
    (product, dict(E=0)), (product, dict(T=0)), (product, dict(M=0, ldc=1)), (grad_b, dict(E=0)), (grad_b, dict(T=0)),
    (grad_b, dict(K=0, lda=1, lddb=1)), (grad_a, dict(E=0)), (grad_a, dict(M=0, lddc=1)), (grad_a, dict(K=0)),
    (i8, dict(M=0)), (i8, dict(N=0)), (i8_grouped, dict(E=0)), (quant, dict(rows=0)),
])
def test_empty_results_need_nothing(call, none):
    assert call(g.lib, **none) == g.GEMM_OK


def test_no_device_reports_cuda_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (product, grad_b, grad_a, i8, i8_grouped, quant):
        assert call(g.lib) == g.GEMM_ERR_CUDA


def test_workspace_query():
    ws = g.gemm_grouped_workspace
    aligned = lambda op, **kw: ws(op, 3, 64, 32, 100, P, 64, 64 * 64, 2 * P, 64)  # noqa: E731
    assert aligned(g.GEMM_GROUPED_PRODUCT) == 0 and aligned(g.GEMM_GROUPED_GRAD_B) == 0
    assert aligned(g.GEMM_GROUPED_GRAD_A) == 3 * 2 * 128              # two tensor maps per expert
    # an odd K: both operands of the product are copied, rows padded to 64 elements
    copies = (3 * 64 * 64 * 2, 100 * 64 * 2)
    rounded = [(c + 255) // 256 * 256 for c in copies]
    assert ws(g.GEMM_GROUPED_PRODUCT, 3, 64, 33, 100, P, 64, 64 * 64, 2 * P, 64) == sum(rounded)
    # K is no sum in grad_b: an odd K with aligned rows needs no copy
    assert ws(g.GEMM_GROUPED_GRAD_B, 3, 64, 33, 100, P, 64, 64 * 64, 2 * P, 64) == 0
    assert ws(g.GEMM_GROUPED_PRODUCT, 3, 64, 32, 100, P + 2, 64, 64 * 64, 2 * P, 64) == rounded[0]
    for bad in ((9, 3, 64, 32, 100), (0, -1, 64, 32, 100), (0, 1025, 64, 32, 100)):
        with pytest.raises(ValueError):
            ws(*bad, P, 64, 64 * 64, 2 * P, 64)


def test_helpers_refuse_shapes_types_and_places():
    f16 = dict(dtype=torch.float16)
    A, Bt, off = torch.zeros(2, 16, 8, **f16), torch.zeros(4, 8, **f16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.tn_grouped(A, Bt, off)
    with pytest.raises(ValueError, match="offsets"):
        g.tn_grouped(A, Bt, off.long())
    with pytest.raises(ValueError, match="offsets"):
        g.tn_grouped(A, Bt, off[:2])
    with pytest.raises(ValueError, match="A must"):
        g.tn_grouped(A.float(), Bt, off)
    with pytest.raises(ValueError, match="Bt"):
        g.tn_grouped(A, Bt.bfloat16(), off)
    with pytest.raises(ValueError, match="Bt"):
        g.tn_grouped(A, Bt[:, :4], off)
    with pytest.raises(ValueError, match="3-D"):
        g.tn_grouped(A[0], Bt, off)
    with pytest.raises(ValueError, match="unit stride"):
        g.tn_grouped(A.transpose(1, 2).contiguous().transpose(1, 2), Bt, off)
    with pytest.raises(ValueError, match="dCt"):
        g.tn_grouped_grad_b(A, Bt, off)
    with pytest.raises(ValueError, match="Bt"):
        g.tn_grouped_grad_a(torch.zeros(5, 16, **f16), Bt, off)
    for call in (lambda: g.tn_grouped([1], Bt, off), lambda: g.tn_grouped_grad_b(A, None, off),
                 lambda: g.tn_grouped_grad_a(Bt, Bt, [0, 4]), lambda: g.i8_tn(1, Bt, off, off), lambda: g.quantize_i8_rows(3)):
        with pytest.raises(ValueError):
            call()
    i8 = dict(dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        g.i8_tn(torch.zeros(16, 8, **i8), torch.zeros(4, 8, **i8), torch.zeros(16), torch.zeros(4))
    with pytest.raises(ValueError, match="scale_a"):
        g.i8_tn_grouped(torch.zeros(2, 16, 8, **i8), torch.zeros(4, 8, **i8), torch.zeros(16), torch.zeros(4), off)
    with pytest.raises(ValueError, match="2-D"):
        g.quantize_i8_rows(torch.zeros(4, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        g.quantize_i8_rows(torch.zeros(4, 4, dtype=torch.float16))


def test_rows_are_cut_into_even_tiles_that_cover_them():
    """The kernel's cut of a group's rows, restated: steps of the MMA's N side spread
    evenly over the fewest tiles; every tile has a row, none is taller than the
    largest, and together they are the group's rows."""
    for largest, step in ((512, 32), (256, 32), (64, 16)):
        for rows in list(range(1, 3000)) + [16383, 16384, 16385, 10 ** 6 + 1]:
            tiles, steps = -(-rows // largest), -(-rows // step)
            each, more = divmod(steps, tiles)
            heights = [(each + (r < more)) * step for r in range(tiles)]
            starts = [(r * each + min(r, more)) * step for r in range(tiles)]
            assert max(heights) <= largest and starts[-1] < rows <= starts[-1] + heights[-1]
            assert all(a + h == b for a, h, b in zip(starts, heights, starts[1:]))


@pytest.mark.parametrize("lib", BINDINGS, ids=lambda b: getattr(b, "__name__", "ctypes"))
@pytest.mark.parametrize("E,M,K,ldda,stride,fits", [
    (2, 16, 8, 8, 128, True), (2, 16, 8, 8, 127, False), (3, 16, 8, 24, 8, True), (3, 16, 8, 23, 8, False),
    (2, 16, 8, 8, 0, False), (2, 16, 8, 4096, 0, False), (2, 16, 8, 4096, 4, False), (2, 16, 8, 4096, 7, False),
    (2, 1, 8, 8, 8, True), (2, 1, 8, 8, 7, False), (2, 1, 8, 8, 0, False), (2, 1, 8, 4096, 0, False),
    (1, 16, 8, 8, 0, True)])
def test_weight_gradients_that_overlap_are_refused(lib, E, M, K, ldda, stride, fits):
    """Two experts' dA may alternate row by row, but no element may belong to both."""
    at = {(e * stride + m * ldda + k) for e in range(E) for m in range(M) for k in range(K)}
    assert (len(at) == E * M * K) == fits
    if fits and torch.cuda.is_available():
        return                                     # (no pointer here may reach a kernel)
    status = grad_a(lib, E=E, M=M, K=K, lddc=max(M, 1), ldda=ldda, stride_da=stride, ws=5 * P, n=1 << 20)
    if fits:
        assert status == g.GEMM_ERR_CUDA           # (past the checks: there is no device)
    else:
        assert status == g.GEMM_ERR_INVALID_ARG and "overlap" in g.last_error()


BIG = 2 ** 31 - 256


@pytest.mark.parametrize("lib", BINDINGS, ids=lambda b: getattr(b, "__name__", "ctypes"))
@pytest.mark.parametrize("op,E,M,K,T,ldx,stride,ldy", [
    (0, 2, 16, 8, 4, 7, 128, 8), (0, 2, 16, 8, 4, 8, 128, 7), (0, 2, 16, 8, 4, 1, 128, 8), (0, 2, 16, 0, 4, 0, 0, 1),
    (1, 2, 16, 8, 4, 7, 128, 16), (1, 2, 16, 8, 4, 8, 128, 15), (2, 2, 16, 8, 4, 15, 0, 8), (2, 2, 16, 8, 4, 16, 0, 7),
    (3, 1, 16, 16, 4, 15, 0, 16), (3, 1, 16, 16, 4, 16, 0, 15), (3, 1, 16, 16, 4, 16, 0, 0),
    (0, 1024, BIG, BIG - 1, 4, BIG, 0, BIG), (0, 1024, BIG, BIG, 4, BIG, 8, BIG), (2, 1, BIG, 8, BIG, BIG + 8, 0, 8)])
def test_workspace_of_a_call_that_is_refused(lib, op, E, M, K, T, ldx, stride, ldy):
    """Leading dimensions below the rows they hold, and copies of more than 2^63 bytes."""
    assert lib.gemm_grouped_workspace(op, E, M, K, T, P, ldx, stride, 2 * P, ldy) == -1


def test_copies_past_63_bits_are_refused():
    big = dict(E=1024, M=BIG, K=BIG - 1, lda=BIG, ldb=BIG, ldc=BIG, stride_a=0, ws=5 * P, n=2 ** 62)
    assert product(g.lib, **big) == g.GEMM_ERR_UNSUPPORTED and "copies" in g.last_error()
    assert g.gemm_grouped_workspace(0, 1, 1 << 20, BIG - 1, 4, P, BIG, 0, 2 * P, BIG) > 2 ** 51
