"""Products with 4-bit weights and group scales, and their quantiser, on the GPU against 64-bit forms."""
import pytest
import torch

from tests.grouped_helpers import HALF_STEP, normals, padded
from tests.sink_helpers import assert_within, sum_error

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

DTYPES = [torch.float16, torch.bfloat16]
GROUPS = [32, 64, 128, 256]


def unpack(q, cols):
    q = q.contiguous().view(torch.int8)
    return torch.stack(((q << 4) >> 4, q >> 4), -1).flatten(1)[:, :cols]


def operands(M, N, K, group, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = torch.randint(0, 256, (M, (K + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = ((0.5 + torch.rand(M, -(-K // group), generator=g, device="cuda")) / 16).to(dtype)
    return A, scale, normals(N, K, seed=seed + 1, dtype=dtype)


def check(A, scale, Bt, group, C=None, stream=None):
    N, K = Bt.shape
    dtype = Bt.dtype
    C = tn.w4_tn(A, Bt, scale, group, C=C, stream=stream)
    tn.gemm_poll_device_status()
    W = unpack(A, K).double() * scale.double()[:, torch.arange(K, device="cuda") // group] if K else torch.zeros(A.shape[0], 0, device="cuda").double()
    ref = Bt.double() @ W.t()
    size = Bt.double().abs() @ W.abs().t()
    # a group's sum as sum_error says; then a product and an addition per group and at most 16 warps' sums, each off by
    # half a step of at most `size`
    bound = HALF_STEP[dtype] * ref.abs() * 1.01 + sum_error(size, min(group, 128)) + (2 * -(-K // min(group, 128)) + 16) * 2.0 ** -24 * size + torch.finfo(dtype).tiny
    assert_within(C, ref, bound, "C")
    return C


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 1, 2), (3, 2, 31), (16, 1, 128), (17, 3, 129), (64, 8, 256), (100, 9, 300), (33, 16, 1000),
                                   (1000, 17, 520), (257, 64, 264), (20, 70, 2048), (70, 5, 4099)])
def test_product(M, N, K, group, dtype):
    check(*operands(M, N, K, group, dtype), group)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,group", [(12288, 1, 512, 128), (10007, 7, 257, 32), (9999, 16, 384, 64), (20000, 33, 160, 128), (9729, 64, 129, 256)])
def test_many_rows(M, N, K, group, dtype):
    check(*operands(M, N, K, group, dtype), group)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("M,N,K", [(1, 9, 1), (65, 16, 31), (130, 17, 100), (64, 33, 257), (200, 64, 300), (7, 70, 1000), (300, 130, 511), (128, 12, 2047)])
def test_aligned_rows_of_odd_lengths(M, N, K, group, dtype):
    """Rows on 16-byte boundaries whose ends lie anywhere, what follows them not read: NaN and other codes there."""
    A, scale, Bt = operands(M, N, K, group, dtype)
    plain = check(A, scale, Bt, group)
    A2, B2 = padded(A, -(-A.shape[1] // 16) * 16 + 16, 0x77), padded(Bt, -(-K // 8) * 8 + 8, float("nan"))
    got = check(A2, scale, B2, group)
    assert float((got.double() - plain.double()).abs().max()) <= 2 * HALF_STEP[dtype] * float(plain.abs().max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lda,lds,ldb,ldc", [(144, 5, 264, 100), (131, 3, 257, 77), (130, 9, 300, 78), (132, 4, 258, 80)])
@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
def test_strides_and_bases(lda, lds, ldb, ldc, shift, dtype):
    M, N, K, group = 77, 11, 256, 128
    A, scale, Bt = operands(M, N, K, group, dtype)
    plain = check(A, scale, Bt, group)

    def at(t, ld, by):                             # t's values with row stride ld, `by` elements off the buffer's start
        buf = torch.full((t.shape[0] * ld + by,), 99 if t.dtype == torch.uint8 else float("nan"), dtype=t.dtype, device="cuda")
        view = buf[by:].as_strided(t.shape, (ld, 1))
        view.copy_(t)
        return view
    C = padded(torch.zeros(N, M, device="cuda", dtype=dtype), ldc, 5.0)
    got = tn.w4_tn(at(A, lda, shift), at(Bt, ldb, shift), at(scale, lds, shift), group, C=C)
    # (aligned rows take another kernel for 11 tokens: its sums are cut elsewhere)
    exact = Bt.double() @ (unpack(A, K).double() * scale.double()[:, torch.arange(K, device="cuda") // group]).t()
    size = Bt.double().abs() @ (unpack(A, K).double() * scale.double()[:, torch.arange(K, device="cuda") // group]).abs().t()
    assert_within(got, exact, HALF_STEP[dtype] * exact.abs() * 1.01 + sum_error(size, 128) + 20 * 2.0 ** -24 * size + torch.finfo(dtype).tiny)
    whole = got.as_strided((N, ldc), (ldc, 1))
    assert bool((whole[:-1, M:] == 5).all())


def test_rows_at_the_ends_of_their_memory():
    """Unaligned rows that end where an allocation does: what follows the last one is not read (it is another's)."""
    for K in (255, 256, 257, 383, 384, 385):
        M, N = 33, 3
        A, scale, Bt = operands(M, N, K, 32, torch.bfloat16)
        big = torch.full((A.numel() + Bt.numel() * 2 + 64,), 255, dtype=torch.uint8, device="cuda")
        a = big[1:1 + A.numel()].view(A.shape)
        a.copy_(A)
        nan = torch.full((Bt.numel() + 9,), float("nan"), dtype=torch.bfloat16, device="cuda")
        b = nan[1:1 + Bt.numel()].view(Bt.shape)
        b.copy_(Bt)
        assert torch.equal(check(a, scale, b, 32), tn.w4_tn(A, Bt, scale, 32))


@pytest.mark.parametrize("dtype", DTYPES)
def test_exact_integers(dtype):
    """Small integers and scales of one: every sum is exact."""
    M, N, K = 300, 20, 640
    g = torch.Generator(device="cuda").manual_seed(3)
    A = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    A[0], A[1], A[2] = 0x88, 0x77, 0x80                              # -8 throughout; 7; 0 and -8
    B = (torch.randint(0, 33, (N, K), generator=g, device="cuda") == 0).to(dtype)
    ref = B.double() @ unpack(A, K).double().t()
    for group in GROUPS:
        scale = torch.ones(M, -(-K // group), device="cuda", dtype=dtype)
        got = tn.w4_tn(A, B, scale, group)
        assert torch.equal(got.double(), ref.to(dtype).double())


def test_infinities_and_nan_stay_where_they_are():
    A, scale, Bt = operands(64, 10, 300, 64, torch.float16)
    Bt[3, 17], Bt[7, 299] = float("nan"), float("inf")
    scale[5, 2] = float("nan")
    C = tn.w4_tn(A, Bt, scale, 64)
    bad = ~torch.isfinite(C)
    assert bool(bad[:, 5].all()) and bool(bad[3].all()) and bool(torch.isnan(C[3]).all())
    bad[3], bad[7], bad[:, 5] = False, False, False
    assert not bool(bad.any())


def test_empty():
    for M, N, K in ((0, 3, 64), (5, 0, 64), (5, 3, 0)):
        A, scale, Bt = operands(M, N, K, 32, torch.bfloat16)
        C = tn.w4_tn(A, Bt, scale, 32, C=torch.full((N, M), 3.0, device="cuda", dtype=torch.bfloat16))
        assert C.shape == (N, M) and not bool(C.any())
    q, s = tn.quantize_w4_rows(torch.zeros(0, 70, device="cuda"), 32, dtype=torch.float16)
    assert q.shape == (0, 35) and s.shape == (0, 3)
    q, s = tn.quantize_w4_rows(torch.zeros(3, 0, device="cuda"), 32, dtype=torch.float16)
    assert q.shape == (3, 0) and s.shape == (3, 0)


def quant64(x, group, dtype):
    rows, cols = x.shape
    pad = torch.zeros(rows, -(-cols // group) * group, device="cuda", dtype=torch.float64)
    pad[:, :cols] = x
    pad = pad.view(rows, -1, group)
    # the FP32 product by the FP32 number next to 1 / 7, as the header defines the scale
    scale = (pad.abs().amax(2).float() * torch.full((), 1 / 7, dtype=torch.float32, device="cuda")).to(dtype)
    by = scale.double()[..., None]
    q = torch.where(by > 0, (pad / torch.where(by > 0, by, 1.0)).round().clamp(-8, 7), 0.0)
    bad = ~torch.isfinite(scale)
    q[bad] = 0
    scale[bad] = float("nan")
    return q.flatten(1)[:, :cols].to(torch.int8), scale


def same(x, y):
    return torch.equal(torch.nan_to_num(x, nan=-1.0), torch.nan_to_num(y, nan=-1.0)) and torch.equal(torch.isnan(x), torch.isnan(y))


@pytest.mark.parametrize("source", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 32), (2, 33), (9, 255), (4, 256), (7, 1000), (3, 1027), (2000, 264)])
def test_quantiser(rows, cols, group, dtype, source):
    x = normals(rows, cols, seed=rows + cols, dtype=torch.float32) * torch.exp(2 * normals(rows, 1, seed=5, dtype=torch.float32))
    x = x.to(source)
    x[rows // 2, : cols // 2] = 0                                    # groups of zeros
    for ld in (cols, cols + 3, cols + 8):
        v = padded(x, ld, float("nan"))
        q, scale = tn.quantize_w4_rows(v, group, dtype=dtype)
        q64, s64 = quant64(v, group, dtype)
        assert torch.equal(unpack(q, cols), q64) and torch.equal(scale, s64)
        if cols % 2:
            assert not bool((q[:, -1] >> 4).any())


@pytest.mark.parametrize("source", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,ld", [(20001, 40, 40), (15001, 257, 257), (6001, 1029, 1032), (100003, 8, 24)])
def test_quantiser_of_many_rows(rows, cols, ld, source):
    """Several rows to a warp, each read while the one before it is worked on."""
    x = padded(normals(rows, cols, seed=rows, dtype=torch.float32).mul_(torch.arange(rows, device="cuda")[:, None] % 7).to(source), ld, float("inf"))
    for dtype, group in ((torch.float16, 32), (torch.bfloat16, 256)):
        q, scale = tn.quantize_w4_rows(x, group, dtype=dtype)
        q64, s64 = quant64(x, group, dtype)
        assert torch.equal(unpack(q, cols), q64) and torch.equal(scale, s64)


@pytest.mark.parametrize("source", [torch.float32, torch.float16, torch.bfloat16])
def test_quantiser_at_borders(source):
    """Quotients at and next to a half, and scales at the ends of their types."""
    dtype = torch.bfloat16 if source == torch.bfloat16 else torch.float16
    steps = torch.arange(-15, 16, device="cuda", dtype=torch.float64) / 2
    rows = []
    for s in (1.0, 1.5, 2.0 ** -10, 3.0 * 2.0 ** -12, 2.0 ** 8):
        x = torch.zeros(32, device="cuda", dtype=torch.float64)
        x[:31] = steps * s
        x[0], x[30], x[31] = 0.5 * s, -0.5 * s, 7.0 * s
        rows.append(x)
        if source == torch.float32:
            rows.append(x * (1 + 2.0 ** -23))
            rows.append(x * (1 - 2.0 ** -24))
    x = torch.stack(rows).to(source)
    if source == torch.float32:                                      # every half, a step above and a step below
        up, down = torch.nextafter(x, x + 1), torch.nextafter(x, x - 1)
        up[:, 31], down[:, 31] = x[:, 31], x[:, 31]
        x = torch.cat((x, up, down))
    q, scale = tn.quantize_w4_rows(x, 32, dtype=dtype)
    q64, s64 = quant64(x, 32, dtype)
    assert torch.equal(unpack(q, 32), q64) and torch.equal(scale, s64)
    # far ends: the smallest numbers, the largest, infinities and NaN
    tops = [0.0, 1e-45, 1e-40, 1e-38, 1e-30, 6e-8, 3e-7, 4.2e-7, 1e-6, 6e4, 4.5e5, 4.6e5, 1e30, 3e38, float("inf"), float("nan")]
    x = normals(len(tops), 64, seed=9, dtype=torch.float32).clamp_(-1, 1)
    x[:, 0] = 1
    x = (x * torch.tensor(tops, device="cuda")[:, None]).to(source)
    for d in DTYPES:
        q, scale = tn.quantize_w4_rows(x, 64, dtype=d)
        q64, s64 = quant64(x, 64, d)
        assert same(scale, s64), (scale, s64)
        assert torch.equal(unpack(q, 64), q64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantised_layer(dtype):
    """A layer quantised and used: quantiser and product together, also captured and replayed."""
    M, K, N, group = 500, 700, 5, 64
    W, x = (normals(M, K, seed=1, dtype=torch.float32) * K ** -0.5).to(dtype), normals(N, K, seed=2, dtype=dtype)
    q, scale = tn.quantize_w4_rows(W, group)
    C = check(q, scale, x, group)
    exact = x.double() @ W.double().t()
    # a weight is off by half a step of its group, at most amax / 14 (and the scale's rounding): of random signs
    assert float((C.double() - exact).norm() / exact.norm()) < 0.25
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tn.w4_tn(q, x, scale, group)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q2, scale2 = tn.quantize_w4_rows(W, group)
        C2 = tn.w4_tn(q2, x, scale2, group)
    W.copy_(normals(M, K, seed=11, dtype=torch.float32) * K ** -0.5)
    graph.replay()
    torch.cuda.synchronize()
    q, scale = tn.quantize_w4_rows(W, group)
    assert torch.equal(q, q2) and torch.equal(scale, scale2) and torch.equal(tn.w4_tn(q, x, scale, group), C2)
