"""8-bit integer products and the row quantiser on the GPU, against 64-bit forms."""
import pytest
import torch

from tests.grouped_helpers import HALF_STEP, offsets_of, padded

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_gemm_tn_gb300 as g

TYPES = [torch.float16, torch.bfloat16]


def codes(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=gen, device="cuda").to(torch.int8)


def scales(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (0.5 + torch.rand(*shape, generator=gen, device="cuda")) * 2.0 ** -10


def assert_scaled(got, sums, sa, sb, terms, dtype):
    """got against sums * sa * sb: half a step of the type, one FP32 rounding for
    each of the two scalings, and the FP32 sum's own (as in assert_near; sums of
    magnitudes at most terms * 2^14)."""
    ref = sums * sa.double() * sb.double()
    off = (terms + 15) // 16 * 17 * 2.0 ** -24 * terms * 2.0 ** 14 if terms * 2 ** 14 > 2 ** 24 else 0.0
    bound = ref.abs() * (HALF_STEP[dtype] * 1.001 + 2.0 ** -22) + off * sa.double() * sb.double() + torch.finfo(dtype).tiny
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (8, 1, 16), (128, 16, 128), (257, 3, 80), (64, 65, 63), (130, 300, 1000),
                                   (512, 64, 2048), (1000, 513, 333), (33, 100, 5), (300, 17, 144), (129, 128, 400),
                                   (2000, 100, 1040), (128, 129, 256), (40, 1, 4096), (640, 112, 16), (20000, 33, 128),
                                   (256, 257, 128), (300, 300, 144), (1000, 700, 400), (512, 1025, 2064), (77, 5000, 64), (8, 600, 16)]
                         # CTA pairs: tiles past one and a half waves of single CTAs
                         + [(2000, 1000, 400), (1290, 1537, 333), (1000, 4000, 48), (4096, 1025, 144), (520, 4097, 2064),
                            (33, 16000, 16), (300, 5000, 5), (129, 8000, 1040)]
                         # few tiles with long sums: split over clusters of 2, 4 and 8
                         + [(128, 16, 1536), (100, 5, 16384), (128, 64, 3100), (257, 33, 8191), (2000, 17, 2064),
                            (8192, 9, 2048), (1, 1, 100000), (2300, 65, 6000), (300, 200, 12300)])
def test_i8_product(M, N, K, dtype):
    A, Bt, sa, sb = codes(M, K, seed=1), codes(N, K, seed=2), scales(M, seed=3), scales(N, seed=4)
    C = g.i8_tn(A, Bt, sa, sb, dtype=dtype)
    g.gemm_poll_device_status()
    assert C.shape == (N, M) and C.dtype == dtype
    assert_scaled(C, Bt.double() @ A.double().t(), sa[None, :], sb[:, None], K, dtype)


@pytest.mark.parametrize("counts,M,K", [([1], 16, 16), ([0, 3, 0, 1], 128, 64), ([70, 0, 300], 200, 208), ([5, 6], 31, 33),
                                        ([1] * 40, 384, 272), ([64, 0, 65, 3], 130, 128), ([200, 10, 100], 136, 112),
                                        ([300, 0, 600], 264, 272), ([193, 192, 1000, 2], 520, 1040),
                                        ([3000, 0, 2600, 193], 520, 272), ([2192, 1930, 1000, 2], 520, 1040), ([9000, 100], 264, 33),
                                        ([3, 0, 70, 1], 200, 5000), ([1], 96, 20000), ([200, 9], 129, 2049)])
def test_i8_grouped(counts, M, K):
    E, T = len(counts), sum(counts)
    off = offsets_of(counts)
    A, Bt, sa, sb = codes(E, M, K, seed=1), codes(T, K, seed=2), scales(E, M, seed=3), scales(T, seed=4)
    C = g.i8_tn_grouped(A, Bt, sa, sb, off, dtype=torch.bfloat16)
    g.gemm_poll_device_status()
    b = off.tolist()
    for e in range(E):
        r = slice(b[e], b[e + 1])
        assert_scaled(C[r], Bt[r].double() @ A[e].double().t(), sa[e][None, :], sb[r][:, None], K, torch.bfloat16)


def grouped_sums(A, Bt, b):
    return torch.cat([Bt[b[e]:b[e + 1]].double() @ A[e].double().t() for e in range(A.shape[0])])


def test_extreme_codes_and_long_sums():
    """Sums past 2^24: of equal products they are exact in FP32 anyway, of mixed ones
    within the FP32 sum's bound."""
    for N in (3, 600):                              # widened on the way, and widened first
        for K in (1024, 16384):
            A = torch.full((130, K), -128, dtype=torch.int8, device="cuda")
            Bt = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
            one = torch.ones(130, device="cuda")
            C = g.i8_tn(A, Bt, one * 2.0 ** -20, torch.ones(N, device="cuda"))
            assert bool((C == K * 2.0 ** -6).all())
            A, Bt = codes(130, K, seed=5).clamp_(min=100), codes(N, K, seed=6)
            sa, sb = scales(130, seed=7) * 2.0 ** -6, scales(N, seed=8)
            C = g.i8_tn(A, Bt, sa, sb, dtype=torch.bfloat16)
            assert_scaled(C, Bt.double() @ A.double().t(), sa[None, :], sb[:, None], K, torch.bfloat16)


def long_codes(kind, M, N, K, seed):
    """Codes whose sums are about 0 (mixed), pass 2^24 many times over (same), or pass it
    and come back to a small number (cancel)."""
    A, Bt = codes(M, K, seed=seed), codes(N, K, seed=seed + 1)
    if kind == "mixed":
        return A, Bt
    A, Bt = (t.int().abs().clamp(64, 127).to(torch.int8) for t in (A, Bt))
    if kind == "cancel":
        half = K // 2
        A[:, K - half:] = -A[:, :half]
        Bt[:, K - half:] = Bt[:, :half]
        A[:, ::997] = codes(M, (K + 996) // 997, seed=seed + 2)
    return A, Bt


def scaled_once(sums, sa, sb, dtype):
    """The exact sums rounded to FP32, scaled in FP32 by the channel and then by the token,
    and rounded to the type: each step as the operator's definition has it."""
    return ((sums.float() * sa) * sb).to(dtype)


@pytest.mark.parametrize("kind", ["mixed", "same", "cancel"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1024), (1, 1, 1025), (64, 65, 2049), (129, 16, 3000), (100, 5, 16384), (300, 200, 12300),
                                   (832, 32, 12160), (20000, 40, 4096), (33, 64, 100000), (16, 3, 131071),
                                   # CTA pairs
                                   (2000, 1000, 1024), (2000, 1000, 1025), (520, 4097, 2064), (1290, 1537, 8191), (4096, 600, 16384), (8192, 257, 3001)])
def test_i8_sums_are_exact(M, N, K, kind):
    A, Bt = long_codes(kind, M, N, K, seed=K)
    sa, sb = scales(M, seed=3), scales(N, seed=4) / 64
    sums = Bt.double() @ A.double().t()
    for dtype in TYPES:
        C = g.i8_tn(A, Bt, sa, sb, dtype=dtype)
        g.gemm_poll_device_status()
        assert torch.equal(C, scaled_once(sums, sa[None, :], sb[:, None], dtype))


@pytest.mark.parametrize("kind", ["same", "cancel"])
@pytest.mark.parametrize("counts,M,K", [([3, 0, 70, 1], 200, 5000), ([200, 9], 129, 2049), ([1], 96, 20000),
                                        ([2192, 1930, 1000, 2], 520, 2080), ([3000, 0, 2600, 193], 520, 4001), ([40] * 40, 1000, 1500)])
def test_i8_grouped_sums_are_exact(counts, M, K, kind):
    E, T, off = len(counts), sum(counts), offsets_of(counts)
    A, Bt = long_codes(kind, E * M, T, K, seed=K)
    A, sa, sb = A.view(E, M, K), scales(E, M, seed=3), scales(T, seed=4) / 64
    b = off.tolist()
    rows = torch.cat([sa[e].expand(b[e + 1] - b[e], M) for e in range(E)])
    C = g.i8_tn_grouped(A, Bt, sa, sb, off)
    g.gemm_poll_device_status()
    assert torch.equal(C, scaled_once(grouped_sums(A, Bt, b), rows, sb[:, None], torch.float16))


@pytest.mark.parametrize("M,N", [(16, 3), (300, 5000)])
@pytest.mark.parametrize("K", [131071, 131072, 140001])
def test_i8_sums_at_the_end_of_32_bits(M, N, K):
    """Of 131071 terms the largest sum is 2^31 - 2^14; longer ones are FP32 sums of exact
    runs of 1024 terms: one rounding for each run, and for each part of a split sum."""
    one = torch.ones(M, device="cuda") * 2.0 ** -16
    A, Bt = (torch.full((n, K), -128, dtype=torch.int8, device="cuda") for n in (M, N))
    C = g.i8_tn(A, Bt, one, torch.ones(N, device="cuda"))
    assert bool((C == torch.tensor(float(K) / 4, device="cuda").half()).all())
    C = g.i8_tn(A, -(Bt + 1), one, torch.ones(N, device="cuda"))              # 127 * -128
    assert bool((C == torch.tensor(-float(K) * 127 / 512, device="cuda").half()).all())
    A, Bt = long_codes("cancel", M, N, K, seed=5)
    sa, sb = scales(M, seed=3), scales(N, seed=4) / 64
    C = g.i8_tn(A, Bt, sa, sb)
    g.gemm_poll_device_status()
    sums = Bt.double() @ A.double().t()
    if K <= 131071:
        assert torch.equal(C, scaled_once(sums, sa[None, :], sb[:, None], torch.float16))
    else:
        size = Bt.double().abs() @ A.double().abs().t()
        scale = sa.double()[None, :] * sb.double()[:, None]
        bound = ((K + 1023) // 1024 + 8) * 2.0 ** -24 * size * scale + (sums * scale).abs() * (2.0 ** -11 * 1.001 + 2.0 ** -22) + 2.0 ** -24
        assert bool(((C.double() - sums * scale).abs() <= bound).all())


@pytest.mark.parametrize("N", [5, 64, 600, 20000])
def test_every_code_widens_exactly(N):
    """A's rows hold all 256 values, Bt picks one term per row."""
    K = 256
    A = torch.arange(-128, 128, device="cuda").to(torch.int8).repeat(16, 1)
    Bt = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    at = (torch.arange(N, device="cuda") * 37) % K
    Bt[torch.arange(N, device="cuda"), at] = 1
    C = g.i8_tn(A, Bt, torch.ones(16, device="cuda"), torch.ones(N, device="cuda"))
    assert torch.equal(C, A[0, at].half()[:, None].expand(N, 16))
    C = g.i8_tn(Bt, A, torch.ones(N, device="cuda"), torch.ones(16, device="cuda"))
    assert torch.equal(C, A[0, at].half()[None, :].expand(16, N))


@pytest.mark.parametrize("M,N,K,pad", [(200, 17, 144, 16), (200, 17, 144, 1), (130, 600, 48, 32), (65, 3, 33, 0),
                                       (130, 9000, 48, 32), (130, 9000, 48, 1), (65, 3, 4001, 3), (200, 70, 2064, 16)])
def test_i8_strides(M, N, K, pad):
    A, Bt = padded(codes(M, K, seed=1), K + pad, 99), padded(codes(N, K, seed=2), K + pad, -77)
    sa, sb = scales(M, seed=3), scales(N, seed=4)
    C = padded(torch.full((N, M), 5.5, dtype=torch.float16, device="cuda"), M + pad, 5.5)
    g.i8_tn(A, Bt, sa, sb, C=C)
    assert_scaled(C, Bt.double() @ A.double().t(), sa[None, :], sb[:, None], K, torch.float16)
    assert bool((C.as_strided((N, M + pad), (M + pad, 1))[:, M:] == 5.5).all())


def test_i8_rows_of_no_expert_and_bad_offsets():
    M, K, T = 136, 80, 90
    A, Bt, sa, sb = codes(3, M, K, seed=1), codes(T, K, seed=2), scales(3, M, seed=3), scales(T, seed=4)
    for table in ([10, 30, 30, 80], [-4, 50, 20, 70], [0, 200, 0, 0]):
        b, top = [], 0
        for o in table:
            top = max(top, min(max(o, 0), T))
            b.append(top)
        C = torch.full((T, M), 5.5, dtype=torch.bfloat16, device="cuda")
        g.i8_tn_grouped(A, Bt, sa, sb, torch.tensor(table, dtype=torch.int32, device="cuda"), C=C)
        rows = slice(b[0], b[3])
        sa_rows = torch.cat([sa[e].expand(b[e + 1] - b[e], M) for e in range(3)])
        assert_scaled(C[rows], grouped_sums(A, Bt, b), sa_rows, sb[rows][:, None], K, torch.bfloat16)
        assert bool((C[:b[0]] == 5.5).all()) and bool((C[b[3]:] == 5.5).all())


def test_i8_scales_of_zero_nan_and_infinity_stay_in_their_row_and_column():
    M, N, K = 140, 70, 64
    A, Bt, sa, sb = codes(M, K, seed=1), codes(N, K, seed=2), scales(M, seed=3), scales(N, seed=4)
    clean = g.i8_tn(A, Bt, sa, sb)
    sa[3], sa[130], sb[5], sb[69] = 0, float("nan"), float("nan"), 0
    C = g.i8_tn(A, Bt, sa, sb)
    assert bool(C[5].isnan().all()) and bool(C[:, 130].isnan().all())
    keep_n, keep_m = torch.ones(N, dtype=torch.bool), torch.ones(M, dtype=torch.bool)
    keep_n[[5, 69]] = False
    keep_m[[3, 130]] = False
    assert torch.equal(C[keep_n][:, keep_m], clean[keep_n][:, keep_m])
    assert bool((C[69][keep_m] == 0).all()) and bool((C[keep_n, 3] == 0).all())


def test_i8_empty_sums():
    i8 = dict(dtype=torch.int8, device="cuda")
    C = torch.full((5, 40), 9.0, dtype=torch.float16, device="cuda")
    g.i8_tn(torch.zeros(40, 0, **i8), torch.zeros(5, 0, **i8), torch.ones(40, device="cuda"), torch.ones(5, device="cuda"), C=C)
    assert bool((C == 0).all())


@pytest.mark.parametrize("rows", [700, 15000])
def test_i8_captured_on_two_streams(rows):
    cases = [(codes(3, 200, 144, seed=i), codes(150, 144, seed=i + 1), scales(3, 200, seed=i + 2), scales(150, seed=i + 3),
              offsets_of([100, 0, 50])) for i in (1, 20)]
    wide = [(codes(96, 80, seed=i), codes(rows, 80, seed=i + 1), scales(96, seed=i + 2), scales(rows, seed=i + 3)) for i in (40, 60)]
    run = [lambda c=c, w=w: (g.i8_tn_grouped(*c), g.i8_tn(*w)) for c, w in zip(cases, wide)]
    want = [r() for r in run]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in run:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(r())
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(out, w))
    g.gemm_poll_device_status()


@pytest.mark.parametrize("N,mode", [(20, 1), (20, 2), (20, 3), (700, 1), (700, 2), (3000, 1), (3000, 2), (3000, 3)])
def test_i8_stalled_role_reports_a_timeout(N, mode):
    """20 and 700 rows: single CTAs, with 20 in clusters that share a tile's sum; 3000:
    CTA pairs (mode 3: the producers of all but a cluster's first CTA)."""
    args = codes(600, 2048, seed=1), codes(N, 2048, seed=2), scales(600, seed=3), scales(N, seed=4)
    want = g.i8_tn(*args)
    g.gemm_poll_device_status()
    g.gemm_set_wait_limit_ns(20_000_000)
    g.gemm_debug_inject_stall(mode)
    try:
        g.i8_tn(*args)
        with pytest.raises(g.GemmError) as e:
            g.gemm_poll_device_status()
        assert e.value.status == g.GEMM_ERR_TIMEOUT
    finally:
        g.gemm_debug_inject_stall(0)
        g.gemm_set_wait_limit_ns(0)
    assert torch.equal(g.i8_tn(*args), want)
    g.gemm_poll_device_status()


@pytest.mark.parametrize("M,N,K", [(832, 32, 12160), (2048, 16, 4096), (100, 130, 9000)])
def test_i8_split_sums_repeat_bit_for_bit_beside_others(M, N, K):
    """Parts of a sum are joined in one order, whatever else runs."""
    args = codes(M, K, seed=1), codes(N, K, seed=2), scales(M, seed=3), scales(N, seed=4)
    other = codes(512, 640, seed=5), codes(900, 640, seed=6), scales(512, seed=7), scales(900, seed=8)
    want = g.i8_tn(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.i8_tn(*args)
    s = torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s):
            g.i8_tn(*other)
            got.append(g.i8_tn(*args))
        graph.replay()
    torch.cuda.synchronize()
    g.gemm_poll_device_status()
    assert all(torch.equal(x, want) for x in got + [out])


def test_past_2_31_elements():
    M, K, E = 4096, 4096, 130
    A = torch.zeros(E, M, K, dtype=torch.int8, device="cuda")
    A[E - 1] = codes(M, K, seed=1)
    Bt, sa, sb = codes(40, K, seed=2), torch.zeros(E, M, device="cuda"), scales(40, seed=3)
    sa[E - 1] = scales(M, seed=4)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 40
    C = g.i8_tn_grouped(A, Bt, sa, sb, off)
    assert_scaled(C, Bt.double() @ A[E - 1].double().t(), sa[E - 1][None, :], sb[:, None], K, torch.float16)


def test_quantised_layer_together():
    """Weights by channel and tokens by row to 8 bits, then the product: near the
    unquantised one by the two quantisations' half steps."""
    T, M, K = 37, 300, 512
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in ((T, K), (M, K)))
    qx, sx = g.quantize_i8_rows(x)
    qw, sw = g.quantize_i8_rows(w)
    y = g.i8_tn(qw, qx, sw, sx, dtype=torch.bfloat16)
    g.gemm_poll_device_status()
    # |x - q s| <= s / 2 for either operand
    x64, w64 = x.double(), w.double()
    bound = (sx.double()[:, None] / 2 * w64.abs().sum(1) + x64.abs().sum(1, keepdim=True) * sw.double() / 2
             + K * sx.double()[:, None] * sw.double() / 4)
    ref = x64 @ w64.t()
    assert bool(((y.double() - ref).abs() <= bound * 1.001 + (ref.abs() + bound) * 2.0 ** -8).all())


def rows64(x):
    top = x.double().abs().amax(1, keepdim=True) if x.shape[1] else torch.zeros(x.shape[0], 1, device=x.device).double()
    q = torch.where(top > 0, (x.double() * 127 / top).round(), torch.zeros_like(x.double()))
    return q, top[:, 0] / 127


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 16), (5, 2048), (17, 1000), (300, 513), (2, 40000), (2, 70001), (3, 66000), (2000, 37), (1300, 200), (1301, 2049), (1500, 4097), (5, 16385), (3, 9000), (4, 32768), (2, 32770)])
def test_quantise_rows(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows * 131 + cols)
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * 3).to(dtype)
    x[0] = 0
    q, s = g.quantize_i8_rows(x)
    want, scale = rows64(x)
    assert torch.equal(q.double(), want)
    assert torch.equal(s, scale.float())


def exact_codes(row):
    """round(127 x / amax), ties to even, in rational arithmetic."""
    from fractions import Fraction
    x = [Fraction(float(v)) for v in row]
    top = max(abs(v) for v in x)
    return [round(127 * v / top) if top else 0 for v in x]        # (Fraction rounds ties to even)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
def test_quantise_borders_and_ties(dtype):
    """Values on and either side of every border of two codes, for row maxima with odd
    and even mantissas."""
    rows = []
    for top in (1.0, 127.0, 254.0, 1.5, 3.1415, 0.8203125, 100.375):
        top = float(torch.tensor(top, dtype=dtype))
        row = torch.tensor([(n + 0.5) * top / 127 for n in range(127)], dtype=torch.float64).to(dtype)
        up = torch.nextafter(row.float(), torch.full_like(row.float(), 1e9)) if dtype == torch.float32 else (row.view(torch.int16) + 1).view(dtype)
        down = torch.nextafter(row.float(), torch.zeros_like(row.float())) if dtype == torch.float32 else (row.view(torch.int16) - 1).view(dtype)
        rows.append(torch.cat([torch.tensor([top], dtype=dtype), row, -row, up.to(dtype), -down.to(dtype), down.to(dtype)]).clamp(-top, top))
    x = torch.stack(rows)
    q, s = g.quantize_i8_rows(x.cuda())
    for r in range(x.shape[0]):
        assert q[r].cpu().tolist() == exact_codes(x[r].double().tolist()), r
    assert torch.equal(s.cpu(), (x.double().abs().amax(1) / 127).float())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 64, 100, 2049, 9000])
def test_quantise_extreme_rows(cols, dtype):
    info = torch.finfo(dtype)
    gen = torch.Generator(device="cuda").manual_seed(cols)
    base = torch.rand(6, cols, generator=gen, device="cuda", dtype=torch.float64) * 2 - 1
    tiny = info.smallest_normal
    x = torch.stack([base[0] * info.max, base[1] * tiny * 0.9, base[2] * tiny * 300, base[3] * 0, base[4], base[5] * info.max]).to(dtype)
    x[3] = -0.0
    x[4, -1] = float("nan")
    x[5, cols // 2] = float("-inf")
    q, s = g.quantize_i8_rows(x)
    want, scale = rows64(x[:4])
    assert torch.equal(q[:4].double(), want)
    assert torch.equal(s[:4], scale.float())
    assert bool(s[4:].isnan().all()) and bool((q[4:] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,ld,base", [(4, 100, 104, 0), (4, 100, 103, 0), (7, 33, 40, 1), (3, 1, 9, 3), (1400, 50, 57, 5),
                                               (9, 2100, 2107, 2), (3, 17000, 17001, 1), (2, 50001, 50003, 3)])
def test_quantise_strides_and_bases(rows, cols, ld, base, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    room = torch.randn(base + rows * ld, generator=gen, device="cuda").mul_(50).to(dtype)
    x = room[base:].as_strided((rows, cols), (ld, 1))
    for q_base, q_ld in ((0, cols), (0, cols + 5), (3, cols + 8), (8, cols // 16 * 16 + 16)):
        out = torch.full((q_base + rows * q_ld + 16,), 55, dtype=torch.int8, device="cuda")
        scale = torch.zeros(rows, device="cuda")
        g.gemm_quantize_i8_rows(x, {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dtype], rows, cols, ld,
                                out.data_ptr() + q_base, q_ld, scale)
        q = out[q_base:].as_strided((rows, cols), (q_ld, 1))
        want, s = rows64(x)
        assert torch.equal(q.double(), want) and torch.equal(scale, s.float())
        q.fill_(55)
        assert bool((out == 55).all())               # nothing beside the codes was written


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [16383, 32765, 49000, 49001, 49007, 49008, 49009, 49100, 49135, 49136, 49137, 49153, 65535])
def test_quantise_unaligned_rows_about_the_most_that_is_staged(cols, dtype):
    """Rows that start on no 16-byte boundary, either side of the lengths where the
    staged codes outgrow shared memory and one kernel follows another."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    room = torch.randn(3 * (cols + 1), generator=gen, device="cuda").to(dtype)
    for x in (room[1:].as_strided((3, cols), (cols + 1, 1)), room[:2 * cols].view(2, cols), room[1:1 + cols].view(1, cols)):
        q, s = g.quantize_i8_rows(x)
        want, scale = rows64(x)
        assert torch.equal(q.double(), want) and torch.equal(s, scale.float())


def test_quantise_empty_and_dependent_launches():
    q, s = g.quantize_i8_rows(torch.zeros(5, 0, device="cuda"))
    assert q.shape == (5, 0) and bool((s == 0).all())
    q, s = g.quantize_i8_rows(torch.zeros(0, 7, device="cuda"))
    assert q.shape == (0, 7) and s.shape == (0,)
    x = torch.zeros(40, 300, device="cuda", dtype=torch.bfloat16)
    src = torch.randn(40, 300, device="cuda").bfloat16()
    w, sw = codes(64, 300, seed=1), scales(64, seed=2)
    want_q, want_s = g.quantize_i8_rows(src)
    want = g.i8_tn(w, want_q, sw, want_s)
    for _ in range(30):
        x.zero_()
        x.copy_(src)
        q, s = g.quantize_i8_rows(x)
        assert torch.equal(g.i8_tn(w, q, sw, s), want)
    assert torch.equal(q, want_q)
