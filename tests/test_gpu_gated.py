"""Gated projections and their gradients on the GPU against their 64-bit forms."""
import pytest
import torch

from tests.grouped_helpers import normals, offsets_of, padded
from tests.sink_helpers import act64, assert_within, gated64, gated_bound, gated_grad64

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

ACTS = ["silu", "gelu", "gelu_tanh"]
DTYPES = [torch.float16, torch.bfloat16]


def operands(E, T, M, K, dtype, seed=1):
    return (normals(E, 2 * M, K, seed=seed, dtype=torch.float32).mul_(K ** -0.5).to(dtype) if K else torch.empty(E, 2 * M, 0, device="cuda", dtype=dtype),
            normals(T, K, seed=seed + 1, dtype=dtype), normals(T, M, seed=seed + 2, dtype=dtype))


def check(A, Bt, dH, offsets, bounds, act, dtype, stream=None):
    dense = offsets is None
    W = A[0] if dense else A
    H, P = tn.tn_gated(W, Bt, offsets, act=act, keep=True, stream=stream)
    alone = tn.tn_gated(W, Bt, offsets, act=act, stream=stream)
    H64, P64, off = gated64(A, Bt, bounds, act)
    rows = slice(bounds[0], bounds[-1])
    assert torch.equal(H[rows], alone[rows])
    assert_within(P, P64, off + 2.0 ** -126, "P")
    assert_within(H, H64, gated_bound(P64, off, act, dtype), "H")
    dA, dB = tn.tn_gated_grad(W, Bt, P, dH, offsets, act=act, stream=stream)
    tn.gemm_poll_device_status()
    rA, rB, eA, eB = gated_grad64(A, Bt, P, dH, bounds, act, dtype)
    assert_within(dA.view(A.shape), rA, eA, "dA")
    assert_within(dB, rB, eB, "dB")
    return H, P, dA, dB


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,M,K", [(1, 1, 1), (1, 64, 64), (3, 17, 33), (1, 1000, 520), (33, 16, 8), (65, 200, 136), (130, 129, 72),
                                   (300, 513, 264), (777, 1000, 1000), (2048, 512, 256), (1, 4096, 2048), (16, 2048, 4096),
                                   (300, 5000, 256), (64, 6000, 100), (65, 6001, 128), (1000, 3000, 520)])
def test_dense(T, M, K, dtype):
    A, Bt, dH = operands(1, T, M, K, dtype)
    check(A, Bt, dH, None, [0, T], ACTS[(T + M + K) % 3], dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,M,K,lead", [([5, 0, 1, 40], 48, 64, 0), ([0, 130, 0, 300, 2], 136, 200, 3), ([257, 255, 0], 300, 24, 0),
                                             ([1] * 40, 72, 96, 0)])
def test_experts(counts, M, K, lead, dtype, act):
    offsets = offsets_of(counts, lead)
    bounds = offsets.tolist()
    T = bounds[-1] + 2
    A, Bt, dH = operands(len(counts), T, M, K, dtype)
    # rows of no expert hold what must not be read
    for t in (Bt, dH):
        t[:lead] = float("nan")
        t[bounds[-1]:] = float("inf")
    H = torch.full((T, M), 7.0, device="cuda", dtype=dtype)
    P = torch.full((T, 2 * M), 7.0, device="cuda")
    dB = torch.full((T, K), 7.0, device="cuda", dtype=dtype)
    check(A, Bt, dH, offsets, bounds, act, dtype)
    tn.tn_gated(A, Bt, offsets, act=act, H=H, P=P)
    tn.tn_gated_grad(A, Bt, P, dH, offsets, act=act, dBt=dB)
    for t in (H, P, dB):
        assert bool((t[:lead] == 7).all()) and bool((t[bounds[-1]:] == 7).all())
        assert bool(torch.isfinite(t[lead:bounds[-1]]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,M,K,lead", [([0, 0, 3, 0, 1], 40, 64, 0), ([1] * 13, 24, 136, 0), ([0] * 40 + [2] + [0] * 30 + [5], 17, 72, 3),
                                             ([0] * 31 + [1, 1, 9], 33, 200, 1), ([14, 0], 100, 512, 0), ([0, 0, 0], 24, 64, 5),
                                             ([3, 1, 0, 2], 1600, 136, 0), ([1, 4, 0, 0, 5], 900, 520, 4)])
def test_few_tokens_by_expert(counts, M, K, lead, dtype):
    """At most 16 rows: experts found among many without, and tiles for two CTAs an SM and for more."""
    offsets = offsets_of(counts, lead)
    bounds = offsets.tolist()
    T = bounds[-1] + 2
    assert T <= 16
    A, Bt, dH = operands(len(counts), T, M, K, dtype)
    rows = slice(lead, bounds[-1])
    Bt[:lead] = float("nan")
    Bt[bounds[-1]:] = float("inf")
    H, P = torch.full((T, M), 7.0, device="cuda", dtype=dtype), torch.full((T, 2 * M), 7.0, device="cuda")
    act = ACTS[len(counts) % 3]
    tn.tn_gated(A, Bt, offsets, act=act, H=H, P=P)
    tn.gemm_poll_device_status()
    H64, P64, off = gated64(A, Bt, bounds, act)
    assert_within(P[rows], P64[rows], (off + 2.0 ** -126)[rows], "P")
    assert_within(H[rows], H64[rows], gated_bound(P64, off, act, dtype)[rows], "H")
    for t in (H, P):
        assert bool((t[:lead] == 7).all()) and bool((t[bounds[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 8, 9, 16])
@pytest.mark.parametrize("M", [4864, 4865])
def test_few_tokens_and_many_rows(T, M, dtype):
    """16 rows a CTA: 304 of them, and one more."""
    A, Bt, dH = operands(1, T, M, 72, dtype)
    check(A, Bt, dH, None, [0, T], "silu", dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lda,ldb,ldh", [(72, 80, 56), (65, 67, 51), (64, 65, 50)])
def test_strides(lda, ldb, ldh, dtype):
    E, T, M, K = 3, 150, 50, 64
    counts = [70, 0, 80]
    offsets, bounds = offsets_of(counts), [0, 70, 70, 150]
    A, Bt, dH = operands(E, T, M, K, dtype)
    A, Bt, dH = padded(A, lda, float("nan")), padded(Bt, ldb, float("nan")), padded(dH, ldh, float("nan"))
    H, P, dA, dB = check(A, Bt, dH, offsets, bounds, "silu", dtype)
    # the results into padded rows, the padding left as it was
    Hp, Pp = padded(torch.zeros_like(H), ldh + 3, 5.0), padded(torch.zeros_like(P), 2 * M + 3, 5.0)
    dAp, dBp = padded(torch.zeros_like(dA), lda + 1, 5.0), padded(torch.zeros_like(dB), ldb + 1, 5.0)
    tn.tn_gated(A, Bt, offsets, H=Hp, P=Pp)
    tn.tn_gated_grad(A, Bt, Pp, dH, offsets, dA=dAp, dBt=dBp)
    for got, want in ((Hp, H), (Pp, P), (dAp, dA), (dBp, dB)):
        assert torch.equal(got, want)
        whole = got.as_strided((*got.shape[:-1], got.stride(-2)), got.stride())
        assert bool((whole[..., got.shape[-1]:] == 5).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_sums_and_results(dtype):
    A, Bt, dH = operands(2, 10, 24, 0, dtype)
    offsets = offsets_of([4, 6])
    H, P = tn.tn_gated(A, Bt, offsets, keep=True)
    assert not bool(H.any()) and not bool(P.any())
    dA, dB = tn.tn_gated_grad(A, Bt, P, dH, offsets)
    assert dA.shape == (2, 48, 0) and dB.shape == (10, 0)
    # no token
    A, Bt, dH = operands(1, 0, 24, 40, dtype)
    H, P = tn.tn_gated(A[0], Bt, keep=True)
    dA, dB = tn.tn_gated_grad(A[0], Bt, P, dH)
    assert H.shape == (0, 24) and dB.shape == (0, 40) and dA.shape == (48, 40) and not bool(dA.any())
    dA, _ = tn.tn_gated_grad(A, Bt, P, dH, offsets_of([0]))
    assert not bool(dA.any())
    # no result
    A, Bt, dH = operands(1, 10, 0, 40, dtype)
    H, P = tn.tn_gated(A[0], Bt, keep=True)
    dB = torch.full((10, 40), 3.0, device="cuda", dtype=dtype)
    dA, dB = tn.tn_gated_grad(A[0], Bt, P, dH, dBt=dB)
    assert H.shape == (10, 0) and dA.shape == (0, 40) and not bool(dB.any())
    tn.gemm_poll_device_status()


def test_one_gradient_alone():
    A, Bt, dH = operands(1, 100, 48, 72, torch.bfloat16)
    _, P = tn.tn_gated(A[0], Bt, keep=True)
    dA, dB = tn.tn_gated_grad(A[0], Bt, P, dH)
    a, none = tn.tn_gated_grad(A[0], Bt, P, dH, want_b=False)
    assert none is None and torch.equal(a, dA)
    none, b = tn.tn_gated_grad(A[0], Bt, P, dH, want_a=False)
    assert none is None and torch.equal(b, dB)


def test_same_rows_whatever_the_path():
    """A token's result does not depend on how many others the call has, within rounding; and calls repeat bit by bit."""
    A, Bt, dH = operands(1, 1500, 264, 512, torch.float16)
    H, P = tn.tn_gated(A[0], Bt, keep=True)
    first = tn.tn_gated_grad(A[0], Bt, P, dH)
    for _ in range(3):
        again, P2 = tn.tn_gated(A[0], Bt, keep=True)
        assert torch.equal(again, H) and torch.equal(P2, P)
        for x, y in zip(tn.tn_gated_grad(A[0], Bt, P, dH), first):
            assert torch.equal(x, y)


def test_values_at_the_ends():
    """Gates far out, infinities and NaN: each stays in its own row and result."""
    K = 16
    A = torch.zeros(1, 8, K, device="cuda", dtype=torch.bfloat16)
    A[0, 0, 0] = A[0, 1, 1] = A[0, 2, 2] = A[0, 3, 3] = 1        # gates: the first four terms
    A[0, 4:, 4] = 1                                             # up: the fifth
    x = torch.zeros(3, K, device="cuda", dtype=torch.bfloat16)
    x[0, :5] = torch.tensor([200.0, -200.0, 0.0, 1.0, 2.0])
    x[1, :5] = torch.tensor([1.0, 2.0, 3.0, float("nan"), 1.0])
    x[2, :5] = torch.tensor([1.0, 2.0, 3.0, 4.0, 1.0])
    for act in ACTS:
        H = tn.tn_gated(A[0], x, act=act)
        assert H[0].tolist()[:3] == [400.0, 0.0, 0.0]
        assert bool(torch.isnan(H[1]).all())                    # NaN is a term of every sum of its row
        want = act64(torch.tensor([1.0, 2.0, 3.0, 4.0], dtype=torch.float64), act)[0]
        assert bool(((H[2].double().cpu() - want).abs() <= 2.0 ** -8 * want).all())


def test_captured_and_replayed():
    A, Bt, dH = operands(2, 200, 64, 128, torch.bfloat16)
    offsets = offsets_of([150, 50])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tn.tn_gated(A, Bt, offsets, keep=True)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        H, P = tn.tn_gated(A, Bt, offsets, act="gelu", keep=True)
        dA, dB = tn.tn_gated_grad(A, Bt, P, dH, offsets, act="gelu")
    for seed in (5, 6):
        A2, B2, d2 = operands(2, 200, 64, 128, torch.bfloat16, seed)
        A.copy_(A2), Bt.copy_(B2), dH.copy_(d2)
        offsets.copy_(offsets_of([10 * seed, 200 - 10 * seed]))
        g.replay()
        torch.cuda.synchronize()
        H2, P2 = tn.tn_gated(A, Bt, offsets, act="gelu", keep=True)
        want = (H2, P2, *tn.tn_gated_grad(A, Bt, P2, dH, offsets, act="gelu"))
        for x, y in zip((H, P, dA, dB), want):
            assert torch.equal(x, y)


def test_other_stream():
    A, Bt, dH = operands(1, 300, 64, 100, torch.float16)        # (K = 100: copies in the workspace)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        check(A, Bt, dH, None, [0, 300], "silu", torch.float16, stream=s) if _ == 0 else None
        H, P = tn.tn_gated(A[0], Bt, keep=True, stream=s)
        dA, dB = tn.tn_gated_grad(A[0], Bt, P, dH, stream=s)
        del H, P
    s.synchronize()
    H, P = tn.tn_gated(A[0], Bt, keep=True)
    for x, y in zip(tn.tn_gated_grad(A[0], Bt, P, dH), (dA, dB)):
        assert torch.equal(x, y)
