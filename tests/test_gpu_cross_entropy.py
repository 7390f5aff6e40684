"""Softmax cross entropy of a projection, and its gradients, on the GPU against their 64-bit forms."""
import pytest
import torch

from tests.grouped_helpers import normals, padded
from tests.sink_helpers import assert_within, loss64, loss_grad64

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

DTYPES = [torch.float16, torch.bfloat16]


def operands(N, M, K, dtype, seed=1, spread=2.5):
    A = normals(M, K, seed=seed, dtype=torch.float32).mul_(spread * max(K, 1) ** -0.5).to(dtype)
    Bt = normals(N, K, seed=seed + 1, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    targets = torch.randint(0, M, (N,), generator=g, device="cuda")
    dloss = torch.rand(N, generator=g, device="cuda") / N
    return A, Bt, targets, dloss


def check(A, Bt, targets, dloss, dtype, stream=None):
    loss, lse = tn.tn_cross_entropy(A, Bt, targets, stream=stream)
    loss_ref, lse_ref, e_loss, e_lse, _, _ = loss64(A, Bt, targets)
    assert_within(lse, lse_ref, e_lse, "lse")
    assert_within(loss, loss_ref, e_loss, "loss")
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, stream=stream)
    tn.gemm_poll_device_status()
    rA, rB, eA, eB = loss_grad64(A, Bt, targets, dloss, dtype, lse)
    assert_within(dA, rA, eA, "dA")
    assert_within(dB, rB, eB, "dB")
    return loss, lse, dA, dB


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", [(1, 1, 1), (1, 2, 8), (2, 33, 17), (31, 32, 64), (1, 5000, 256), (33, 257, 100), (64, 1000, 136),
                                   (130, 4099, 72), (257, 3001, 264), (1000, 700, 40), (7, 70001, 64),
                                   (5, 900, 4104), (64, 3000, 1096), (300, 2100, 2048), (257, 40000, 1100)])
def test_loss_and_gradients(N, M, K, dtype):
    A, Bt, targets, dloss = operands(N, M, K, dtype)
    check(A, Bt, targets, dloss, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", [(40000, 3500, 48), (20000, 7777, 48), (4000, 40000, 72), (65537, 9217, 24)])
def test_pieces_of_the_vocabulary(N, M, K, dtype):
    """Several pieces: sums that go on from one to the next (also in parts), targets in each of them, a last one of one class."""
    A, Bt, targets, dloss = operands(N, M, K, dtype)
    assert tn.gemm_cross_entropy_workspace(1, M, N, K, A, K, Bt, K) < 2 * N * M
    n = min(N, M)
    targets[:n] = torch.arange(M - n, M, device="cuda")
    check(A, Bt, targets, dloss, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", [(1, 20000, 200), (64, 30000, 136), (65, 30001, 64), (500, 20011, 264), (1021, 9000, 520), (2500, 4100, 1000)])
def test_sums_in_parts(N, M, K, dtype):
    """Few tokens and many classes: the token gradient's sums in parts."""
    A, Bt, targets, dloss = operands(N, M, K, dtype)
    first = check(A, Bt, targets, dloss, dtype)
    again = tn.tn_cross_entropy_grad(A, Bt, targets, first[1], dloss)
    assert torch.equal(first[2], again[0]) and torch.equal(first[3], again[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_ignored_tokens(dtype):
    A, Bt, targets, dloss = operands(300, 1003, 64, dtype)
    targets[::3] = -100
    targets[1] = -1
    dloss[::3] = float("nan")                          # nobody looks at it
    loss, lse, dA, dB = check(A, Bt, targets, torch.where(targets < 0, 0.0, dloss), dtype)
    assert not bool(loss[targets < 0].any()) and not bool(dB[targets < 0].any())
    dA2, dB2 = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    assert torch.equal(dA, dA2) and torch.equal(dB, dB2)
    targets[:] = -100                                  # all of them
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    assert not bool(loss.any()) and not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M", [(40, 1000), (600, 2000)])
def test_long_sums_lose_nothing(N, M, dtype):
    """8192 terms: sums of 1024, each short by 64 steps' truncations at most (2^-24 of the running sum each, half of
    that on average, and the running sum half of the whole), all logits alike: the loss within 2^-18 of itself."""
    A, Bt, targets, dloss = operands(N, M, 8192, dtype)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    ref, lse_ref, _, _, _, _ = loss64(A, Bt, targets)
    assert float((loss.double() - ref).norm() / ref.norm()) < 2.0 ** -18
    assert float((lse.double() - lse_ref).norm() / lse_ref.norm()) < 2.0 ** -19


@pytest.mark.parametrize("N", [3900, 3000, 1537])
def test_a_mean_loss_rounds_no_gradient_alike(N):
    """dloss = 1 / N for all tokens: not a number of 8 bits, and the targets' d = -1 / N nearly.  Rounded itself it would be
    off by the same 0.2 % everywhere; the 2-norm of the error stays that of random roundings, at most 2^-9 each
    (d's and the result's: 1.5 x 2^-9 in the norm, were all at their largest 2^-8.5)."""
    A, Bt, targets, _ = operands(N, 5000, 64, torch.bfloat16, spread=0.5)
    dloss = torch.full((N,), 1 / N, device="cuda")
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    rA, rB, _, _ = loss_grad64(A, Bt, targets, dloss, torch.bfloat16, lse)
    for got, ref in ((dA, rA), (dB, rB)):
        assert float((got.double() - ref).norm() / ref.norm()) < 2.0 ** -8.5
        along = float((got.double() * ref).sum() / (ref * ref).sum()) - 1       # the error they share
        assert abs(along) < 2.0 ** -11


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_loss_gradient_that_is_not_finite(dtype, bad):
    """One token's; the others' rows stay what they are, gradients in the hundreds among them."""
    A, Bt, targets, dloss = operands(70, 100, 64, dtype)
    dloss *= 70 * 900
    lse = tn.tn_cross_entropy(A, Bt, targets)[1]
    kept = dloss.clone()
    kept[7] = 0
    _, rB, _, eB = loss_grad64(A, Bt, targets, kept, dtype, lse)
    dloss[7] = bad
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    others = torch.arange(70, device="cuda") != 7
    assert_within(dB[others], rB[others], eB[others], "dB")
    assert not bool(torch.isfinite(dB[7]).any()) and not bool(torch.isfinite(dA).any())


def test_targets_that_are_no_class():
    A, Bt, targets, dloss = operands(70, 100, 64, torch.bfloat16)
    targets[3], targets[40] = 100, 1 << 40
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    assert torch.isnan(loss).nonzero().flatten().tolist() == [3, 40] and bool(torch.isfinite(lse).all())
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    assert torch.isnan(dB).all(1).nonzero().flatten().tolist() == [3, 40] and int(torch.isnan(dB).any(1).sum()) == 2
    assert bool(torch.isnan(dA).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_logits_far_apart(dtype):
    """Rows whose logits differ by thousands, and by nothing: one class takes all, or all share."""
    N, M, K = 64, 500, 64
    A, Bt, targets, dloss = operands(N, M, K, dtype, spread=8.0)
    Bt[::2] *= 100.0
    Bt[1] = 0.0
    check(A, Bt, targets, dloss, dtype)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    assert abs(float(lse[1]) - float(torch.log(torch.tensor(500.0)))) < 1e-6 * 7


def test_infinities_and_nan_stay_in_their_token():
    A, Bt, targets, dloss = operands(100, 300, 32, torch.float16)
    Bt[5, 0], Bt[50, 1] = float("nan"), float("inf")
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    assert torch.isnan(loss).nonzero().flatten().tolist() == [5, 50]
    _, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, want_a=False)
    assert torch.isnan(dB).any(1).nonzero().flatten().tolist() == [5, 50]


@pytest.mark.parametrize("scale", [1e-30, 1.0, 65536.0, 1e30])
def test_gradients_of_any_scale(scale):
    """fp16 gradients of a loss's gradient far from one: the softmax's own are scaled on the way."""
    N, M, K = 100, 2000, 64
    A, Bt, targets, dloss = operands(N, M, K, torch.bfloat16)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    rA, rB, eA, eB = loss_grad64(A, Bt, targets, dloss * scale, torch.bfloat16, lse)
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss * scale)
    assert_within(dA, rA, eA, "dA")
    assert_within(dB, rB, eB, "dB")
    if scale <= 65536.0:
        A, Bt = A.half(), Bt.half()
        loss, lse = tn.tn_cross_entropy(A, Bt, targets)
        dloss = dloss * scale
        dloss[::2] *= 2.0 ** -12
        rA, rB, eA, eB = loss_grad64(A, Bt, targets, dloss, torch.float16, lse)
        dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
        assert_within(dA, rA, eA, "dA")
        assert_within(dB, rB, eB, "dB")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lda,ldb", [(72, 80), (65, 67), (64, 65)])
def test_strides(lda, ldb, dtype):
    A, Bt, targets, dloss = operands(150, 301, 64, dtype)
    A, Bt = padded(A, lda, float("nan")), padded(Bt, ldb, float("nan"))
    _, lse, dA, dB = check(A, Bt, targets, dloss, dtype)
    dAp, dBp = padded(torch.zeros_like(dA), lda + 1, 5.0), padded(torch.zeros_like(dB), ldb + 1, 5.0)
    tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, dA=dAp, dBt=dBp)
    for got, want in ((dAp, dA), (dBp, dB)):
        assert torch.equal(got, want)
        whole = got.as_strided((got.shape[0], got.stride(0)), got.stride())
        assert bool((whole[:, got.shape[1]:] == 5).all())


def test_empty():
    A, Bt, targets, dloss = operands(0, 100, 64, torch.bfloat16)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    assert loss.shape == lse.shape == (0,) and dB.shape == (0, 64) and not bool(dA.any())
    A, Bt, targets, dloss = operands(50, 100, 0, torch.bfloat16)          # logits of 0
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    want = torch.log(torch.tensor(100.0, dtype=torch.float64))
    assert float((loss.double().cpu() - want).abs().max()) < 2e-6 and torch.equal(loss, lse)
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    assert dA.shape == (100, 0) and dB.shape == (50, 0)


def test_one_gradient_alone_and_again():
    A, Bt, targets, dloss = operands(500, 2000, 128, torch.bfloat16)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    a, none = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, want_b=False)
    assert none is None and torch.equal(a, dA)
    none, b = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, want_a=False)
    assert none is None and torch.equal(b, dB)
    loss2, lse2 = tn.tn_cross_entropy(A, Bt, targets)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)


def test_captured_and_replayed():
    A, Bt, targets, dloss = operands(200, 1500, 96, torch.float16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        loss, lse = tn.tn_cross_entropy(A, Bt, targets)
        tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        loss, lse = tn.tn_cross_entropy(A, Bt, targets)
        dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    for seed in (5, 6):
        for x, y in zip((A, Bt, targets, dloss), operands(200, 1500, 96, torch.float16, seed)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        want = tn.tn_cross_entropy(A, Bt, targets)
        want += tn.tn_cross_entropy_grad(A, Bt, targets, want[1], dloss)
        for x, y in zip((loss, lse, dA, dB), want):
            assert torch.equal(x, y)
