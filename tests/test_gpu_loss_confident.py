"""The loss's gradients of tokens whose target has nearly all of the mass: what is left of 1 - p is small, and it must
not drown in what the logits of the two passes differ by."""
import pytest
import torch

from tests.grouped_helpers import HALF_STEP, normals

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

DTYPES = [torch.float16, torch.bfloat16]


def lse_error(lse):
    """What an lse from 16 to 64 may be off beside its logits: half a step of FP32 (2^-20 below 32, else 2^-19), and the sum of
    exponentials, near one, which is rounded by at most 2^-24 in each addition that it goes through with its largest part, 32 at
    most (15 of a piece's, 16 and 9 of the join's): 2^-19 in all."""
    assert 16 < float(lse.min()) and float(lse.max()) < 64
    return torch.where(lse < 32, 2.0 ** -20, 2.0 ** -19).double() + 2.0 ** -19


def confident(N, M, K, dtype, shift, gap, seed=1):
    """Logits of shift + N(0, 0.3^2), each token's own target `gap` above the others."""
    Bt = normals(N, K, seed=seed, dtype=torch.float32)
    A = normals(M, K, seed=seed + 1, dtype=torch.float32) * (0.3 * K ** -0.5)
    Bt[:, 0], A[:, 0] = 4.0, shift / 4
    targets = torch.randperm(M, generator=torch.Generator().manual_seed(seed + 2))[:N].cuda()
    A[targets] += gap / K * Bt                                     # (each a class of its own; |Bt|^2 is about K)
    A[:, 0] = shift / 4
    return A.to(dtype), Bt.to(dtype), targets


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K,shift,gap", [(40, 3000, 4096, 16.0, 14.0), (64, 2000, 8192, 10.0, 15.0), (300, 4000, 4096, 14.0, 15.0),
                                             (257, 3000, 8192, 12.0, 16.0), (1000, 2500, 4104, 16.0, 15.0), (5, 1000, 16384, 8.0, 14.0),
                                             (130, 3000, 1024, 14.0, 15.0), (200, 3000, 1100, 14.0, 14.0)])
def test_what_is_left_of_a_probability(N, M, K, shift, gap, dtype):
    """Each token's row of dB against 64 bits with the exact log-sum-exp.  At the target: lse_error, as both passes' logits are
    the same sums.  Elsewhere d is off by p's relative error (the logits' own, below 2^-13 here, and the exponential's).  Then d is
    rounded, and the result."""
    A, Bt, targets = confident(N, M, K, dtype, shift, gap)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    dloss = torch.ones(N, device="cuda")
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    tn.gemm_poll_device_status()
    Z = Bt.double() @ A.double().t()
    exact = torch.logsumexp(Z, 1)
    rounded = lse_error(exact)
    rows = torch.arange(N, device="cuda")
    d = torch.exp(Z - exact[:, None])
    d[rows, targets] = torch.expm1(Z[rows, targets] - exact)
    left = -d[rows, targets]
    assert float(left.min()) > 2e-5 and float(left.median()) < 4e-2
    half = HALF_STEP[dtype]
    W = A.double()
    off = d.abs() * (1.01 * half + 2.0 ** -13)
    off[rows, targets] += rounded
    want = d @ W
    bound = off @ W.abs()
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    bad = (dB.double() - want).abs() - (bound + half * want.abs() + tiny + (M / 16 * 17) * 2.0 ** -24 * (d.abs() @ W.abs()))
    assert float(bad.max()) <= 0
    # and in the norm of a row.  The target's d is off by the lse's error and by half a step of its own, both times the norm of
    # the target's row of A (whose first column, 4 or less, all classes share: it cancels in dB, sum d = 0, but not in d's rounding).
    # The other classes' roundings are of random sign: four times the root of their squares.  Then the result's, half a step.
    err, size = (dB.double() - want).norm(dim=1), want.norm(dim=1)
    at = W[targets].norm(dim=1)
    rest = d.clone()
    rest[rows, targets] = 0
    others = (rest.square() @ W.square().sum(1, keepdim=True))[:, 0].sqrt()
    limit = at * (rounded + half * left) + 4 * half * others + 2.0 ** -13 * left * at + half * size + tiny * K ** 0.5
    assert bool((err <= limit).all()), float((err / limit).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(40, 4096), (300, 4096), (600, 8192)])
def test_each_token_adds_up_to_nothing(N, K, dtype):
    """sum over the classes of d is 0: a column of ones in A shows it.  Left are the lse's rounding and d's own, at most half a
    step of each number, of random sign."""
    M = 3000
    A, Bt, targets = confident(N, M, K, dtype, 14.0, 15.0)
    A[:, 1] = 1.0
    Bt[:, 1] = 0.0                                                 # (the column takes no part in the logits)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    _, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, torch.ones(N, device="cuda"), want_a=False)
    Z = Bt.double() @ A.double().t()
    p = torch.softmax(Z, 1)
    rows = torch.arange(N, device="cuda")
    p[rows, targets] = -torch.expm1(torch.log_softmax(Z, 1)[rows, targets])      # sizes of d
    bound = lse_error(torch.logsumexp(Z, 1)) + HALF_STEP[dtype] * p.norm(dim=1) * 4 + HALF_STEP[dtype] * 2.0 ** -10
    assert bool((dB[:, 1].double().abs() <= bound).all()), float((dB[:, 1].double().abs() / bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", [(40, 2000, 4096), (300, 3000, 8192), (1, 500, 2056), (700, 20011, 3000)])
def test_long_sums_repeat_and_share_their_segments(N, M, K, dtype):
    """Ordinary logits over long sums: gradients repeat bit by bit, and each alone is what it is with the other."""
    A = normals(M, K, seed=4, dtype=torch.float32).mul_(2.5 * K ** -0.5).to(dtype)
    Bt = normals(N, K, seed=5, dtype=dtype)
    targets = torch.randint(0, M, (N,), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    targets[::5] = -1
    _, lse = tn.tn_cross_entropy(A, Bt, targets)
    dloss = torch.rand(N, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    again = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    alone = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, want_b=False)[0]
    tn.gemm_poll_device_status()
    assert torch.equal(dA, again[0]) and torch.equal(dB, again[1]) and torch.equal(dA, alone)
    Z = Bt.double() @ A.double().t()
    d = torch.softmax(Z, 1)
    d[torch.arange(N, device="cuda"), targets.clamp(min=0)] -= 1
    d *= torch.where(targets < 0, 0.0, dloss.double())[:, None]
    for got, want in ((dA, d.t() @ Bt.double()), (dB, d @ A.double())):
        assert float((got.double() - want).norm()) <= 1.5 * HALF_STEP[dtype] * float(want.norm()) + 1e-12


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,M,K", [(40, 3000, 512), (300, 2000, 1024), (1000, 3000, 64), (257, 40000, 136)])
def test_small_losses(N, M, K, dtype):
    """Losses of 1e-4 to 1e-2 where the lse is near 30: log(1 + rest), which the lse's rounding is no part of.  Off are the sum of
    exponentials (2^-19, as in lse_error), the logarithm, and the rest by its logits' differences, each logit by a few steps of the
    tensor cores' sum: K / 16 of 17 2^-24 of its terms' sizes, at most 60."""
    A, Bt, targets = confident(N, M, K, dtype, 14.0, 15.0)
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    tn.gemm_poll_device_status()
    Z = Bt.double() @ A.double().t()
    want = -torch.log_softmax(Z, 1)[torch.arange(N, device="cuda"), targets]
    logits = (min(K, 1024) + 15) // 16 * 17 * 2.0 ** -24 * 60 * 2
    assert bool(((loss.double() - want).abs() <= 2.0 ** -19 + want * (logits + 2.0 ** -20)).all())
    assert float((loss.double() - want).norm() / want.norm()) < 1e-3
