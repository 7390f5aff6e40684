"""The loss over large vocabularies, tightly: no class is missing wherever it stands, and the weight gradient's rows are in their
places on both sides of every border of pieces."""
import pytest
import torch

from tests.grouped_helpers import normals

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

DTYPES = [torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [40, 300])
@pytest.mark.parametrize("M", [32003, 70001, 131071, 1000003])
def test_large_vocabularies_lose_nothing(M, N, dtype):
    """A class is 1e-5 to 1e-6 of the mass here, a block of 32 some 1e-3 to 3e-5.  The sum of exponentials goes through at most
    600 additions (a thread of the join adds its share of the pieces, 1000003 / 32 / 64 at most, then a tree), each rounded by at
    most 2^-24 of itself and of random sign (25 steps in all); the exponentials are 2^-22 off, of random sign too.  So the lse, 11 to
    15, is within 2^-20 of itself in the norm, where a block missing in every token would be 2^-13 to 2^-19 of it."""
    K = 64
    A = normals(M, K, seed=M, dtype=torch.float32).mul_(K ** -0.5).to(dtype)
    Bt = normals(N, K, seed=N, dtype=dtype)
    targets = torch.randint(0, M, (N,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    loss, lse = tn.tn_cross_entropy(A, Bt, targets)
    tn.gemm_poll_device_status()
    want = torch.cat([torch.logsumexp(x.double() @ A.double().t(), 1) for x in Bt.split(32)])
    ref = want - (A[targets].double() * Bt.double()).sum(1)
    assert float((lse.double() - want).norm() / want.norm()) < 2.0 ** -20
    assert float((loss.double() - ref).norm() / ref.norm()) < 2.0 ** -18


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1000, 4099, 32003, 70001, 131071])
def test_all_mass_in_one_class(M, dtype):
    """Each token has its mass in a class of its own (a logit of 30 among zeros): the first, the last, those of the last block of 32,
    and both sides of every border at which the join's slices may begin.  Without that class the lse would be log(M - 1)."""
    pieces = -(-M // 32)
    at = {0, 31, 32, M - 1, M - 2, M // 32 * 32 - 1, M // 32 * 32 % M}
    for slices in (16, 32, 64, 128, 256, 512):
        per = -(-pieces // slices)
        for k in (1, 2, slices // 2, slices - 1):
            at |= {32 * per * k - 1, 32 * per * k}
    at = sorted(c for c in at if 0 <= c < M)
    for N in (len(at), 300):                                       # (also enough of them for other slices)
        classes = torch.tensor((at * (300 // len(at) + 1))[:N], device="cuda")
        K = 64
        A = torch.zeros(M, K, device="cuda")
        Bt = torch.zeros(N, K, device="cuda")
        # token n has column n % 64 of a group of 64 tokens
        loss = torch.empty(N, device="cuda")
        lse = torch.empty(N, device="cuda")
        for i in range(0, N, K):
            own = classes[i:i + K]
            A.zero_()
            A[own, torch.arange(len(own), device="cuda")] = 30.0
            Bt.zero_()
            Bt[torch.arange(i, i + len(own)), torch.arange(len(own), device="cuda")] = 1.0
            got = tn.tn_cross_entropy(A.to(dtype), Bt.to(dtype), classes)
            loss[i:i + K], lse[i:i + K] = got[0][i:i + K], got[1][i:i + K]
        tn.gemm_poll_device_status()
        want = 30 + torch.log1p(torch.tensor((M - 1) * 2.718281828459045 ** -30, dtype=torch.float64))
        assert float((lse.double().cpu() - want).abs().max()) <= 2.0 ** -19
        assert float(loss.abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("N,M", [(40, 1_000_003), (100_000, 2000), (20_000, 20_011), (4096, 70_001)])
def test_sampled_rows_of_the_weight_gradient(N, M):
    """The first rows and the last, and both sides of every border of 256 classes (pieces begin at some of them), against 64 bits.
    d is rounded to 2^-11 of itself, and the result; both of random sign."""
    K, dtype = 64, torch.float16
    A, Bt = normals(M, K, seed=1, dtype=torch.float32).mul_(0.3).to(dtype), normals(N, K, seed=2, dtype=dtype)
    targets = torch.randint(0, M, (N,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    targets[::9] = -1
    _, lse = tn.tn_cross_entropy(A, Bt, targets)
    scale = 4.0 * M / N ** 0.5                                     # results of size one
    dloss = torch.full((N,), scale, device="cuda")
    dA, _ = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss, want_b=False)
    both, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, dloss)
    tn.gemm_poll_device_status()
    assert torch.equal(dA, both)
    edges = torch.arange(256, M, 256, device="cuda")
    rows = torch.cat((torch.arange(5, device="cuda"), edges - 1, edges, torch.arange(M - 5, M, device="cuda"))).unique()
    if len(rows) > 1200:
        rows = rows[torch.linspace(0, len(rows) - 1, 1200, device="cuda").long()]
    exact = torch.cat([torch.logsumexp(x.double() @ A.double().t(), 1) for x in Bt.split(max(1, 100_000_000 // M))])
    d = torch.exp(Bt.double() @ A[rows].double().t() - exact[:, None])
    d -= (targets[:, None] == rows[None, :]).double()
    d *= (targets >= 0).double()[:, None] * scale
    want = d.t() @ Bt.double()
    err, size = (dA[rows].double() - want).norm(dim=1), want.norm(dim=1)
    assert float(size.min()) > 0
    assert float((err / size).max()) < 2.0 ** -9, int((err / size).argmax())
    assert float(err.norm() / size.norm()) < 2.0 ** -11
