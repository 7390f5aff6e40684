"""Overlaps that the gradients allow, and results beside their operands in one buffer."""
import pytest
import torch

from tests.grouped_helpers import normals, offsets_of

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

DTYPES = [torch.float16, torch.bfloat16]


def gated(dtype, by_expert):
    E, T, M, K = (3 if by_expert else 1), 300, 96, 64
    A, x, dH = (normals(*s, seed=i, dtype=torch.float32).to(dtype) for i, s in enumerate(((E, 2 * M, K), (T, K), (T, M))))
    return (A if by_expert else A[0]), x, dH, offsets_of([100, 0, 200]) if by_expert else None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("by_expert", [False, True])
def test_gated_gradients_where_they_may_lie(by_expert, dtype):
    A, x, dH, off = gated(dtype, by_expert)
    _, P = tn.tn_gated(A, x, off, keep=True)
    want = tn.tn_gated_grad(A, x, P, dH, off)

    def same(got, which=(True, True)):
        tn.gemm_poll_device_status()
        for a, b, w in zip(got, want, which):
            assert (a is None and not w) or torch.equal(a, b)
    h = dH.clone()                                                 # dB in dH's memory (64 columns of 96)
    same(tn.tn_gated_grad(A, x, P, h, off, dBt=h[:, :64]))
    p = P.clone()                                                  # dA in P's
    same(tn.tn_gated_grad(A, x, p, dH, off, dA=p.view(-1).view(dtype)[: A.numel()].view(A.shape)))
    a = A.clone()                                                  # dA in A's
    same(tn.tn_gated_grad(a, x, P, dH, off, dA=a))
    y = x.clone()                                                  # dB in B's, alone
    same(tn.tn_gated_grad(A, y, P, dH, off, dBt=y, want_a=False), (False, True))
    both = torch.empty(*A.shape[:-1], 2, A.shape[-1], device="cuda", dtype=dtype)       # A's rows and dA's in turn
    both[..., 0, :] = A
    same(tn.tn_gated_grad(both[..., 0, :], x, P, dH, off, dA=both[..., 1, :]))
    wide = torch.empty(max(A.numel(), x.numel()), device="cuda", dtype=dtype)
    shared = dict(dA=wide[: A.numel()].view(A.shape), dBt=wide[: x.numel()].view(x.shape))
    for bad in (dict(dBt=x), shared):
        with pytest.raises(tn.GemmError, match="overlaps"):
            tn.tn_gated_grad(A, x, P, dH, off, **bad)


@pytest.mark.parametrize("dtype", DTYPES)
def test_loss_gradients_where_they_may_lie(dtype):
    M, N, K = 20000, 9000, 64                                      # two pieces of the vocabulary
    A, x = (normals(*s, seed=i, dtype=torch.float32).mul_(0.3).to(dtype) for i, s in enumerate(((M, K), (N, K))))
    targets = torch.randint(0, M, (N,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    dloss = torch.ones(N, device="cuda")
    _, lse = tn.tn_cross_entropy(A, x, targets)
    want = tn.tn_cross_entropy_grad(A, x, targets, lse, dloss)
    a = A.clone()
    got = tn.tn_cross_entropy_grad(a, x, targets, lse, dloss, dA=a)
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(got[1], want[1])
    y = x.clone()
    _, got = tn.tn_cross_entropy_grad(A, y, targets, lse, dloss, dBt=y, want_a=False)
    assert torch.equal(got, want[1])
    tn.gemm_poll_device_status()
    with pytest.raises(tn.GemmError, match="overlaps"):
        tn.tn_cross_entropy_grad(A, x, targets, lse, dloss, dBt=x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_results_beside_operands(dtype):
    A, x, _, off = gated(dtype, True)
    want = tn.tn_gated(A, x, off)
    row = torch.full((300, 64 + 96), 7.0, device="cuda", dtype=dtype)
    row[:, :64] = x
    tn.tn_gated(A, row[:, :64], off, H=row[:, 64:])
    assert torch.equal(row[:, 64:], want) and torch.equal(row[:, :64], x)
    with pytest.raises(tn.GemmError, match="overlaps"):
        tn.tn_gated(A, row[:, 64:128], off, H=row[:, 64:])
