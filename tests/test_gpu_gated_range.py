"""The gated projections' gradients far from one: dH and P small and large, in fp16 above all, whose numbers
end at 2^-24 and 65504 while the gradients' sums are FP32."""
import pytest
import torch

from tests.grouped_helpers import HALF_STEP, normals, offsets_of
from tests.sink_helpers import act64, act_rel, assert_within, slope_error, sum_error

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

ACTS = ["silu", "gelu", "gelu_tanh"]
HALF = 2.0 ** -11


def reference(A, Bt, P, dH, bounds, act, dtype=torch.float16):
    """(dA, dB, what each may be off): dP rounded once, relative to itself, and not below 2^-29 of the largest (fp16: the largest is at
    least 2^4 when it is rounded, and a step is 2^-24 there; bf16 has FP32's range); FP32 sums; the results rounded once."""
    E, rows, K = A.shape
    M = rows // 2
    half = HALF_STEP[dtype]
    P, dH = P.double(), dH.double()
    g, u = P[:, :M], P[:, M:]
    a, s = act64(g, act)
    dP = torch.cat((dH * u * s, dH * a), 1)
    off = torch.cat(((dH * u).abs() * (slope_error(g) + 2.0 ** -22 * s.abs()), dH.abs() * a.abs() * (act_rel(g) + 2.0 ** -22)), 1)
    inside = dP[bounds[0]:bounds[-1]].abs()
    largest = float(inside[torch.isfinite(inside)].max()) if inside.numel() else 0.0
    off = off + half * (dP.abs() + off) + largest * 2.0 ** -29
    dA, eA = torch.zeros(A.shape, dtype=torch.float64, device="cuda"), torch.zeros(A.shape, dtype=torch.float64, device="cuda")
    dB = torch.full((Bt.shape[0], K), float("nan"), dtype=torch.float64, device="cuda")
    eB = torch.zeros_like(dB)
    for e in range(E):
        r = slice(bounds[e], bounds[e + 1])
        d, o, x, W = dP[r], off[r], Bt[r].double(), A[e].double()
        dA[e], dB[r] = d.t() @ x, d @ W
        eA[e] = o.t() @ x.abs() + sum_error((d.abs() + o).t() @ x.abs(), d.shape[0])
        eB[r] = o @ W.abs() + sum_error((d.abs() + o) @ W.abs(), rows)
    least = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133       # half of the smallest step
    return dA, dB, half * dA.abs() + 1.01 * eA + least, half * dB.abs() + 1.01 * eB + least


def operands(counts, M, K, dtype, seed=1, lead=0, rest=0):
    E, T = len(counts), lead + sum(counts) + rest
    A = normals(E, 2 * M, K, seed=seed, dtype=torch.float32).mul_(K ** -0.5).to(dtype)
    return A, normals(T, K, seed=seed + 1, dtype=dtype), normals(T, M, seed=seed + 2, dtype=torch.float32)


CASES = [([1024], 256, 256, True), ([300], 129, 72, True), ([70, 0, 200], 96, 136, False), ([40, 90, 1], 100, 64, False), ([600, 700], 512, 64, False),
         ([9], 1000, 264, True), ([3, 0, 5], 28, 64, False)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,M,K,dense", CASES)
@pytest.mark.parametrize("power", [-20, -18, -14, -10, 0, 10])
def test_small_and_large_gradients(power, counts, M, K, dense, act):
    """dH of any size that fp16 holds: dA and dB as near as their own roundings and dP's."""
    A, Bt, dH = operands(counts, M, K, torch.float16)
    dH = (dH * 2.0 ** power).half()
    offsets = offsets_of(counts)
    W, off = (A[0], None) if dense else (A, offsets)
    _, P = tn.tn_gated(W, Bt, off, act=act, keep=True)
    if power == 10:
        Bt *= 2.0 ** -8                                            # results that fp16 holds
    dA, dB = tn.tn_gated_grad(W, Bt, P, dH, off, act=act)
    tn.gemm_poll_device_status()
    rA, rB, eA, eB = reference(A, Bt, P, dH, offsets.tolist(), act)
    for got, ref, bound, name in ((dA.view(A.shape), rA, eA, "dA"), (dB, rB, eB, "dB")):
        assert_within(got, ref, bound, name)
        # two roundings of random sign, each 2^-11 of the number at most: well within 2^-11 in the norm (numbers below the
        # type's normal ones, which lose bits as results, left out)
        at = ref.abs() >= 2.0 ** -14
        if int(at.sum()) > 1000:
            assert float((got.double() - ref)[at].norm() / ref[at].norm()) < HALF


@pytest.mark.parametrize("counts,M,K,dense", CASES)
@pytest.mark.parametrize("dh,size", [(2000.0, 40.0), (1.0, 1e5), (2.0 ** -14, 3e8), (65504.0, 1e-3), (1.0, 1e-6), (2.0 ** -10, 2.0 ** -14),
                                     (1.0, 1e30)])
def test_products_of_any_size(dh, size, counts, M, K, dense):
    """dH times P beyond 65504 and far below 2^-24, the sums brought back into fp16's range by B and A."""
    E, T = len(counts), sum(counts)
    _, _, dH = operands(counts, M, K, torch.float16)
    dH = (dH.clamp_(-1, 1) * dh).half()
    P = normals(T, 2 * M, seed=9, dtype=torch.float32)
    P[:, M:] *= size                                               # the gates stay of size one, the up products do not
    # (the gate's gradients are dh size, the up rows' dh: results for the larger of the two)
    back = min(1.0, 256 / (dh * max(size, 1.0)))
    back = max(back, 2.0 ** -20)
    Bt = (normals(T, K, seed=5, dtype=torch.float32) * back).half()
    A = (normals(E, 2 * M, K, seed=6, dtype=torch.float32) * back).half()
    offsets = offsets_of(counts)
    W, off = (A[0], None) if dense else (A, offsets)
    dA, dB = tn.tn_gated_grad(W, Bt, P, dH, off)
    tn.gemm_poll_device_status()
    rA, rB, eA, eB = reference(A, Bt, P, dH, offsets.tolist(), "silu")
    for got, ref, bound, name in ((dA.view(A.shape), rA, eA, "dA"), (dB, rB, eB, "dB")):
        fits = ref.abs() < 60000                                   # (what a result of fp16 can hold)
        assert_within(torch.where(fits, got.double(), 0.0), torch.where(fits, ref, 0.0), bound, name)
        assert bool((torch.isinf(got) | (got.abs() > 50000))[ref.abs() > 66000].all())


@pytest.mark.parametrize("dense", [True, False])
def test_all_gradients_zero(dense):
    counts = [100] if dense else [60, 0, 40]
    A, Bt, dH = operands(counts, 64, 72, torch.float16)
    off = None if dense else offsets_of(counts)
    W = A[0] if dense else A
    _, P = tn.tn_gated(W, Bt, off, keep=True)
    for h, p in ((torch.zeros_like(dH).half(), P), (dH.half(), torch.zeros_like(P))):
        dA, dB = tn.tn_gated_grad(W, Bt, p, h, off)
        assert not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("power", [-18, 0])
def test_what_is_not_finite_stays_in_its_token(power, bad):
    counts, M, K = [70, 130], 64, 72
    A, Bt, dH = operands(counts, M, K, torch.float16)
    dH = (dH * 2.0 ** power).half()
    offsets = offsets_of(counts)
    _, P = tn.tn_gated(A, Bt, offsets, keep=True)
    clean = dH.clone()
    clean[7] = 0
    _, rB, _, eB = reference(A, Bt, P, clean, offsets.tolist(), "silu")
    dH[7, 3] = bad
    dA, dB = tn.tn_gated_grad(A, Bt, P, dH, offsets)
    others = torch.arange(200, device="cuda") != 7
    assert_within(dB[others], rB[others], eB[others], "dB")
    assert not bool(torch.isfinite(dB[7]).any()) and bool(torch.isfinite(dA[1]).all())
    bad_rows = ~torch.isfinite(dA[0]).all(1)
    assert bad_rows.nonzero().flatten().tolist() == [3, M + 3]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_of_no_expert_decide_nothing(dtype):
    """Large numbers in rows that belong to no expert leave every bit of the results as it is."""
    counts, M, K, lead, rest = [40, 0, 90], 96, 64, 5, 9
    A, Bt, dH = operands(counts, M, K, dtype, lead=lead, rest=rest)
    dH = (dH * 2.0 ** -16).to(dtype)
    offsets = offsets_of(counts, lead)
    T = Bt.shape[0]
    P = torch.zeros(T, 2 * M, device="cuda")
    tn.tn_gated(A, Bt, offsets, P=P)
    rows = slice(lead, T - rest)
    dA, dB = tn.tn_gated_grad(A, Bt, P, dH, offsets)
    for t in (dH, P):
        t[:lead] = 60000.0
        t[T - rest:] = -60000.0
    dA2, dB2 = tn.tn_gated_grad(A, Bt, P, dH, offsets)
    assert torch.equal(dA, dA2) and torch.equal(dB[rows], dB2[rows])
    rA, rB, eA, eB = reference(A, Bt, P, dH, offsets.tolist(), "silu", dtype)
    assert_within(dA, rA, eA, "dA")
    assert_within(dB, rB, eB, "dB")


@pytest.mark.parametrize("M", [1, 4, 28, 29, 31, 32, 60, 61, 64, 96])
@pytest.mark.parametrize("T", [1, 2, 7, 305, 700])
def test_rows_that_end_anywhere(T, M):
    """2 M on both sides of whole 16-byte units and of 64 elements, more and fewer rows than two CTAs an SM; a workspace of NaN."""
    A, Bt, dH = operands([T], M, 40, torch.float16)
    dH = (dH * 2.0 ** -17).half()
    _, P = tn.tn_gated(A[0], Bt, keep=True)
    dA, dB = torch.empty_like(A[0]), torch.empty_like(Bt)
    n = tn.gemm_gated_workspace(1, 1, 1, M, 40, T, A, 40, 0, Bt, 40)
    ws = torch.full((n // 2 + 512,), float("nan"), device="cuda", dtype=torch.float16)
    base = -ws.data_ptr() % 256 // 2
    tn.gemm_tn_gated_grad(tn.GEMM_IN_F16, tn.GEMM_ACT_SILU, 1, M, 40, T, A, 40, 0, Bt, 40, None, P, 2 * M, dH, M, dA, 40, 0, dB, 40,
                          ws.data_ptr() + 2 * base, n)
    tn.gemm_poll_device_status()
    rA, rB, eA, eB = reference(A, Bt, P, dH, [0, T], "silu")
    assert_within(dA[None], rA, eA, "dA")
    assert_within(dB, rB, eB, "dB")
    assert bool(torch.isnan(ws[base + n // 2:]).all()) and bool(torch.isnan(ws[:base]).all())


def test_captured_and_replayed_with_other_sizes():
    """The factors are taken anew at each replay: dH and P of other sizes than at capture."""
    A, Bt, dH = operands([200], 64, 128, torch.float16)
    dH = dH.half()
    _, P = tn.tn_gated(A[0], Bt, keep=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tn.tn_gated_grad(A[0], Bt, P, dH)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dA, dB = tn.tn_gated_grad(A[0], Bt, P, dH)
    first = dH.clone()
    for power, size in ((-18, 1.0), (0, 3000.0), (4, 1e-4), (0, 1.0)):
        dH.copy_(first * 2.0 ** power)
        P.copy_(normals(200, 128, seed=7, dtype=torch.float32) * size)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = tn.tn_gated_grad(A[0], Bt, P, dH)
        assert torch.equal(dA, want[0]) and torch.equal(dB, want[1])
