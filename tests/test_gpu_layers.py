"""The gated projections, the vocabulary's loss and the 4-bit products as a program uses them: together, from
several threads, in two graphs at once, on streams, through the bounded waits, and at sizes past 32 bits."""
import threading

import pytest
import torch

from tests.grouped_helpers import HALF_STEP, normals, offsets_of
from tests.sink_helpers import assert_within, gated64, gated_bound, loss64, sum_error

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")


def model(dtype, E=4, T=300, K=128, M=192, V=1000, seed=1):
    up = normals(E, 2 * M, K, seed=seed, dtype=torch.float32).mul_(K ** -0.5).to(dtype)
    down = normals(E, K, M, seed=seed + 1, dtype=torch.float32).mul_(M ** -0.5).to(dtype)
    head = normals(V, K, seed=seed + 2, dtype=torch.float32).mul_(2 * K ** -0.5).to(dtype)
    x = normals(T, K, seed=seed + 3, dtype=dtype)
    counts = [T // 3, 0, T // 2, T - T // 3 - T // 2]
    targets = torch.randint(0, V, (T,), generator=torch.Generator(device="cuda").manual_seed(seed + 4), device="cuda")
    targets[::7] = -100
    return up, down, head, x, offsets_of(counts), targets


def step(up, down, head, x, offsets, targets):
    """One training step of an expert layer and a head: every product the library's."""
    H, P = tn.tn_gated(up, x, offsets, keep=True)
    y = tn.tn_grouped(down, H, offsets)
    loss, lse = tn.tn_cross_entropy(head, y, targets)
    valid = targets >= 0
    dloss = valid.float() / valid.sum()
    d_head, dy = tn.tn_cross_entropy_grad(head, y, targets, lse, dloss)
    dH = tn.tn_grouped_grad_b(down, dy, offsets)
    d_down = tn.tn_grouped_grad_a(dy, H, offsets)
    d_up, dx = tn.tn_gated_grad(up, x, P, dH, offsets)
    return (loss * dloss).sum(), d_up, d_down, d_head, dx


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_training_step(dtype):
    """Against the same step in 64 bits by autograd.  Every gradient passes four products and roundings to 16 bits in
    turn, each off by half a step of random sign: within 8 half steps in the 2-norm."""
    parts = model(dtype)
    got = step(*parts)
    tn.gemm_poll_device_status()
    up, down, head, x, offsets, targets = parts
    bounds = offsets.tolist()
    leaves = [t.double().requires_grad_() for t in (up, down, head, x)]
    u, d, h, xx = leaves
    M = u.shape[1] // 2
    rows = []
    for e in range(len(bounds) - 1):
        p = xx[bounds[e]:bounds[e + 1]] @ u[e].t()
        rows.append((torch.nn.functional.silu(p[:, :M]) * p[:, M:]) @ d[e].t())
    loss = torch.nn.functional.cross_entropy(torch.cat(rows) @ h.t(), targets)
    loss.backward()
    loss = float(loss.detach())
    assert abs(float(got[0]) - loss) < 8 * HALF_STEP[dtype] * loss
    for g, leaf in zip(got[1:], leaves):
        assert float((g.double() - leaf.grad).norm() / leaf.grad.norm()) < 8 * HALF_STEP[dtype]


def test_a_training_step_in_graphs_beside_an_eager_one():
    """Two captured steps replayed on two streams at once, each with its own workspaces, while eager steps run."""
    first, second = model(torch.bfloat16, seed=1), model(torch.bfloat16, seed=20)
    want = [step(*first), step(*second)]
    graphs = []
    for parts in (first, second):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(*parts)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = step(*parts)
        graphs.append((g, s, out))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, out in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager = step(*first)
        torch.cuda.synchronize()
        for (_, _, out), ref in zip(graphs, want):
            for a, b in zip(out, ref):
                assert torch.equal(a, b)
        for a, b in zip(eager, want[0]):
            assert torch.equal(a, b)
    tn.gemm_poll_device_status()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_decode_step_in_four_bits(dtype):
    """A dense layer and head held in 4 bits, one to forty tokens: each product against its own weights in 64 bits."""
    K, M, V, group = 256, 320, 9000, 64
    up, down, head = (normals(*s, seed=i, dtype=torch.float32).mul_(s[1] ** -0.5).to(dtype) for i, s in enumerate(((2 * M, K), (K, M), (V, K))))
    qs = [tn.quantize_w4_rows(w, group) for w in (up, down, head)]
    for T in (1, 3, 8, 9, 16, 33, 40):
        x = normals(T, K, seed=T, dtype=dtype)
        for (q, s), w, a in zip(qs, (up, down, head), (x, None, x)):
            a = normals(T, w.shape[1], seed=T + 1, dtype=dtype) if a is None else a
            codes = q.contiguous().view(torch.int8)
            codes = torch.stack(((codes << 4) >> 4, codes >> 4), -1).flatten(1).double()
            W = codes * s.double().repeat_interleave(group, 1)[:, : w.shape[1]]
            assert float((W - w.double()).abs().max()) <= float(w.double().abs().max()) / 12
            got = tn.w4_tn(q, a, s, group)
            ref, size = a.double() @ W.t(), a.double().abs() @ W.abs().t()
            assert_within(got, ref, HALF_STEP[dtype] * 1.01 * ref.abs() + sum_error(size, group) + 64 * 2.0 ** -24 * size + torch.finfo(dtype).tiny)


def test_several_threads_on_their_streams():
    parts = [model(torch.bfloat16, seed=s) for s in (1, 11, 21, 31)]
    want = [step(*p) for p in parts]
    torch.cuda.synchronize()
    got, errors = [None] * len(parts), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[i] = step(*parts[i])
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(parts))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


CALLS = {
    "gated, one CTA a tile": lambda: tn.tn_gated(normals(64, 512, seed=1, dtype=torch.bfloat16), normals(40, 512, seed=2, dtype=torch.bfloat16)),
    "gated, pairs": lambda: tn.tn_gated(normals(4096, 512, seed=1, dtype=torch.bfloat16), normals(1000, 512, seed=2, dtype=torch.bfloat16)),
    "loss, one CTA a tile": lambda: tn.tn_cross_entropy(normals(700, 4096, seed=1, dtype=torch.bfloat16), normals(10, 4096, seed=2, dtype=torch.bfloat16),
                                                        torch.zeros(10, dtype=torch.int64, device="cuda")),
    "loss, pairs, segments": lambda: tn.tn_cross_entropy(normals(20000, 3000, seed=1, dtype=torch.bfloat16).mul_(0.02), normals(600, 3000, seed=2, dtype=torch.bfloat16),
                                                         torch.zeros(600, dtype=torch.int64, device="cuda")),
    "loss gradients": lambda: tn.tn_cross_entropy_grad(normals(9000, 512, seed=1, dtype=torch.bfloat16).mul_(0.02), normals(600, 512, seed=2, dtype=torch.bfloat16),
                                                       torch.zeros(600, dtype=torch.int64, device="cuda"), torch.full((600,), 9.0, device="cuda"),
                                                       torch.ones(600, device="cuda")),
}


@pytest.mark.parametrize("mode", [1, 2, 3])
@pytest.mark.parametrize("name", list(CALLS))
def test_a_wait_that_runs_out(name, mode):
    """A stalled MMA thread or producer: reported, and the next call is right.  (Mode 3, the second CTA's producer, has
    nothing to stall where one CTA takes a tile's whole sum: 8 blocks are too few to split.)"""
    want = CALLS[name]()
    tn.gemm_poll_device_status()
    tn.gemm_set_wait_limit_ns(50_000_000)
    tn.gemm_debug_inject_stall(mode)
    try:
        CALLS[name]()
        if mode != 3 or name != "gated, one CTA a tile":
            with pytest.raises(tn.GemmError) as err:
                tn.gemm_poll_device_status()
            assert err.value.status == tn.GEMM_ERR_TIMEOUT
    finally:
        tn.gemm_debug_inject_stall(0)
        tn.gemm_set_wait_limit_ns(0)
    tn.gemm_poll_device_status()
    again = CALLS[name]()
    tn.gemm_poll_device_status()
    for a, b in zip(want if isinstance(want, tuple) else (want,), again if isinstance(again, tuple) else (again,)):
        assert torch.equal(a, b)


def test_results_and_codes_past_32_bits():
    """More than 2^31 bytes of products, of codes and of logits' gradients: sampled rows."""
    T, M, K = 70000, 16384, 16                                  # P: 70000 x 32768 floats, 2^33 bytes
    A, Bt = normals(2 * M, K, seed=1, dtype=torch.bfloat16), normals(T, K, seed=2, dtype=torch.bfloat16)
    H, P = tn.tn_gated(A, Bt, keep=True)
    dH = torch.zeros(T, M, device="cuda", dtype=torch.bfloat16)
    at = torch.tensor([0, 1, 35000, T - 2, T - 1], device="cuda")
    dH[at] = 1
    dA, dB = tn.tn_gated_grad(A, Bt, P, dH)
    tn.gemm_poll_device_status()
    # (five rows alone take another kernel, whose sums round elsewhere: both against 64 bits)
    H64, P64, off = gated64(A[None], Bt[at], [0, 5], "silu")
    few, kept = tn.tn_gated(A, Bt[at].contiguous(), keep=True)
    for h, p in ((H[at], P[at]), (few, kept)):
        assert_within(p, P64, off + 2.0 ** -126, "P")
        assert_within(h, H64, gated_bound(P64, off, "silu", torch.bfloat16), "H")
    dA2, dB2 = tn.tn_gated_grad(A, Bt[at].contiguous(), P[at], dH[at].contiguous())
    # the same five rows: the sums over 2 M in other parts, those over the rows among zeros
    assert float((dB[at].double() - dB2.double()).norm() / dB2.double().norm()) < 2.0 ** -7
    assert float((dA.double() - dA2.double()).norm() / dA2.double().norm()) < 2.0 ** -7
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not bool(dB[rest].any())
    del P, H, dH
    torch.cuda.empty_cache()
    M, K = 9 << 16, 8192                                         # 589824 rows of 4096 bytes of codes: past 2^31
    A = torch.randint(0, 256, (M, K // 2), device="cuda", dtype=torch.uint8)
    scale = torch.ones(M, K // 128, device="cuda", dtype=torch.bfloat16)
    x = (torch.rand(2, K, device="cuda") < 0.01).to(torch.bfloat16)
    C = tn.w4_tn(A, x, scale, 128)
    at = torch.tensor([0, 5, M // 2, M - 1], device="cuda")
    codes = A[at].view(torch.int8)
    codes = torch.stack(((codes << 4) >> 4, codes >> 4), -1).flatten(1).double()
    assert torch.equal(C[:, at].double(), (x.double() @ codes.t()).to(torch.bfloat16).double())


def test_many_classes_and_many_tokens():
    """A vocabulary of a million and a batch of a hundred thousand tokens: sampled tokens."""
    for N, M, K in ((40, 1_000_003, 64), (100_000, 2000, 64)):
        A, Bt = normals(M, K, seed=1, dtype=torch.float32).mul_(0.3).half(), normals(N, K, seed=2, dtype=torch.float16)
        targets = torch.randint(0, M, (N,), device="cuda")
        loss, lse = tn.tn_cross_entropy(A, Bt, targets)
        at = torch.arange(0, N, max(1, N // 40), device="cuda")
        ref, lse_ref, off, off_lse, _, _ = loss64(A, Bt[at], targets[at])
        assert_within(loss[at], ref, off, "loss")
        assert_within(lse[at], lse_ref, off_lse, "lse")
        dA, dB = tn.tn_cross_entropy_grad(A, Bt, targets, lse, torch.ones(N, device="cuda"))
        tn.gemm_poll_device_status()
        p = torch.softmax(Bt[at].double() @ A.double().t(), 1)
        p[torch.arange(len(at), device="cuda"), targets[at]] -= 1
        want = p @ A.double()
        assert float((dB[at].double() - want).norm() / want.norm()) < 2 * HALF_STEP[torch.float16]
        # sums over the tokens: each column of d adds up to the softmax's mass less the targets'
        assert bool(torch.isfinite(dA).all())
