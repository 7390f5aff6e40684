"""The fp16 gated gradients' factors and the loss gradient's segments as a program meets them: in two graphs at once beside eager
calls, from threads, and through the bounded waits."""
import threading

import pytest
import torch

from tests.grouped_helpers import normals, offsets_of

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")


def layer(seed, power, E=4, T=300, K=1152, M=192, V=700):
    """Expert layer and head in fp16, gradients of size 2^power: each layer needs a factor of its own; sums of two segments."""
    up = normals(E, 2 * M, K, seed=seed, dtype=torch.float32).mul_(K ** -0.5).half()
    head = normals(V, K, seed=seed + 1, dtype=torch.float32).mul_(2 * K ** -0.5).half()
    x = normals(T, K, seed=seed + 2, dtype=torch.float16)
    dH = (normals(T, M, seed=seed + 3, dtype=torch.float32) * 2.0 ** power).half()
    targets = torch.randint(0, V, (T,), generator=torch.Generator(device="cuda").manual_seed(seed + 4), device="cuda")
    return up, head, x, dH, offsets_of([T // 3, 0, T // 2, T - T // 3 - T // 2]), targets


def step(up, head, x, dH, offsets, targets):
    _, P = tn.tn_gated(up, x, offsets, keep=True)
    d_up, dx = tn.tn_gated_grad(up, x, P, dH, offsets)
    d_one, dx_one = tn.tn_gated_grad(up[0], x, P, dH)              # (the same tokens through one expert)
    _, lse = tn.tn_cross_entropy(head, x, targets)
    d_head, dy = tn.tn_cross_entropy_grad(head, x, targets, lse, torch.ones_like(lse))
    return d_up, dx, d_one, dx_one, d_head, dy


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_graphs_beside_eager_calls():
    parts = [layer(1, -18), layer(20, 3)]
    want = [step(*p) for p in parts]
    assert all(bool(torch.isfinite(t).all()) for w in want for t in w)
    graphs = []
    for p in parts:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(*p)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = step(*p)
        graphs.append((g, s, out))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, out in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager = step(*parts[0])
        torch.cuda.synchronize()
        for (_, _, out), ref in zip(graphs, want):
            same(out, ref)
        same(eager, want[0])
    tn.gemm_poll_device_status()


def test_several_threads():
    parts = [layer(s, p) for s, p in ((1, -19), (11, 0), (21, 6), (31, -10))]
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
        same(a, b)


def loss_gradients(N):
    A, x = normals(9000, 3000, seed=1, dtype=torch.bfloat16).mul_(0.02), normals(N, 3000, seed=2, dtype=torch.bfloat16)
    return tn.tn_cross_entropy_grad(A, x, torch.zeros(N, dtype=torch.int64, device="cuda"), torch.full((N,), 9.0, device="cuda"),
                                    torch.ones(N, device="cuda"))


def gated_gradients(T):
    up, _, x, dH, offsets, _ = layer(5, -12, T=T, K=512)
    P = normals(T, 384, seed=9, dtype=torch.float32)
    return tn.tn_gated_grad(up, x, P, dH, offsets)


CALLS = {"loss gradients, pairs, segments": lambda: loss_gradients(600), "loss gradients, one CTA a tile": lambda: loss_gradients(20),
         "gated gradients by expert, one CTA a tile": lambda: gated_gradients(90), "gated gradients by expert, pairs": lambda: gated_gradients(3000)}


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("name", list(CALLS))
def test_a_wait_that_runs_out(name, mode):
    """A stalled MMA thread or producer: reported, and the next call is right."""
    want = CALLS[name]()
    tn.gemm_poll_device_status()
    tn.gemm_set_wait_limit_ns(50_000_000)
    tn.gemm_debug_inject_stall(mode)
    try:
        CALLS[name]()
        with pytest.raises(tn.GemmError) as err:
            tn.gemm_poll_device_status()
        assert err.value.status == tn.GEMM_ERR_TIMEOUT
    finally:
        tn.gemm_debug_inject_stall(0)
        tn.gemm_set_wait_limit_ns(0)
    tn.gemm_poll_device_status()
    again = CALLS[name]()
    tn.gemm_poll_device_status()
    same(again, want)
