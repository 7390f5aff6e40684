"""The gated projections', the loss's and the 4-bit products' helpers on a stream of the
caller's: their results and workspaces are neither taken from what kernels of the current
stream still use, nor given away while those read them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_gemm_tn_gb300 as g


def randn(*shape, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def calls():
    N, M, K = 600, 640, 264                     # results of several blocks of 512 KiB
    wide, tokens, dH = randn(2 * M, K, seed=1, scale=K ** -0.5), randn(N, K, seed=2), randn(N, M, seed=3)
    experts = randn(3, 2 * M, K, seed=4, scale=K ** -0.5)
    off = torch.tensor([0, 200, 200, N], dtype=torch.int32, device="cuda")
    kept, kept_by_expert = g.tn_gated(wide, tokens, keep=True)[1], g.tn_gated(experts, tokens, off, keep=True)[1]
    vocabulary, targets = randn(9000, K, seed=5, scale=K ** -0.5), torch.arange(N, device="cuda") * 14
    lse, dloss = g.tn_cross_entropy(vocabulary, tokens, targets)[1], torch.rand(N, device="cuda")
    # rows of 263 terms: the operands go through copies in the workspace
    odd, odd_tokens = randn(2 * M, K - 1, seed=6, scale=K ** -0.5), randn(N, K - 1, seed=7)
    weights, few = randn(2048, 1024, seed=8), randn(24, 1024, seed=9)
    q, s = g.quantize_w4_rows(weights, 64)
    return {
        "tn_gated": lambda t: g.tn_gated(wide, tokens, keep=True, stream=t),
        "tn_gated by expert": lambda t: g.tn_gated(experts, tokens, off, act="gelu", stream=t),
        "tn_gated of copies": lambda t: g.tn_gated(odd, odd_tokens, stream=t),
        "tn_gated of few": lambda t: g.tn_gated(wide, tokens[:5], stream=t),
        "tn_gated_grad": lambda t: g.tn_gated_grad(wide, tokens, kept, dH, stream=t),
        "tn_gated_grad by expert": lambda t: g.tn_gated_grad(experts, tokens, kept_by_expert, dH, off, stream=t),
        "tn_cross_entropy": lambda t: g.tn_cross_entropy(vocabulary, tokens, targets, stream=t),
        "tn_cross_entropy_grad": lambda t: g.tn_cross_entropy_grad(vocabulary, tokens, targets, lse, dloss, stream=t),
        "w4_tn": lambda t: g.w4_tn(q, few, s, 64, stream=t),
        "quantize_w4_rows": lambda t: g.quantize_w4_rows(weights, 32, stream=t),
    }


NAMES = ["tn_gated", "tn_gated by expert", "tn_gated of copies", "tn_gated of few", "tn_gated_grad",
         "tn_gated_grad by expert", "tn_cross_entropy", "tn_cross_entropy_grad", "w4_tn", "quantize_w4_rows"]


def tensors(result):
    return list(result) if isinstance(result, (tuple, list)) else [result]


def same(result, want):
    return all(torch.equal(r, w) for r, w in zip(tensors(result), want))


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_results_on_another_stream(name, as_handle):
    call, side = calls()[name], torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    want = tensors(call(None))
    torch.cuda.synchronize()
    warm = call(stream)
    side.synchronize()
    assert same(warm, want)
    del warm
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # a freed block that the current stream has yet to read
    size = want[0].numel() * want[0].element_size()
    x = torch.full((size,), 77, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    y = x.clone()
    del x
    first = call(stream)
    torch.cuda.synchronize()
    assert bool((y == 77).all()) and same(first, want)
    # results that the current stream has yet to read when they are released
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    copies = [t.clone() for t in tensors(first)]
    del first
    with torch.cuda.stream(side):
        junk = [torch.full_like(w, 1) for w in want for _ in range(3)]
    torch.cuda.synchronize()
    assert same(copies, want)
    del junk
    g.gemm_poll_device_status()


def test_captured_calls_on_a_forked_stream():
    made, side = calls(), torch.cuda.Stream()
    want = {name: tensors(made[name](None)) for name in NAMES}
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for name in NAMES:
            got[name] = made[name](side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for name in got:
            for t in tensors(got[name]):
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name in got:
            assert same(got[name], want[name]), name
    g.gemm_poll_device_status()


@pytest.mark.parametrize("name", NAMES)
def test_both_bindings(name, monkeypatch):
    """The same results through ctypes as through the CPython-API binding."""
    if g.fast is None:
        pytest.skip("the CPython-API binding was not built (no Python.h)")
    call, results = calls()[name], []
    for binding in (g.fast, g.lib):
        monkeypatch.setattr(g, "calls", binding)
        results.append(tensors(call(None)))
    g.gemm_poll_device_status()
    assert same(*results)
