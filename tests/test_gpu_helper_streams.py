"""The helpers' results on a stream of the caller's: their memory is neither taken from
what kernels of the current stream still use, nor given away while those read it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_gemm_tn_gb300 as g

N = 1024            # results of 2 MiB


def ints(*shape, seed, dtype, top=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0 if dtype is torch.uint8 else -top, top + 1, shape, generator=gen, device="cuda").to(dtype)


def calls():
    f16, i8, u8 = torch.float16, torch.int8, torch.uint8
    A, B = ints(N, 64, seed=1, dtype=f16), ints(N, 64, seed=2, dtype=f16)
    experts, off = ints(2, N, 64, seed=3, dtype=f16), torch.tensor([0, 400, N], dtype=torch.int32, device="cuda")
    dC, wide = ints(N, N, seed=4, dtype=f16), ints(2, 64, N, seed=5, dtype=f16)
    qa, qb, q3 = ints(N, 64, seed=6, dtype=i8), ints(N, 64, seed=7, dtype=i8), ints(2, N, 64, seed=8, dtype=i8)
    ones, ones2, unit = torch.ones(N, device="cuda"), torch.ones(2, N, device="cuda"), torch.ones(1, device="cuda")
    ea, eb = ints(N, 64, seed=9, dtype=u8, top=80), ints(N, 64, seed=10, dtype=u8, top=80)
    x = torch.randn(N * 2, N, device="cuda").to(f16)
    narrow, rows = ints(N, 512, seed=11, dtype=f16), ints(N, 64, seed=12, dtype=f16)
    return {
        "f16_tn": lambda s: g.f16_tn(A, B, stream=s),
        "f16_tn_softmax_stats": lambda s: g.f16_tn_softmax_stats(A, B, 0.125, stream=s),
        "f8e4m3_tn": lambda s: g.f8e4m3_tn(ea, eb, 1.0, 0.5, stream=s),
        "f8e4m3_tn_dscale": lambda s: g.f8e4m3_tn_dscale(ea, eb, unit, unit, stream=s),
        "quantize_e4m3": lambda s: g.quantize_e4m3(x, stream=s),
        "tn_grouped": lambda s: g.tn_grouped(experts, B, off, stream=s),
        "tn_grouped_grad_b": lambda s: g.tn_grouped_grad_b(wide, rows, off, stream=s),
        "tn_grouped_grad_a": lambda s: g.tn_grouped_grad_a(dC, narrow, off, stream=s),
        "i8_tn": lambda s: g.i8_tn(qa, qb, ones, ones, stream=s),
        "i8_tn_grouped": lambda s: g.i8_tn_grouped(q3, qb, ones2, ones, off, stream=s),
        "quantize_i8_rows": lambda s: g.quantize_i8_rows(x, stream=s),
    }


NAMES = ["f16_tn", "f16_tn_softmax_stats", "f8e4m3_tn", "f8e4m3_tn_dscale", "quantize_e4m3", "tn_grouped",
         "tn_grouped_grad_b", "tn_grouped_grad_a", "i8_tn", "i8_tn_grouped", "quantize_i8_rows"]


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
    torch.cuda._sleep(100_000_000)
    y = x.clone()
    del x
    first = call(stream)
    torch.cuda.synchronize()
    assert bool((y == 77).all()) and same(first, want)
    # a result that the current stream has yet to read when it is released
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copies = [t.clone() for t in tensors(first)]
    del first
    with torch.cuda.stream(side):
        junk = [torch.full_like(w, 1) for w in want for _ in range(3)]
    torch.cuda.synchronize()
    assert same(copies, want)
    del junk
    g.gemm_poll_device_status()


def test_a_captured_call_on_a_forked_stream():
    """The same calls with a stream argument inside a graph's capture, replayed."""
    made, side = calls(), torch.cuda.Stream()
    want = {name: tensors(made[name](None)) for name in NAMES}
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for name in NAMES[5:]:
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
