"""8-bit integer products and the row quantiser on the GPU, against 64-bit forms."""
import pytest
import torch

from tests.grouped_helpers import HALF_STEP, offsets_of, padded

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_gemm_tn_gb300 as g

TYPES = [torch.float16, torch.bfloat16]


def codes(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=gen, device="cuda").to(torch.int8)


def scales(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (0.5 + torch.rand(*shape, generator=gen, device="cuda")) * 2.0 ** -10


def assert_scaled(got, sums, sa, sb, terms, dtype):
    """got against sums * sa * sb: half a step of the type, one FP32 rounding for
    each of the two scalings, and the FP32 sum's own (as in assert_near; sums of
    magnitudes at most terms * 2^14)."""
    ref = sums * sa.double() * sb.double()
    off = (terms + 15) // 16 * 17 * 2.0 ** -24 * terms * 2.0 ** 14 if terms * 2 ** 14 > 2 ** 24 else 0.0
    bound = ref.abs() * (HALF_STEP[dtype] * 1.001 + 2.0 ** -22) + off * sa.double() * sb.double() + torch.finfo(dtype).tiny
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (8, 1, 16), (128, 16, 128), (257, 3, 80), (64, 65, 63), (130, 300, 1000),
                                   (512, 64, 2048), (1000, 513, 333), (33, 100, 5), (300, 17, 144), (129, 128, 400),
                                   (2000, 100, 1040), (128, 129, 256), (40, 1, 4096), (640, 112, 16), (20000, 33, 128)])
def test_i8_product(M, N, K, dtype):
    A, Bt, sa, sb = codes(M, K, seed=1), codes(N, K, seed=2), scales(M, seed=3), scales(N, seed=4)
    C = g.i8_tn(A, Bt, sa, sb, dtype=dtype)
    g.gemm_poll_device_status()
    assert C.shape == (N, M) and C.dtype == dtype
    assert_scaled(C, Bt.double() @ A.double().t(), sa[None, :], sb[:, None], K, dtype)


@pytest.mark.parametrize("counts,M,K", [([1], 16, 16), ([0, 3, 0, 1], 128, 64), ([70, 0, 300], 200, 208), ([5, 6], 31, 33),
                                        ([1] * 40, 384, 272), ([64, 0, 65, 3], 130, 128), ([200, 10, 100], 136, 112)])
def test_i8_grouped(counts, M, K):
    E, T = len(counts), sum(counts)
    off = offsets_of(counts)
    A, Bt, sa, sb = codes(E, M, K, seed=1), codes(T, K, seed=2), scales(E, M, seed=3), scales(T, seed=4)
    C = g.i8_tn_grouped(A, Bt, sa, sb, off, dtype=torch.bfloat16)
    g.gemm_poll_device_status()
    b = off.tolist()
    for e in range(E):
        r = slice(b[e], b[e + 1])
        assert_scaled(C[r], Bt[r].double() @ A[e].double().t(), sa[e][None, :], sb[r][:, None], K, torch.bfloat16)


def rows64(x):
    top = x.double().abs().amax(1, keepdim=True) if x.shape[1] else torch.zeros(x.shape[0], 1, device=x.device).double()
    q = torch.where(top > 0, (x.double() * 127 / top).round(), torch.zeros_like(x.double()))
    return q, top[:, 0] / 127


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 16), (5, 2048), (17, 1000), (300, 513), (2, 40000), (2, 70001), (3, 66000), (2000, 37), (1300, 200), (1301, 2049), (1500, 4097), (5, 16385), (3, 9000), (4, 32768), (2, 32770)])
def test_quantise_rows(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows * 131 + cols)
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * 3).to(dtype)
    x[0] = 0
    q, s = g.quantize_i8_rows(x)
    want, scale = rows64(x)
    assert torch.equal(q.double(), want)
    assert torch.equal(s, scale.float())
