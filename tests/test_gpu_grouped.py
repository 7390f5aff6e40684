"""Products grouped by expert and their gradients on the GPU, against 64-bit forms.

Small-integer inputs keep every sum below 2^24, where FP32 sums are exact in any
order, so those cases are compared bit for bit with the once-rounded sum."""
import pytest
import torch

from tests.grouped_helpers import (assert_near, grad_a64, grad_b64, normals, offsets_of, padded, product64, small_ints)

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import dense_gemm_tn_gb300 as g

TYPES = [torch.float16, torch.bfloat16]

# (rows per expert, M, K): one token; empty experts first, last and between; single
# rows; rows past one, two and several tiles of the N side; sums and widths that
# are not a block's or a tile's; widths that are no multiple of 8 (operand copies)
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0], 64, 64),
    ([5, 0, 3, 0], 128, 128),
    ([1, 1, 1, 1, 1, 1, 1, 1], 256, 72),
    ([16, 17, 15], 136, 200),
    ([64, 65, 63], 264, 136),
    ([0, 257, 0, 31], 520, 264),
    ([300, 200], 1000, 392),
    ([513, 7, 1025], 384, 640),
    ([129], 2048, 1024),
    ([33, 40], 65, 63),
    ([100, 3], 127, 129),
    ([300, 90], 99, 255),
    ([256, 256], 1, 1),
    ([70], 17, 1),
    ([200, 300], 1, 640),
]


def bounds_of(offsets):
    return offsets.tolist()


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("counts,M,K", SHAPES)
def test_product_and_gradients_bit_exact(counts, M, K, dtype):
    E, T = len(counts), sum(counts)
    off = offsets_of(counts)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(E, M, K), (T, K), (T, M)], 1))
    C = g.tn_grouped(A, Bt, off)
    dBt = g.tn_grouped_grad_b(A, dCt, off)
    dA = g.tn_grouped_grad_a(dCt, Bt, off)
    g.gemm_poll_device_status()
    b = bounds_of(off)
    assert torch.equal(C, product64(A, Bt, b).to(dtype))
    assert torch.equal(dBt, grad_b64(A, dCt, b).to(dtype))
    assert torch.equal(dA, grad_a64(dCt, Bt, b).to(dtype))
