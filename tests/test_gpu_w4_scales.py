"""The 4-bit quantiser's scales and codes against max / 7, over enough groups for the quotient's borders to be met."""
import pytest
import torch

from tests.grouped_helpers import normals

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")


def divided(x, group, dtype):
    """(codes, scales): max / 7 in FP32 and rounded, x / scale in 64 bits."""
    rows, cols = x.shape
    pad = torch.zeros(rows, -(-cols // group) * group, device="cuda", dtype=torch.float64)
    pad[:, :cols] = x
    pad = pad.view(rows, -1, group)
    scale = (pad.abs().amax(2).float() / torch.full((), 7.0, device="cuda")).to(dtype)
    by = scale.double()[..., None]
    q = torch.where(by > 0, (pad / torch.where(by > 0, by, 1.0)).round().clamp(-8, 7), 0.0)
    return q.flatten(1)[:, :cols].to(torch.int8), scale


def unpack(q, cols):
    q = q.contiguous().view(torch.int8)
    return torch.stack(((q << 4) >> 4, q >> 4), -1).flatten(1)[:, :cols]


@pytest.mark.parametrize("source", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,group", [(8192, 8192, 128), (2000, 264, 32), (20001, 40, 32), (15001, 257, 32), (6001, 1029, 256), (100003, 8, 32),
                                             (4096, 4096, 64)])
def test_scales_are_the_maximum_by_seven(rows, cols, group, dtype, source):
    x = normals(rows, cols, seed=rows, dtype=torch.float32).mul_(1 + torch.arange(rows, device="cuda")[:, None] % 7).to(source)
    q, scale = tn.quantize_w4_rows(x, group, dtype=dtype)
    tn.gemm_poll_device_status()
    q64, s64 = divided(x, group, dtype)
    assert torch.equal(scale, s64)
    assert torch.equal(unpack(q, cols), q64)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_maxima_next_to_borders(dtype):
    """Maxima on both sides of 7 t for numbers t half-way between two scales, and 7 t itself, where 16-bit scales tie."""
    bits = 12 if dtype == torch.float16 else 9                      # t: a bit more than the type has
    t = torch.arange(2 ** (bits - 1) + 1, 2 ** bits, 2, device="cuda", dtype=torch.float64)
    tops = []
    for e in (-13, -3, 0, 4):
        exact = 7 * t * 2.0 ** (e - bits + 1)
        f = exact.float()
        assert torch.equal(f.double(), exact)
        tops += [f, torch.nextafter(f, f * 2), torch.nextafter(f, f * 0)]
    top = torch.cat(tops)
    x = normals(len(top), 32, seed=3, dtype=torch.float32).clamp_(-1, 1) * top[:, None]
    x[:, 17] = -top
    q, scale = tn.quantize_w4_rows(x, 32, dtype=dtype)
    q64, s64 = divided(x, 32, dtype)
    assert torch.equal(scale, s64) and torch.equal(unpack(q, 32), q64)
