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
    ([1000, 40], 1032, 264),
    ([2000], 1544, 512),
    ([2] * 70, 200, 136),
    ([31, 33, 32, 1], 256, 4096),
    # more tiles than one wave of single CTAs: CTA pairs
    ([257, 0, 31, 5000], 520, 264),
    ([513, 7, 4025], 384, 640),
    ([3000, 200], 1000, 392),
    ([300, 4900], 129, 127),
    ([10000, 3], 99, 255),
    ([20000], 1, 1),
    ([40] * 30, 700, 520),
    # few tiles with long sums, of the product or the gradient: split over clusters
    ([5], 128, 1536),
    ([3, 0, 64, 65], 200, 4104),
    ([1], 8, 20000),
    ([700], 136, 3333),
    ([2, 31], 9001, 72),
    ([90, 0, 1], 2064, 260),
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


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("counts,M,K", [([3, 5], 256, 2048), ([200, 77, 300], 520, 1000), ([700, 900], 640, 1536),
                                        ([5000, 3333], 640, 1536), ([9, 0, 70], 136, 9000), ([20, 3], 7000, 264)])
def test_normal_values_within_the_derived_bound(counts, M, K, dtype):
    E, T = len(counts), sum(counts)
    off = offsets_of(counts)
    A, Bt, dCt = (normals(*s, seed=i, dtype=dtype) for i, s in enumerate([(E, M, K), (T, K), (T, M)], 1))
    b = bounds_of(off)
    assert_near(g.tn_grouped(A, Bt, off), product64(A, Bt, b), product64(A.abs(), Bt.abs(), b), K, dtype, "product")
    assert_near(g.tn_grouped_grad_b(A, dCt, off), grad_b64(A, dCt, b), grad_b64(A.abs(), dCt.abs(), b), M, dtype, "grad_b")
    assert_near(g.tn_grouped_grad_a(dCt, Bt, off), grad_a64(dCt, Bt, b), grad_a64(dCt.abs(), Bt.abs(), b), max(counts),
                dtype, "grad_a")


@pytest.mark.parametrize("counts,M,K", [([130, 0, 700, 41], 392, 520), ([1300, 0, 7000, 41], 392, 520), ([13, 0, 70, 4], 2056, 4104)])
def test_repeats_bit_for_bit(counts, M, K):
    off, T = offsets_of(counts), sum(counts)
    A, Bt, dCt = (normals(*s, seed=i, dtype=torch.bfloat16)
                  for i, s in enumerate([(4, M, K), (T, K), (T, M)], 1))
    calls = (lambda: g.tn_grouped(A, Bt, off), lambda: g.tn_grouped_grad_b(A, dCt, off),
             lambda: g.tn_grouped_grad_a(dCt, Bt, off))
    for call in calls:
        first = call()
        for _ in range(5):
            assert torch.equal(call(), first)


# (rows per expert, M, K, padding of A's, Bt's and the results' rows, of the expert blocks): strides that the
# TMA takes in place and strides it does not; the padding holds NaN and must not be read, and not be written
STRIDES = [([40, 7], 72, 136, 8, 0), ([40, 7], 72, 136, 1, 0), ([300, 0, 90], 264, 200, 24, 64),
           ([300, 0, 90], 264, 200, 3, 5), ([20, 30], 65, 33, 7, 0), ([1, 70], 129, 1, 9, 1),
           ([3000, 0, 4090], 264, 200, 24, 64), ([3000, 0, 4090], 264, 200, 3, 5), ([9000, 90], 65, 33, 7, 0),
           ([20, 0, 3], 72, 2056, 8, 0), ([20, 0, 3], 72, 2051, 1, 3)]


@pytest.mark.parametrize("counts,M,K,pad,block_pad", STRIDES)
def test_strides_and_padding(counts, M, K, pad, block_pad):
    dtype, E, T = torch.bfloat16, len(counts), sum(counts)
    nan, off = float("nan"), offsets_of(counts)
    b = bounds_of(off)
    A0, B0, D0 = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(E, M, K), (T, K), (T, M)], 1))
    room = torch.full((E, M * (K + pad) + block_pad), nan, dtype=dtype, device="cuda")
    A = room.as_strided((E, M, K), (M * (K + pad) + block_pad, K + pad, 1))
    A.copy_(A0)
    Bt, dCt = padded(B0, K + pad, nan), padded(D0, M + pad, nan)
    mark = 7.25
    C = padded(torch.full((T, M), mark, dtype=dtype, device="cuda"), M + pad, mark)
    dB = padded(torch.full((T, K), mark, dtype=dtype, device="cuda"), K + pad, mark)
    room_d = torch.full((E, M * (K + pad) + block_pad), mark, dtype=dtype, device="cuda")
    dA = room_d.as_strided((E, M, K), (M * (K + pad) + block_pad, K + pad, 1))
    g.tn_grouped(A, Bt, off, C=C)
    g.tn_grouped_grad_b(A, dCt, off, dBt=dB)
    g.tn_grouped_grad_a(dCt, Bt, off, dA=dA)
    g.gemm_poll_device_status()
    assert torch.equal(C, product64(A0, B0, b).to(dtype))
    assert torch.equal(dB, grad_b64(A0, D0, b).to(dtype))
    assert torch.equal(dA, grad_a64(D0, B0, b).to(dtype))
    for view, whole in ((C, C.as_strided((T, M + pad), (M + pad, 1))), (dB, dB.as_strided((T, K + pad), (K + pad, 1)))):
        assert bool((whole[:, view.shape[1]:] == mark).all())
    gaps = room_d[:, : M * (K + pad)].view(E, M, K + pad)[..., K:]
    assert bool((gaps == mark).all()) and bool((room_d[:, M * (K + pad):] == mark).all())


def test_misaligned_bases_and_shared_or_interleaved_experts():
    dtype, counts, M, K = torch.float16, [33, 20], 72, 64
    off = offsets_of(counts)
    b = bounds_of(off)
    flat = small_ints(2 * M * K + 53 * K + 8, seed=3, dtype=dtype)
    A, Bt = flat[1:1 + 2 * M * K].view(2, M, K), flat[3 + 2 * M * K:3 + 2 * M * K + 53 * K].view(53, K)
    assert torch.equal(g.tn_grouped(A, Bt, off), product64(A, Bt, b).to(dtype))
    one = small_ints(1, M, K, seed=4, dtype=dtype).expand(2, M, K)                   # both experts share their weights
    assert torch.equal(g.tn_grouped(one, Bt, off), product64(one, Bt, b).to(dtype))
    mixed = small_ints(M, 2, K, seed=5, dtype=dtype).transpose(0, 1)                 # experts' rows alternate in memory
    assert torch.equal(g.tn_grouped(mixed, Bt, off), product64(mixed, Bt, b).to(dtype))
    out = torch.zeros(M, 2, K, dtype=dtype, device="cuda").transpose(0, 1)
    dCt = small_ints(53, M, seed=6, dtype=dtype)
    g.tn_grouped_grad_a(dCt, Bt, off, dA=out)
    assert torch.equal(out, grad_a64(dCt, Bt, b).to(dtype))


@pytest.mark.parametrize("lead,counts,tail", [(5, [3, 0, 40], 9), (0, [0, 0], 17), (64, [300], 1), (1, [64, 65], 200)])
def test_rows_of_no_expert_are_neither_read_nor_written(lead, counts, tail):
    dtype, M, K = torch.bfloat16, 136, 200
    E, T = len(counts), lead + sum(counts) + tail
    off = offsets_of(counts, lead)
    b = bounds_of(off)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(E, M, K), (T, K), (T, M)], 1))
    for t in (Bt, dCt):
        t[:lead] = float("nan")
        t[b[-1]:] = float("inf")
    C, dB = (torch.full((T, n), 3.5, dtype=dtype, device="cuda") for n in (M, K))
    g.tn_grouped(A, Bt, off, C=C)
    g.tn_grouped_grad_b(A, dCt, off, dBt=dB)
    dA = g.tn_grouped_grad_a(dCt, Bt, off)
    rows = slice(lead, b[-1])
    assert torch.equal(C[rows], product64(A, Bt, b)[rows].to(dtype))
    assert torch.equal(dB[rows], grad_b64(A, dCt, b)[rows].to(dtype))
    assert torch.equal(dA, grad_a64(dCt, Bt, b).to(dtype))
    for t in (C, dB):
        assert bool((t[:lead] == 3.5).all()) and bool((t[b[-1]:] == 3.5).all())


def test_infinities_and_nans_stay_with_their_expert():
    dtype, counts, M, K = torch.float16, [37, 50, 21], 264, 136
    off = offsets_of(counts)
    b = bounds_of(off)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(3, M, K), (108, K), (108, M)], 1))
    clean = [g.tn_grouped(A, Bt, off), g.tn_grouped_grad_b(A, dCt, off), g.tn_grouped_grad_a(dCt, Bt, off)]
    A[1], Bt[b[1]:b[2]], dCt[b[1]:b[2]] = float("nan"), float("inf"), float("nan")
    dirty = [g.tn_grouped(A, Bt, off), g.tn_grouped_grad_b(A, dCt, off), g.tn_grouped_grad_a(dCt, Bt, off)]
    for c, d, own in zip(clean, dirty, [slice(b[1], b[2])] * 2 + [slice(1, 2)]):
        others = torch.ones(c.shape[0], dtype=torch.bool, device="cuda")
        others[own] = False
        assert torch.equal(c[others], d[others])
        assert bool(d[own].isnan().all())


@pytest.mark.parametrize("table", [[0, 30, 10, 64], [-5, 20, 20, 90], [0, 200, 300, 64], [50, 40, 30, 20], [64, 64, 64, 64]])
def test_offsets_out_of_order_or_range_stay_inside(table):
    """Each offset is read as if it were at least the ones before it and at most T."""
    dtype, M, K, T = torch.float16, 72, 80, 64
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    b, top = [], 0
    for o in table:
        top = max(top, min(max(o, 0), T))
        b.append(top)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(3, M, K), (T, K), (T, M)], 1))
    C, dB = (torch.full((T, n), 3.5, dtype=dtype, device="cuda") for n in (M, K))
    g.tn_grouped(A, Bt, off, C=C)
    g.tn_grouped_grad_b(A, dCt, off, dBt=dB)
    dA = g.tn_grouped_grad_a(dCt, Bt, off)
    g.gemm_poll_device_status()
    for got, ref in ((C, product64(A, Bt, b)), (dB, grad_b64(A, dCt, b))):
        assert torch.equal(got, torch.where(ref.isnan(), torch.full_like(ref, 3.5), ref).to(dtype))
    assert torch.equal(dA, grad_a64(dCt, Bt, b).to(dtype))


@pytest.mark.parametrize("table", [[0, 0, 30, 30, 10, 64, 64], [-5, -9, 20, 90, 80, 70, 64], [64, 3, 50, 63, 64, 65, 9],
                                   [0, 30, 10, 20, 31, 31, 64]])
@pytest.mark.parametrize("M,K", [(65, 63), (300, 137)])
def test_copied_weights_of_experts_without_rows(table, M, K):
    """Weights that have to be copied are so for experts with rows alone: the others' may
    hold anything, and no expert with rows is left out whatever the order of the offsets."""
    dtype, T, E = torch.bfloat16, 64, 6
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    b, top = [], 0
    for o in table:
        top = max(top, min(max(o, 0), T))
        b.append(top)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(E, M, K), (T, K), (T, M)], 1))
    for e in range(E):
        if b[e] == b[e + 1]:
            A[e] = float("nan")
    junk = torch.full((1 << 22,), float("nan"), device="cuda")           # what the workspace may be made of
    del junk
    C, dB = (torch.full((T, n), 3.5, dtype=dtype, device="cuda") for n in (M, K))
    g.tn_grouped(A, Bt, off, C=C)
    g.tn_grouped_grad_b(A, dCt, off, dBt=dB)
    g.gemm_poll_device_status()
    for got, ref in ((C, product64(A, Bt, b)), (dB, grad_b64(A, dCt, b))):
        assert torch.equal(got, torch.where(ref.isnan(), torch.full_like(ref, 3.5), ref).to(dtype))


def test_empty_sums_and_sizes():
    off = offsets_of([3, 0, 5])
    f16 = dict(dtype=torch.float16, device="cuda")
    C = torch.full((8, 40), 9.0, **f16)
    g.tn_grouped(torch.zeros(3, 40, 0, **f16), torch.zeros(8, 0, **f16), off, C=C)
    assert bool((C == 0).all())
    dB = torch.full((10, 24), 9.0, **f16)
    g.tn_grouped_grad_b(torch.zeros(3, 0, 24, **f16), torch.zeros(10, 0, **f16), off, dBt=dB)
    assert bool((dB[:8] == 0).all()) and bool((dB[8:] == 9).all())
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    dA = g.tn_grouped_grad_a(torch.zeros(0, 40, **f16), torch.zeros(0, 24, **f16), none, dA=torch.full((3, 40, 24), 9.0, **f16))
    assert bool((dA == 0).all())
    assert g.tn_grouped(torch.zeros(3, 40, 24, **f16), torch.zeros(0, 24, **f16), none).shape == (0, 40)
    assert g.tn_grouped(torch.zeros(3, 0, 24, **f16), torch.zeros(8, 24, **f16), off).shape == (8, 0)
    g.gemm_poll_device_status()


@pytest.mark.parametrize("E", [333, 1024])
def test_many_experts(E):
    gen = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 4, (E,), generator=gen).tolist()
    off = offsets_of(counts)
    b, T = bounds_of(off), sum(counts)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=torch.float16) for i, s in enumerate([(E, 40, 24), (T, 24), (T, 40)], 1))
    assert torch.equal(g.tn_grouped(A, Bt, off), product64(A, Bt, b).half())
    assert torch.equal(g.tn_grouped_grad_b(A, dCt, off), grad_b64(A, dCt, b).half())
    assert torch.equal(g.tn_grouped_grad_a(dCt, Bt, off), grad_a64(dCt, Bt, b).half())


def test_gradients_against_differences():
    """C is linear in Bt and in A, so a difference of two products, weighted with dC,
    is the gradient's product with the step; small integers make both sides exact."""
    counts, M, K, dtype = [50, 0, 83, 130], 136, 72, torch.float16
    off = offsets_of(counts)
    A, Bt, dCt, dir_a, dir_b = (small_ints(*s, seed=i, dtype=dtype, top=2) for i, s in enumerate(
        [(4, M, K), (263, K), (263, M), (4, M, K), (263, K)], 1))
    base = g.tn_grouped(A, Bt, off).double()
    by_b = ((g.tn_grouped(A, Bt + dir_b, off).double() - base) * dCt.double()).sum()
    by_a = ((g.tn_grouped(A + dir_a, Bt, off).double() - base) * dCt.double()).sum()
    assert float(by_b) == float((g.tn_grouped_grad_b(A, dCt, off).double() * dir_b.double()).sum())
    assert float(by_a) == float((g.tn_grouped_grad_a(dCt, Bt, off).double() * dir_a.double()).sum())


@pytest.mark.parametrize("table", [[5, 8, 8, 50], [0, 30, 10, 64], [-5, 20, 20, 90], [50, 40, 30, 20], [64, 64, 64, 64]])
def test_split_sums_with_rows_of_no_expert_and_infinities(table):
    """Sums long enough to be split over clusters (K of the product, M of the gradient):
    tables as above, one expert's values infinite or NaN, strided and unaligned results."""
    M, K, T, dtype = 2064, 2056, 64, torch.bfloat16
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    b, top = [], 0
    for o in table:
        top = max(top, min(max(o, 0), T))
        b.append(top)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=dtype) for i, s in enumerate([(3, M, K), (T, K), (T, M)], 1))
    A[1], Bt[:b[0]], Bt[b[3]:], dCt[:b[0]], dCt[b[3]:] = (float("nan"),) * 5
    Bt[b[2]:b[3]][:1, 7] = float("inf")
    narrow = A[:, :130], dCt[:, :130]                      # the product's A (a part of its rows), the gradient's by its columns
    for call, A_, R, pad in ((g.tn_grouped, narrow[0], Bt, 3), (g.tn_grouped_grad_b, A[..., :136], dCt, 8)):
        ref = (product64 if call is g.tn_grouped else grad_b64)(A_, R, b)
        room = torch.full((T, ref.shape[1] + pad), 3.5, dtype=dtype, device="cuda")
        out = room[:, : ref.shape[1]]
        call(A_, R, off, **{"C" if call is g.tn_grouped else "dBt": out})
        g.gemm_poll_device_status()
        assert bool((room[:, ref.shape[1]:] == 3.5).all())
        owned = torch.zeros(T, dtype=torch.bool, device="cuda")
        owned[b[0]:b[3]] = True
        assert bool((out[~owned] == 3.5).all())
        assert torch.equal(out[owned].isnan(), ref[owned].to(dtype).isnan())
        finite = ~ref[owned].isnan()
        assert torch.equal(out[owned][finite], ref[owned].to(dtype)[finite])


def test_past_2_31_elements():
    """Weights, tokens and results of more than 2^31 elements: offsets in 64 bits."""
    M, K, E = 4096, 4096, 130                      # 2.18e9 weights
    A = torch.zeros(E, M, K, dtype=torch.float16, device="cuda")
    A[E - 1] = small_ints(M, K, seed=1, dtype=torch.float16, top=1)
    T = 530000                                     # 2.17e9 token elements and results
    Bt = torch.zeros(T, K, dtype=torch.float16, device="cuda")
    Bt[-300:] = small_ints(300, K, seed=2, dtype=torch.float16, top=1)
    off = torch.full((E + 1,), T - 300, dtype=torch.int32, device="cuda")
    off[0], off[E] = 0, T
    C = g.tn_grouped(A, Bt, off)
    g.gemm_poll_device_status()
    want = (Bt[-300:].double() @ A[E - 1].double().t()).half()
    assert torch.equal(C[-300:], want) and float(C[:1000].abs().max()) == 0
    dB = g.tn_grouped_grad_b(A, C, off)
    assert torch.equal(dB[-300:], (C[-300:].double() @ A[E - 1].double()).half())
    del dB
    dA = g.tn_grouped_grad_a(C, Bt, off, dA=A)
    assert torch.equal(dA[E - 1], (want.double().t() @ Bt[-300:].double()).half()) and float(dA[E - 2].abs().max()) == 0


@pytest.mark.parametrize("M", [2 ** 31 - 256, 2 ** 31 - 512])
def test_weight_gradient_of_the_most_rows(M):
    """As many rows of dA as a call may have: their number of tiles in 32 bits."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    dCt = torch.randint(-3, 4, (1, M), generator=gen, device="cuda", dtype=torch.int8).half()
    dA = torch.full((1, M, 1), 9.0, dtype=torch.float16, device="cuda")
    g.tn_grouped_grad_a(dCt, torch.full((1, 1), 2.0, dtype=torch.float16, device="cuda"), offsets_of([1]), dA=dA)
    g.gemm_poll_device_status()
    assert torch.equal(dA.view(-1), dCt.view(-1) * 2)


# ------------------------------------------------------------------ streams, graphs, threads
def small_case(seed, dtype=torch.bfloat16):
    counts = [40, 0, 130, 9]
    off = offsets_of(counts)
    A, Bt, dCt = (small_ints(*s, seed=seed + i, dtype=dtype) for i, s in enumerate([(4, 200, 137), (179, 137), (179, 200)]))
    return A, Bt, dCt, off


def results(A, Bt, dCt, off, stream=None):
    return [g.tn_grouped(A, Bt, off, stream=stream), g.tn_grouped_grad_b(A, dCt, off, stream=stream),
            g.tn_grouped_grad_a(dCt, Bt, off, stream=stream)]


def wanted(A, Bt, dCt, off):
    b = bounds_of(off)
    return [product64(A, Bt, b).to(A.dtype), grad_b64(A, dCt, b).to(A.dtype), grad_a64(dCt, Bt, b).to(A.dtype)]


@pytest.mark.parametrize("as_int", [False, True])
def test_other_streams(as_int):
    """K = 137 copies the operands: the workspace belongs to the call's stream."""
    case = small_case(1)
    want = wanted(*case)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append(results(*case, stream=s.cuda_stream if as_int else s))
        junk = torch.full((1 << 20,), float("nan"), device="cuda")       # what torch may put into freed memory meanwhile
        del junk
    s.synchronize()
    for r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, want))
    with torch.cuda.stream(s):
        inside = results(*case)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(inside, want))


@pytest.mark.parametrize("kind", ["none", "object", "handle", "default_object", "default_handle"])
def test_the_workspace_belongs_to_the_calls_stream(kind):
    """A freed block is handed out again to its own stream alone, so the workspace's
    comes back for that stream.  (The default stream's handle is 0.)"""
    g.quantize_i8_rows(torch.zeros(1, 1, device="cuda"))          # (the helpers' torch is looked up by their first call)
    device, side, default = torch.device("cuda", 0), torch.cuda.Stream(), torch.cuda.default_stream()
    stream, own = {"none": (None, default), "object": (side, side), "handle": (side.cuda_stream, side),
                   "default_object": (default, default), "default_handle": (default.cuda_stream, default)}[kind]
    n = 3 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ws = g._workspace(device, stream, n)
    at = ws.data_ptr()
    del ws
    with torch.cuda.stream(own):
        again = torch.empty(n, dtype=torch.uint8, device=device)
    assert again.data_ptr() == at


def helper_calls(T, M, K, E):
    """Each helper of the grouped and 8-bit products with operands that are contiguous (its
    short way) and the same with an output given (its long way); small integers."""
    counts = [T // E] * (E - 1) + [T - T // E * (E - 1)]
    off = offsets_of(counts)
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=torch.float16) for i, s in enumerate([(E, M, K), (T, K), (T, M)], 1))
    qa, qb, sa, sb = A.to(torch.int8), Bt.to(torch.int8), torch.full((E, M), 0.5, device="cuda"), torch.ones(T, device="cuda")
    new = lambda *s: torch.full(s, 9.0, dtype=torch.float16, device="cuda")  # noqa: E731
    return {
        "tn_grouped": (lambda **kw: g.tn_grouped(A, Bt, off, **kw), dict(C=new(T, M))),
        "tn_grouped_grad_b": (lambda **kw: g.tn_grouped_grad_b(A, dCt, off, **kw), dict(dBt=new(T, K))),
        "tn_grouped_grad_a": (lambda **kw: g.tn_grouped_grad_a(dCt, Bt, off, **kw), dict(dA=new(E, M, K))),
        "i8_tn": (lambda **kw: g.i8_tn(qa[0], qb, sa[0], sb, **kw), dict(C=new(T, M))),
        "i8_tn_grouped": (lambda **kw: g.i8_tn_grouped(qa, qb, sa, sb, off, **kw), dict(C=new(T, M))),
    }


@pytest.mark.parametrize("name", ["tn_grouped", "tn_grouped_grad_b", "tn_grouped_grad_a", "i8_tn", "i8_tn_grouped"])
@pytest.mark.parametrize("T,M,K,E", [(70, 40, 24, 3), (70, 40, 23, 3), (1, 1, 1, 1), (0, 8, 8, 2), (5, 0, 8, 2), (5, 8, 0, 2),
                                     (5, 1, 9, 2), (5, 9, 1, 2)])
def test_both_ways_through_a_helper_agree(name, T, M, K, E):
    call, out = helper_calls(T, M, K, E)[name]
    short, longer = call(), call(**out)
    g.gemm_poll_device_status()
    given = next(iter(out.values()))
    assert longer.data_ptr() == given.data_ptr() and short.dtype == longer.dtype
    assert short.shape == longer.shape and torch.equal(short, longer)


def wrong_arguments():
    f16, i8 = dict(dtype=torch.float16, device="cuda"), dict(dtype=torch.int8, device="cuda")
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    A, Bt, dCt = torch.zeros(2, 16, 8, **f16), torch.zeros(5, 8, **f16), torch.zeros(5, 16, **f16)
    qa, qb, sa, sb = torch.zeros(2, 16, 8, **i8), torch.zeros(5, 8, **i8), torch.ones(2, 16, device="cuda"), torch.ones(5, device="cuda")
    for o in (off.long(), off[:2], off.cpu(), off[None]):
        yield lambda o=o: g.tn_grouped(A, Bt, o)
        yield lambda o=o: g.tn_grouped_grad_b(A, dCt, o)
        yield lambda o=o: g.i8_tn_grouped(qa, qb, sa, sb, o)
        if o.numel() == 3:
            yield lambda o=o: g.tn_grouped_grad_a(dCt, Bt, o)
    for b in (Bt.bfloat16(), Bt[:, :4].contiguous(), Bt.cpu(), Bt[0], Bt.float()):
        yield lambda b=b: g.tn_grouped(A, b, off)
        yield lambda b=b: g.tn_grouped_grad_b(A, b, off)
        if b.dtype != torch.float16 or b.shape[0] != 5 or not b.is_cuda:
            yield lambda b=b: g.tn_grouped_grad_a(dCt, b, off)
    for a in (A.bfloat16(), A[0], A.cpu(), A.float()):
        yield lambda a=a: g.tn_grouped(a, Bt, off)
        yield lambda a=a: g.tn_grouped_grad_b(a, dCt, off)
    yield lambda: g.tn_grouped_grad_a(dCt[:4], Bt, off)
    for s in (sb[:4], sb.double(), sb.cpu(), sb[None], torch.ones(10, device="cuda")[::2]):
        yield lambda s=s: g.i8_tn(qa[0], qb, sa[0], s)
        yield lambda s=s: g.i8_tn_grouped(qa, qb, sa, s, off)
    for s in (sa[0], sa.half(), sa.cpu(), sa.t(), sa[:1]):
        yield lambda s=s: g.i8_tn_grouped(qa, qb, s, sb, off)
    yield lambda: g.i8_tn(qa[0], qb, sa, sb)
    for q in (qb.to(torch.uint8), qb[:, :4].contiguous(), qb.cpu(), qb[0]):
        yield lambda q=q: g.i8_tn(qa[0], q, sa[0], sb)
        yield lambda q=q: g.i8_tn_grouped(qa, q, sa, sb, off)
    yield lambda: g.i8_tn(qa[0], qb, sa[0], sb, dtype=torch.float32)
    yield lambda: g.i8_tn(qa[0], qb, sa[0], sb, C=torch.zeros(5, 16, **f16), dtype=torch.bfloat16)
    yield lambda: g.tn_grouped(A, Bt, off, C=torch.zeros(5, 16, **f16).bfloat16())
    yield lambda: g.tn_grouped(A, Bt, off, C=torch.zeros(5, 15, **f16))
    yield lambda: g.tn_grouped_grad_a(dCt, Bt, off, dA=torch.zeros(1, 16, 8, **f16).expand(2, 16, 8))


def test_helpers_refuse_what_does_not_fit_on_a_gpu():
    """Nothing slips past the checks on a helper's short way."""
    for i, call in enumerate(wrong_arguments()):
        try:
            call()
        except (ValueError, g.GemmError):
            continue
        raise AssertionError(f"call {i} was not refused")
    g.gemm_poll_device_status()


def test_captured_replayed_and_two_graphs_at_once():
    cases = [small_case(1), small_case(50)]
    for c in cases:
        results(*c)                                 # first calls set kernel attributes
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(results(*c))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for step in range(4):
        for i, c in enumerate(cases):               # new values, and other groups, at the same addresses
            c[0].copy_(small_ints(*c[0].shape, seed=100 + 7 * step + i, dtype=c[0].dtype))
            c[3].copy_(offsets_of([[40, 0, 130, 9], [0, 0, 0, 179], [1, 2, 3, 173], [170, 3, 3, 3]][step]))
        torch.cuda.synchronize()
        for _ in range(10):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            assert all(torch.equal(x, y) for x, y in zip(out, wanted(*c)))
    g.gemm_poll_device_status()


def test_two_threads_on_two_streams():
    import threading
    cases = [small_case(1), small_case(90)]
    want = [wanted(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = results(*cases[i])
                s.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                    bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_offsets_and_inputs_written_just_before_the_call():
    """The kernels start early (programmatic dependent launch) but wait for the kernel
    before them on the stream before they read."""
    dtype, M, K, T = torch.float16, 256, 128, 300
    A, src = small_ints(2, M, K, seed=1, dtype=dtype), small_ints(T, K, seed=2, dtype=dtype)
    Bt, off = torch.zeros_like(src), torch.zeros(3, dtype=torch.int32, device="cuda")
    for cut in (0, 1, 77, 299, 300):
        want = product64(A, src, [0, cut, T]).to(dtype)
        torch.cuda.synchronize()
        for _ in range(10):
            Bt.zero_()
            off.zero_()
            Bt.copy_(src)
            off[1:2].fill_(cut)
            off[2:3].fill_(T)
            C = g.tn_grouped(A, Bt, off)
            C2 = g.tn_grouped(A, Bt, off)
            assert torch.equal(C, want) and torch.equal(C2, want)


@pytest.mark.parametrize("mode", [1, 2, 3])
def test_a_stalled_part_of_a_split_sum_reports_a_timeout(mode):
    """Mode 1 stalls the MMAs, mode 2 the producer of a cluster's first CTA, mode 3 the others'."""
    off = offsets_of([5, 9])
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=torch.float16) for i, s in enumerate([(2, 2056, 4104), (14, 4104), (14, 2056)], 1))
    for call in (lambda: g.tn_grouped(A[:, :128], Bt, off), lambda: g.tn_grouped_grad_b(A[..., :128], dCt, off)):
        want = call()
        g.gemm_poll_device_status()
        g.gemm_set_wait_limit_ns(20_000_000)
        g.gemm_debug_inject_stall(mode)
        try:
            call()
            with pytest.raises(g.GemmError) as e:
                g.gemm_poll_device_status()
            assert e.value.status == g.GEMM_ERR_TIMEOUT
        finally:
            g.gemm_debug_inject_stall(0)
            g.gemm_set_wait_limit_ns(0)
        assert torch.equal(call(), want)
        g.gemm_poll_device_status()


@pytest.mark.parametrize("mode", [1, 2, 3])
@pytest.mark.parametrize("rows", [8, 3000])
def test_a_stalled_role_reports_a_timeout_and_leaves_the_context_usable(mode, rows):
    """rows 8: single CTAs; 3000: CTA pairs.  (Mode 3, the odd CTA's producer, has
    nothing to stall in a single CTA.)"""
    off = offsets_of([rows, rows])
    A, Bt, dCt = (small_ints(*s, seed=i, dtype=torch.float16)
                  for i, s in enumerate([(2, 520, 1000), (2 * rows, 1000), (2 * rows, 520)], 1))
    calls = [lambda: g.tn_grouped(A, Bt, off), lambda: g.tn_grouped_grad_b(A, dCt, off),
             lambda: g.tn_grouped_grad_a(dCt, Bt, off)]
    want = [c() for c in calls]
    g.gemm_poll_device_status()
    for i, call in enumerate(calls):
        paired = rows > 32 or i == 2
        g.gemm_set_wait_limit_ns(20_000_000)
        g.gemm_debug_inject_stall(mode)
        try:
            call()
            if mode != 3 or paired:
                with pytest.raises(g.GemmError) as e:
                    g.gemm_poll_device_status()
                assert e.value.status == g.GEMM_ERR_TIMEOUT
        finally:
            g.gemm_debug_inject_stall(0)
            g.gemm_set_wait_limit_ns(0)
        assert torch.equal(call(), want[i])
        g.gemm_poll_device_status()


def test_an_expert_layer_forward_and_backward_together():
    """Tokens routed on the device, two grouped products with a gate between them, and
    the whole backward pass from the two gradients, against autograd in 64 bits."""
    dtype, E, T, D, H = torch.bfloat16, 6, 500, 256, 384
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, D, generator=gen, device="cuda").to(dtype)
    up, down = (torch.randn(*s, generator=gen, device="cuda").mul_(s[-1] ** -0.5).to(dtype) for s in ((E, H, D), (E, D, H)))
    expert = torch.randint(0, E - 1, (T,), generator=gen, device="cuda")       # the last expert gets none
    order = torch.argsort(expert, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(expert, minlength=E).cumsum(0)
    xs = x[order].contiguous()
    h = g.tn_grouped(up, xs, off)
    a = torch.relu(h)
    y = g.tn_grouped(down, a, off)
    dy = torch.randn(T, D, generator=gen, device="cuda").to(dtype)
    d_down = g.tn_grouped_grad_a(dy, a, off)
    da = g.tn_grouped_grad_b(down, dy, off)
    dh = da * (h > 0)
    d_up = g.tn_grouped_grad_a(dh, xs, off)
    dx = g.tn_grouped_grad_b(up, dh, off)
    g.gemm_poll_device_status()

    # the same in 64 bits, with the roundings of h, a, da and dh to bf16 that the layer makes
    b = bounds_of(off)
    near = lambda got, ref: float((got.double() - ref).norm() / ref.norm())  # noqa: E731
    up64, down64 = up.double().requires_grad_(), down.double().requires_grad_()
    xs64 = xs.double().requires_grad_()
    h64 = torch.cat([xs64[b[e]:b[e + 1]] @ up64[e].t() for e in range(E)])
    # rounding to bf16 is taken as constant: relu's mask is the rounded h's
    a64 = h64 * (h > 0)
    y64 = torch.cat([a64[b[e]:b[e + 1]] @ down64[e].t() for e in range(E)])
    (y64 * dy.double()).sum().backward()
    # each output is off by its own rounding and those of what it was made from: at
    # most 2^-8 relative each, independent of each other in direction
    assert near(y, y64.detach()) < 2 * 2.0 ** -8 and near(dx, xs64.grad) < 2 * 2.0 ** -8
    assert near(d_down, down64.grad) < 2 * 2.0 ** -8 and near(d_up, up64.grad) < 2 * 2.0 ** -8
    assert float(d_up[E - 1].abs().max()) == 0 and float(d_down[E - 1].abs().max()) == 0
