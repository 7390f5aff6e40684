"""Shared by the tests of the grouped and 8-bit products: 64-bit forms of the
operators and padded layouts."""
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def offsets_of(counts, lead=0):
    o = [lead]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def padded(t, ld, fill):
    """t (rows, cols) or (E, rows, cols) as a view with row stride ld, the padding filled with `fill`."""
    buf = torch.full((*t.shape[:-1], ld), fill, dtype=t.dtype, device=t.device)
    view = buf[..., : t.shape[-1]]
    view.copy_(t)
    return view


def product64(A, Bt, bounds):
    out = torch.full((Bt.shape[0], A.shape[1]), float("nan"), dtype=torch.float64, device=A.device)
    for e in range(A.shape[0]):
        out[bounds[e]:bounds[e + 1]] = Bt[bounds[e]:bounds[e + 1]].double() @ A[e].double().t()
    return out


def grad_b64(A, dCt, bounds):
    out = torch.full((dCt.shape[0], A.shape[2]), float("nan"), dtype=torch.float64, device=A.device)
    for e in range(A.shape[0]):
        out[bounds[e]:bounds[e + 1]] = dCt[bounds[e]:bounds[e + 1]].double() @ A[e].double()
    return out


def grad_a64(dCt, Bt, bounds):
    return torch.stack([dCt[bounds[e]:bounds[e + 1]].double().t() @ Bt[bounds[e]:bounds[e + 1]].double()
                        for e in range(len(bounds) - 1)])


def small_ints(*shape, seed, dtype, top=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dtype)


def normals(*shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def assert_near(got, ref, size, terms, dtype, what=""):
    """|got - ref| within half a step of the result's type plus what an FP32 sum
    of `terms` products may be off: each MMA adds 16 products to the running sum,
    17 addends cut to 24 bits of the largest, which is at most `size` = the sum
    of the products' magnitudes."""
    mmas = (terms + 15) // 16
    bound = HALF_STEP[dtype] * ref.abs() + mmas * 17 * 2.0 ** -24 * size + torch.finfo(dtype).tiny
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} outside, worst {float(((got.double() - ref).abs() / bound).max())}"
