"""The activations and their slopes by themselves, gates from -13 to 13 and further: H and dP of single products, against 64 bits."""
import pytest
import torch

from tests.grouped_helpers import HALF_STEP
from tests.sink_helpers import act64

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")

ACTS = ["silu", "gelu", "gelu_tanh"]


def relative(x, act):
    """What act(x) may be off, relative to itself: silu an exponential of a rounded argument, |x| 2^-23 and 2^-21; gelu the fit and x^2
    rounded, x^2 2^-24 and 2^-21; gelu_tanh an argument of 1.6 (|x| + 0.045 |x|^3) rounded three times."""
    x = x.abs()
    if act == "silu":
        return x * 2.0 ** -23 + 2.0 ** -20
    if act == "gelu":
        return x * x * 2.0 ** -24 + 2.0 ** -20
    return 1.6 * (x + 0.045 * x ** 3) * 2.0 ** -22 + 2.0 ** -20


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,lo", [(torch.float16, -6.5), (torch.bfloat16, -13.0)])
def test_far_gates(dtype, lo, act, few):
    """P = [gate | up] of one product each: gates as the type has them, up a power of two that puts H into the middle of its range."""
    M, K = 2048, 8
    half = HALF_STEP[dtype]                                        # (of the number itself)
    gates = torch.linspace(lo, 13.0, M, device="cuda", dtype=torch.float64).to(dtype)
    want, slope = act64(gates.double(), act)
    A = torch.zeros(2 * M, K, device="cuda", dtype=dtype)
    A[:M, 0] = gates
    T = 3 if few else 300
    Bt = torch.zeros(T, K, device="cuda", dtype=dtype)
    Bt[:, 0], Bt[:, 1] = 1.0, 2.0 ** 10 if dtype == torch.float16 else 1.0
    e = (-torch.log2(want.abs().clamp(min=2.0 ** -140))).round()
    A[M:, 1] = torch.exp2(e.clamp(-4, 14 if dtype == torch.float16 else 120)).to(dtype)
    up = A[M:, 1].double() * Bt[0, 1].double()
    H, P = tn.tn_gated(A, Bt, act=act, keep=True)
    tn.gemm_poll_device_status()
    assert torch.equal(P[0, :M].double(), gates.double()) and torch.equal(P[0, M:].double(), up)
    ref = want * up
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    ok = ref.abs() < torch.finfo(dtype).max
    err = (H.double() - ref).abs()[:, ok]
    # (exp(-x) beyond 2^126, FP32's largest whose reciprocal is a normal number: there the activation may be 0)
    gone = want.abs() <= gates.double().abs() * 2.0 ** -126
    assert bool((err <= (ref.abs() * half * 1.0001 + ref.abs() * relative(gates.double(), act) + tiny + torch.where(gone, ref.abs(), 0.0))[ok]).all())
    # the same gates' gradients: one token whose first column is 1, so that dA's first column is dP
    dH = torch.ones(T, M, device="cuda", dtype=dtype)
    dA, _ = tn.tn_gated_grad(A, Bt[:1].contiguous(), P[:1].contiguous(), dH[:1].contiguous(), act=act, want_b=False)
    tn.gemm_poll_device_status()
    step = half * 2.0002                  # (dP's rounding and the result's)
    dg, du = slope * up, want
    # (a slope is y + x y': near its zeros an absolute error, of the size of its parts)
    parts = (want / gates.double()).abs().nan_to_num(0.5) * (2 + 2 * gates.double().abs())
    fits = dg.abs() < torch.finfo(dtype).max / 2
    largest = float(torch.cat((dg.abs(), du.abs())).max())
    for got, exact, off in ((dA[:M, 0], dg, parts * up * relative(gates.double(), act) * 2), (dA[M:, 0], du, du.abs() * relative(gates.double(), act))):
        bound = exact.abs() * step + off + tiny + torch.where(gone, exact.abs(), 0.0) + largest * 2.0 ** -29 * (dtype == torch.float16)
        assert bool(((got.double() - exact).abs() <= bound)[fits].all()), float((((got.double() - exact).abs() / bound)[fits]).max())
