"""Shared by the tests of the gated projections and of the vocabulary's loss:
64-bit forms and the bounds that follow from the kernels' arithmetic."""
import math

import torch

from tests.grouped_helpers import HALF_STEP


def sum_error(size, terms):
    """What an FP32 sum of `terms` products may be off (grouped_helpers.assert_near)."""
    return (terms + 15) // 16 * 17 * 2.0 ** -24 * size


def act64(x, act):
    """(act(x), act'(x)) in 64 bits."""
    if act == "silu":
        y = torch.sigmoid(x)
        return x * y, y + x * y * (1 - y)
    if act == "gelu":
        y = 0.5 * torch.erfc(-x / math.sqrt(2))
        return x * y, y + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    y = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return x * y, y + x * y * (1 - y) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


def act_rel(x):
    """Relative error of the kernels' y(x) = act(x) / x: an argument rounded a few times (a step of 2^-24 of
    |x|, of x^2 / 2 in erfc's exponent, of 1.6 (|x| + 0.045 |x|^3) in tanh's), exp and the quotient or erfc
    within 2^-20."""
    x = x.abs()
    return (8 + 8 * x + 2 * x * x + 0.3 * x ** 3) * 2.0 ** -23


def slope_error(x):
    """Absolute error of act'(x) = y + x y': y off by act_rel(x), y' = O(y (1 - y) (1 + x^2)) by a few times that."""
    return act_rel(x) * (1 + x.abs()) * 4


def gated64(A, Bt, bounds, act):
    """(H, P, what P may be off) of every expert's rows; NaN elsewhere."""
    E, rows, K = A.shape
    P = torch.full((Bt.shape[0], rows), float("nan"), dtype=torch.float64, device=A.device)
    size = P.clone()
    for e in range(E):
        r = slice(bounds[e], bounds[e + 1])
        P[r] = Bt[r].double() @ A[e].double().t()
        size[r] = Bt[r].double().abs() @ A[e].double().abs().t()
    M = rows // 2
    return act64(P[:, :M], act)[0] * P[:, M:], P, sum_error(size, K)


def gated_bound(P, off, act, dtype):
    M = P.shape[1] // 2
    g, u, og, ou = P[:, :M], P[:, M:], off[:, :M], off[:, M:]
    a = act64(g, act)[0]
    h = a * u
    # |act'| <= 1.13 for all three
    return (HALF_STEP[dtype] * h.abs() + (u.abs() + ou) * (1.13 * og) + a.abs() * ou + (act_rel(g) + 2.0 ** -22) * (h.abs() + ou * a.abs())
            + torch.finfo(dtype).tiny) * 1.01


def gated_grad64(A, Bt, P, dH, bounds, act, dtype):
    """(dA, dB, what each may be off) for products P as they were kept."""
    E, rows, K = A.shape
    M = rows // 2
    P, dH, half = P.double(), dH.double(), HALF_STEP[dtype]
    g, u = P[:, :M], P[:, M:]
    a, s = act64(g, act)
    dP = torch.cat((dH * u * s, dH * a), 1)
    off = torch.cat(((dH * u).abs() * (slope_error(g) + 2.0 ** -22 * s.abs()), dH.abs() * a.abs() * (act_rel(g) + 2.0 ** -22)), 1)
    off = off + half * (dP.abs() + off) + torch.finfo(dtype).tiny * half * 4       # (rounded; below the smallest normal number to a step of it)
    dA = torch.zeros(A.shape, dtype=torch.float64, device=A.device)
    dB = torch.full((Bt.shape[0], K), float("nan"), dtype=torch.float64, device=A.device)
    eA, eB = torch.zeros_like(dA), torch.zeros_like(dB)
    for e in range(E):
        r = slice(bounds[e], bounds[e + 1])
        n = bounds[e + 1] - bounds[e]
        d, o, x, W = dP[r], off[r], Bt[r].double(), A[e].double()
        dA[e], dB[r] = d.t() @ x, d @ W
        eA[e] = o.t() @ x.abs() + sum_error((d.abs() + o).t() @ x.abs(), n)
        eB[r] = o @ W.abs() + sum_error((d.abs() + o) @ W.abs(), rows)
    tiny = torch.finfo(dtype).tiny
    return dA, dB, (half * dA.abs() + 1.01 * eA + tiny), (half * dB.abs() + 1.01 * eB + tiny)


def loss64(A, Bt, targets):
    """(loss, lse, what the loss and the lse may be off, logits, what they may be off)."""
    M, K = A.shape
    Z = Bt.double() @ A.double().t()
    off = sum_error(Bt.double().abs() @ A.double().abs().t(), K)
    lse = torch.logsumexp(Z, 1)
    valid = (targets >= 0) & (targets < M)
    zt = Z.gather(1, targets.clamp(0, M - 1)[:, None])[:, 0]
    loss = torch.where(valid, lse - zt, torch.where(targets < 0, 0.0, float("nan")).double())
    # an exponential within 2^-22 and a step of its argument, at most 0.37 of which is left once it is weighted; one per
    # merge and addition, of which a token's sum goes through fewer than 20 + M / 32; then a logarithm and two roundings
    step = (20 + M / 32) * 2.0 ** -21 + 2.0 ** -22 * (lse.abs() + zt.abs() + 1)
    top = off.amax(1)
    return loss, lse, 2 * top + step, top + step, Z, off


def loss_grad64(A, Bt, targets, dloss, dtype, lse):
    """(dA, dB, what each may be off) with the lse that the call is given."""
    M, K = A.shape
    N = Bt.shape[0]
    _, _, _, _, Z, off = loss64(A, Bt, targets)
    half = HALF_STEP[dtype]
    g = torch.where(targets < 0, 0.0, dloss.double())
    arg = Z - lse.double()[:, None]
    p = torch.exp(arg)
    hot = torch.zeros_like(p)
    rows = torch.arange(N, device=A.device)
    ok = (targets >= 0) & (targets < M)
    hot[rows[ok], targets[ok]] = 1
    d = (p - hot) * g[:, None]
    wrong = p * (torch.expm1(off) + 2.0 ** -21 + arg.abs() * 2.0 ** -23) + 2.0 ** -24 * (p + hot)
    o = wrong * g.abs()[:, None]
    least = float(g.abs().max()) * 2.0 ** -38 if dtype == torch.float16 else 2.0 ** -130
    o = o + half * (d.abs() + o) + least * (g != 0)[:, None]
    x, W = Bt.double(), A.double()
    dA, dB = d.t() @ x, d @ W
    eA = o.t() @ x.abs() + sum_error((d.abs() + o).t() @ x.abs(), N)
    eB = o @ W.abs() + sum_error((d.abs() + o) @ W.abs(), M) + M * 2.0 ** -24 * 2.0 ** -10 * ((d.abs() + o) @ W.abs())
    tiny = torch.finfo(dtype).tiny
    return dA, dB, (half * dA.abs() + 1.01 * eA + tiny), (half * dB.abs() + 1.01 * eB + tiny)


def assert_within(got, ref, bound, what=""):
    """Everywhere |got - ref| <= bound; NaN in ref: not looked at."""
    at = ~torch.isnan(ref)
    bad = at & ~((got.double() - ref).abs() <= bound)
    worst = ((got.double() - ref).abs() / bound)[at]
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {int(at.sum())} outside, worst {float(worst.max())}"
