"""Operators of a language model around the library's products, measured: what is called, on which inputs, and what each call computes.

All are in TN storage: the weights A are row-major (one matrix per expert where there are experts), the tokens Bt are (rows, K) row-major, results are
(rows, M) row-major.

  gated        P = Bt[t] A[e]^T of 2 M rows (M gate rows, then M up rows); H = act(P_gate) * P_up. Without experts, or for every row of expert e's range
  gated_train  the same and its backward pass: dP_gate = dH P_up act'(P_gate), dP_up = dH act(P_gate), dBt = dP A, dA = dP^T Bt
  ce           softmax cross entropy over a vocabulary of M: Z = Bt A^T, lse = log sum exp Z, loss = lse - Z[target]; 0 where the target is negative
  ce_train     the same and its gradients: d = dloss (exp(Z - lse) - [m = target]), dBt = d A, dA = d^T Bt
  w4           C^T[n, m] = sum over groups g of scale[m, g] sum over k in g of q[m, k] Bt[n, k], q 4-bit integers, two to a byte, the even k in the low half
  quant_w4     scale[r, g] = max |x[r, k in g]| / 7 in 16 bits, q[r, k] = round(x / scale) within -8 .. 7, ties to even
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one new token through the gate and up projections of a dense layer: 235 MB of weights for one row
        {"name": "gated_decode_bf16", "op": "gated", "dtype": "bf16", "act": "silu", "E": 1, "active": 1, "T": 1, "M": 14336, "K": 4096},
        # a serving batch's tokens, ragged over the experts, one expert without any
        {"name": "gated_experts_f16", "op": "gated", "dtype": "f16", "act": "gelu_tanh", "E": 16, "active": 15, "T": 1021, "M": 2048, "K": 1024},
        # a prompt of 4096 tokens through a dense layer
        {"name": "gated_prefill_bf16", "op": "gated", "dtype": "bf16", "act": "silu", "E": 1, "active": 1, "T": 4096, "M": 14336, "K": 4096},
        # a training step's tokens through small experts, one without any: its gradient is zeros
        {"name": "gated_train_experts_bf16", "op": "gated_train", "dtype": "bf16", "act": "gelu", "E": 8, "active": 7, "T": 3001, "M": 1024, "K": 2048},
        # a training step through a dense layer
        {"name": "gated_train_f16", "op": "gated_train", "dtype": "f16", "act": "silu", "E": 1, "active": 1, "T": 4096, "M": 14336, "K": 4096},
        # the loss of one short text, as an evaluation takes it, over an odd vocabulary
        {"name": "ce_eval_bf16", "op": "ce", "dtype": "bf16", "N": 257, "M": 50021, "K": 2048},
        # a small training step over an odd vocabulary, a few tokens ignored
        {"name": "ce_train_ragged_f16", "op": "ce_train", "dtype": "f16", "N": 1021, "M": 32003, "K": 1024},
        # a training step of 4096 tokens over 65536 words
        {"name": "ce_train_large_bf16", "op": "ce_train", "dtype": "bf16", "N": 4096, "M": 65536, "K": 4096},
        # one new token through a layer held in 4 bits
        {"name": "w4_decode_bf16", "op": "w4", "dtype": "bf16", "N": 1, "M": 8192, "K": 8192, "group": 128},
        # sixteen sequences' new tokens through a wide layer held in 4 bits
        {"name": "w4_batch_f16", "op": "w4", "dtype": "f16", "N": 16, "M": 28672, "K": 4096, "group": 64},
        # a small layer quantised
        {"name": "quant_w4_small_f16", "op": "quant_w4", "dtype": "f16", "scales": "f16", "rows": 256, "cols": 4096, "group": 32},
        # a large layer quantised
        {"name": "quant_w4_large_bf16", "op": "quant_w4", "dtype": "bf16", "scales": "bf16", "rows": 8192, "cols": 8192, "group": 128},
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over the logarithm of [lo, hi]."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["gated", "gated_train", "gated_train", "ce", "ce_train", "ce_train", "w4", "w4", "quant_w4"])
    unit = rng.choice([1, 8, 64])                               # of the widths: most layers' are round, some are not
    width = lambda lo, hi: max(unit, _log(rng, lo, hi) // unit * unit)  # noqa: E731
    dtype = rng.choice(["f16", "bf16"])
    if op == "quant_w4":
        rows, scales = width(1, 28672), dtype
        dtype = rng.choice([dtype, dtype, "f32"])
        return {"op": op, "dtype": dtype, "scales": scales, "rows": rows, "cols": width(64, max(64, min(16384, (1 << 26) // rows))), "group": rng.choice([32, 64, 128])}
    if op == "w4":
        M, K = width(64, 28672), width(64, 16384)
        return {"op": op, "dtype": dtype, "N": _log(rng, 1, 64), "M": M, "K": K, "group": rng.choice([32, 64, 128])}
    if op.startswith("ce"):
        M, K = width(1000, 131072), width(64, 8192)
        return {"op": op, "dtype": dtype, "N": _log(rng, 1, max(1, min(8192, 1_000_000_000_000 // (M * K)))), "M": M, "K": K}
    E = rng.choice([1, 1, _log(rng, 2, 32)])
    M = width(64, 14336)
    K = width(64, max(64, min(8192, (1 << 27) // (E * M))))
    T = _log(rng, 1, max(1, min(8192, 240_000_000_000 // (M * K))))
    return {"op": op, "dtype": dtype, "act": rng.choice(["silu", "gelu", "gelu_tanh"]), "E": E, "active": min(E, T, rng.choice([E, max(1, E - 1), max(1, E // 4)])), "T": T, "M": M,
            "K": K}


def _counts(case, rs):
    """Rows of each expert: `active` of them have at least one, the rest of the rows fall where the router's preferences say."""
    E, active, T = case["E"], case["active"], case["T"]
    which = rs.permutation(E)[:active]
    like = 0.5 + rs.random_sample(active)
    counts = np.zeros(E, np.int64)
    counts[which] = 1 + rs.multinomial(T - active, like / like.sum())
    return counts


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, dtype = case["op"], TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(to)

    if op == "quant_w4":
        x = normal(case["rows"], case["cols"], scale=case["cols"] ** -0.5)
        x *= torch.exp(0.5 * torch.randn(case["rows"], 1, generator=g, device=dev)).to(dtype)       # channels differ in size
        return {"case": case, "x": x}
    if op == "w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        A = torch.randint(0, 256, (M, (K + 1) // 2), generator=g, device=dev, dtype=torch.uint8)
        scale = ((0.5 + torch.rand(M, -(-K // G), generator=g, device=dev)) * (0.2 * K ** -0.5)).to(dtype)
        return {"case": case, "A": A, "scale": scale, "Bt": normal(N, K)}
    if op.startswith("ce"):
        N, M, K = case["N"], case["M"], case["K"]
        s = {"case": case, "A": normal(M, K, scale=2.5 * K ** -0.5), "Bt": normal(N, K)}            # logits of a few units, as a model in training has
        u = torch.rand(N, generator=g, device=dev, dtype=torch.float64)
        targets = torch.exp(u * math.log(M)).long().clamp_(max=M - 1)                               # few words make up most of a text
        s["targets"] = torch.where(torch.rand(N, generator=g, device=dev) < 0.05, -100, targets)    # padding and prompts are ignored
        valid = s["targets"] >= 0
        s["dloss"] = valid.float() / valid.sum().clamp_(min=1)                                      # of the mean loss
        return s

    E, T, M, K = case["E"], case["T"], case["M"], case["K"]
    counts = _counts(case, np.random.RandomState(seed & 0x7FFFFFFF))
    ends = np.cumsum(counts)
    s = {"case": case, "A": normal(E, 2 * M, K, scale=K ** -0.5), "Bt": normal(T, K)}
    s["offsets"] = torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32, device=dev) if E > 1 else None
    # the same plan as rows of a padded batch: row p of active expert j is token slots[j, p] (where held[j, p]), token t is row back[t] of the batch
    which = np.flatnonzero(counts)
    at = np.arange(int(counts.max()))[None, :]
    held = at < counts[which][:, None]
    start = (ends - counts)[which][:, None]
    s["counts"] = [int(c) for c in counts]
    s["active"] = torch.tensor(which, device=dev)
    s["slots"] = torch.tensor(np.where(held, start + at, 0), device=dev)
    s["held"] = torch.tensor(held, device=dev)
    s["back"] = torch.tensor(np.flatnonzero(held.reshape(-1)), device=dev)
    if op == "gated_train":
        s["dHt"] = normal(T, M)
    return s


def _own(s):
    import dense_gemm_tn_gb300 as tn
    case = s["case"]
    op = case["op"]
    if op == "quant_w4":
        q, scale = tn.quantize_w4_rows(s["x"], case["group"], dtype=TYPES[case["scales"]])
        return _codes(q, case["cols"]), scale
    if op == "w4":
        return tn.w4_tn(s["A"], s["Bt"], s["scale"], case["group"])
    if op.startswith("ce"):
        loss, lse = tn.tn_cross_entropy(s["A"], s["Bt"], s["targets"])
        if op == "ce":
            return loss, lse
        dA, dBt = tn.tn_cross_entropy_grad(s["A"], s["Bt"], s["targets"], lse, s["dloss"])
        return loss, dA, dBt
    A = s["A"] if s["offsets"] is not None else s["A"][0]
    if op == "gated":
        return tn.tn_gated(A, s["Bt"], s["offsets"], act=case["act"])
    H, P = tn.tn_gated(A, s["Bt"], s["offsets"], act=case["act"], keep=True)
    dA, dBt = tn.tn_gated_grad(A, s["Bt"], P, s["dHt"], s["offsets"], act=case["act"])
    return H, dA.view(s["A"].shape), dBt


def _codes(q, cols):
    """The integers that packed 4-bit codes stand for."""
    q = q.view(torch.int8)
    return torch.stack(((q << 4) >> 4, q >> 4), -1).flatten(1)[:, :cols]


def _act(x, kind):
    """(act(x), act'(x))."""
    if kind == "silu":
        y = 1 / (1 + torch.exp(-x))
        return x * y, y * (1 + x * (1 - y))
    if kind == "gelu":
        y = 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
        return x * y, y + x * torch.exp(-0.5 * x * x) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    op = case["op"]
    if op == "quant_w4":
        rows, cols, G = case["rows"], case["cols"], case["group"]
        x = torch.zeros(rows, -(-cols // G) * G, device=s["x"].device, dtype=torch.float64)     # a value next to the border of two codes needs more than 32 bits
        x[:, :cols] = s["x"]
        x = x.view(rows, -1, G)
        scale = (x.abs().amax(2).float() / 7).to(TYPES[case["scales"]])
        by = scale.double()[..., None]
        q = torch.where(by > 0, (x / by).round().clamp(-8, 7), torch.zeros_like(x))
        return q.to(torch.int8).flatten(1)[:, :cols], scale
    if op == "w4":
        K, G = case["K"], case["group"]
        W = _codes(s["A"], K).float() * s["scale"].float()[:, torch.arange(K, device=s["A"].device) // G]
        return (s["Bt"].float() @ W.t()).to(s["Bt"].dtype)
    if op.startswith("ce"):
        A, Bt = s["A"].float(), s["Bt"].float()
        Z = Bt @ A.t()
        top = Z.amax(1, keepdim=True)
        lse = top + torch.log(torch.exp(Z - top).sum(1, keepdim=True))
        valid = s["targets"] >= 0
        row, at = torch.arange(case["N"], device=A.device), s["targets"].clamp(min=0)
        loss = torch.where(valid, lse[:, 0] - Z[row, at], torch.zeros_like(lse[:, 0]))
        if op == "ce":
            return loss, lse[:, 0]
        d = torch.exp(Z - lse)
        d[row, at] -= 1
        d *= torch.where(valid, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
        return loss, (d.t() @ Bt).to(s["A"].dtype), (d @ A).to(s["Bt"].dtype)

    dtype, M = s["A"].dtype, case["M"]
    A, Bt = s["A"][s["active"]].float(), s["Bt"].float()[s["slots"]]
    P = Bt @ A.transpose(1, 2)
    a, da = _act(P[..., :M], case["act"])
    H = (a * P[..., M:]).flatten(0, 1)[s["back"]].to(dtype)
    if op == "gated":
        return H
    dH = s["dHt"].float()[s["slots"]] * s["held"][..., None]
    dP = torch.cat((dH * P[..., M:] * da, dH * a), 2)
    dA = torch.zeros_like(s["A"])
    dA[s["active"]] = (dP.transpose(1, 2) @ Bt).to(dtype)
    return H, dA, (dP @ A).flatten(0, 1)[s["back"]].to(dtype)


def work(case):
    op = case["op"]
    if op == "quant_w4":
        n, groups = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // case["group"])
        return {"bytes": n * TYPES[case["dtype"]].itemsize + (n + 1) // 2 + 2 * groups, "flops": 3 * n}
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * ((K + 1) // 2) + 2 * M * -(-K // case["group"]) + 2 * N * (K + M), "flops": 2 * M * N * K}
    if op.startswith("ce"):
        N, M, K = case["N"], case["M"], case["K"]
        train = op == "ce_train"
        return {"bytes": 2 * (M + N) * K * (2 if train else 1) + N * (8 + 8), "flops": 2 * M * N * K * (3 if train else 1)}
    E, a, T, M, K = (case[k] for k in ("E", "active", "T", "M", "K"))
    if op == "gated":
        return {"bytes": 2 * (2 * a * M * K + T * K + T * M), "flops": 4 * T * M * K}
    return {"bytes": 2 * (2 * (a + E) * M * K + 2 * T * K + 2 * T * M), "flops": 12 * T * M * K}


def _exact_gated(case, s):
    counts, M, kind = s["counts"], case["M"], case["act"]
    H = torch.empty(case["T"], M, dtype=torch.float64, device="cuda")
    train = case["op"] == "gated_train"
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda") if train else None
    dB = torch.empty(s["Bt"].shape, dtype=torch.float64, device="cuda") if train else None
    lo = 0
    for e, n in enumerate(counts):
        rows = slice(lo, lo + n)
        lo += n
        if n == 0:
            continue
        x, W = s["Bt"][rows].double(), s["A"][e].double()
        gate, up = x @ W[:M].T, x @ W[M:].T
        if kind == "silu":
            sig = torch.sigmoid(gate)
            act, slope = gate * sig, sig + gate * sig * (1 - sig)
        elif kind == "gelu":
            cdf = 0.5 * torch.erfc(-gate / math.sqrt(2))
            act, slope = gate * cdf, cdf + gate * torch.exp(-gate ** 2 / 2) / math.sqrt(2 * math.pi)
        else:       # 1 + tanh(z) = 2 sigmoid(2 z)
            z2 = 2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
            sig = torch.sigmoid(z2)
            act = gate * sig
            slope = sig + gate * sig * (1 - sig) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * gate ** 2)
        H[rows] = act * up
        if not train:
            continue
        dh = s["dHt"][rows].double()
        dgate, dup = dh * up * slope, dh * act
        dA[e, :M], dA[e, M:] = dgate.T @ x, dup.T @ x
        dB[rows] = dgate @ W[:M] + dup @ W[M:]
    return (H, dA, dB) if train else H


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("gated"):
        return _exact_gated(case, s)
    if op == "quant_w4":
        scale = torch.stack([part.double().abs().max(dim=1).values / 7.0 for part in s["x"].split(case["group"], dim=1)], dim=1)
        return None, scale
    if op == "w4":
        K, G = case["K"], case["group"]
        out = torch.zeros(case["N"], case["M"], dtype=torch.float64, device="cuda")
        codes = torch.empty(case["M"], 2 * s["A"].shape[1], dtype=torch.float64, device="cuda")
        codes[:, 0::2], codes[:, 1::2] = (s["A"] % 16).double(), (s["A"] // 16).double()
        codes -= 16.0 * (codes >= 8)
        for i, k in enumerate(range(0, K, G)):
            end = min(k + G, K)
            out += s["Bt"][:, k:end].double() @ codes[:, k:end].T * s["scale"][:, i].double()
        return out
    A, train = s["A"].double(), op == "ce_train"
    loss, lse = [], []
    dA = torch.zeros_like(A) if train else None
    dB = []
    for n in range(0, case["N"], 1024):
        x, t, g = s["Bt"][n:n + 1024].double(), s["targets"][n:n + 1024], s["dloss"][n:n + 1024].double()
        logp = torch.einsum("nk,mk->nm", x, A)
        l = torch.logsumexp(logp, 1)
        lse.append(l)
        logp -= l[:, None]
        ignored = t < 0
        loss.append(torch.where(ignored, 0.0, -logp.gather(1, t.clamp(min=0)[:, None])[:, 0]))
        if train:
            p = logp.exp_()
            p.scatter_add_(1, t.clamp(min=0)[:, None], -torch.ones(len(t), 1, dtype=torch.float64, device="cuda"))
            p[ignored] = 0
            p *= g[:, None]
            dA += p.T @ x
            dB.append(p @ A)
    loss = torch.cat(loss)
    return (loss, dA, torch.cat(dB)) if train else (loss, torch.cat(lse))
