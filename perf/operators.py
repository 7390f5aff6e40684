"""The expert and 8-bit integer products, measured: what is called, on which inputs, and what each call computes.

Every operator here is in TN storage, as the library's other products are: the weights A are (M, K) row-major (one such matrix per
expert for the grouped products), the tokens Bt are (rows, K) row-major, and the result C^T is (rows, M) row-major.

  grouped   C^T[t] = A[e] Bt[t] for every row t of expert e's range [offsets[e], offsets[e + 1])
  grad_b    its gradient for the tokens:  dBt[t] = A[e]^T dC^T[t]
  grad_a    its gradient for the weights: dA[e] = sum over e's rows t of dC^T[t] (outer) Bt[t]
  i8        C^T[n, m] = scale_a[m] scale_b[n] sum_k A[m, k] Bt[n, k], A and Bt 8-bit integers
  i8_grouped  the same for every expert's rows, scale_a one row per expert
  quant     scale[r] = max_k |x[r, k]| / 127 and codes round(127 x[r, k] / max), ties to even
"""
import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token routed to eight of 32 experts: the weights of eight experts are read for eight rows
        {"name": "grouped_decode_bf16", "op": "grouped", "dtype": "bf16", "E": 32, "active": 8, "T": 8, "M": 2048, "K": 2048},
        # a serving batch's tokens, ragged over the experts, one expert without any
        {"name": "grouped_ragged_f16", "op": "grouped", "dtype": "f16", "E": 16, "active": 15, "T": 1021, "M": 4096, "K": 1024},
        # a training step's tokens through the wide projection of eight experts
        {"name": "grouped_large_bf16", "op": "grouped", "dtype": "bf16", "E": 8, "active": 8, "T": 16384, "M": 8192, "K": 4096},
        # the gradient for the tokens of many small experts
        {"name": "grad_b_ragged_bf16", "op": "grad_b", "dtype": "bf16", "E": 32, "active": 31, "T": 3001, "M": 1024, "K": 2048},
        # the gradient for the tokens of a training step's wide projection
        {"name": "grad_b_large_f16", "op": "grad_b", "dtype": "f16", "E": 8, "active": 8, "T": 8192, "M": 14336, "K": 4096},
        # the gradient for the weights of many small experts: every expert's matrix is written, also where no token went
        {"name": "grad_a_ragged_bf16", "op": "grad_a", "dtype": "bf16", "E": 32, "active": 30, "T": 3001, "M": 1024, "K": 2048},
        # the gradient for the weights of a training step
        {"name": "grad_a_large_f16", "op": "grad_a", "dtype": "f16", "E": 8, "active": 8, "T": 16384, "M": 4096, "K": 4096},
        # a decode step of sixteen sequences through one 8-bit layer
        {"name": "i8_decode_f16", "op": "i8", "dtype": "f16", "M": 8192, "N": 16, "K": 2048},
        # a prefill of 4096 tokens through one 8-bit layer
        {"name": "i8_large_bf16", "op": "i8", "dtype": "bf16", "M": 8192, "N": 4096, "K": 8192},
        # a serving batch's tokens through sixteen experts held in 8 bits
        {"name": "i8_grouped_bf16", "op": "i8_grouped", "dtype": "bf16", "E": 16, "active": 16, "T": 515, "M": 4096, "K": 2048},
        # the activations of a decode step, quantised for an 8-bit layer
        {"name": "quant_decode_bf16", "op": "quant", "dtype": "bf16", "rows": 16, "cols": 2048},
        # the activations of a long prefill
        {"name": "quant_large_bf16", "op": "quant", "dtype": "bf16", "rows": 16384, "cols": 8192},
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over the logarithm of [lo, hi]."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grad_b", "grad_a", "i8", "i8_grouped", "quant"])
    if op == "quant":
        rows = _log(rng, 1, 16384)
        return {"op": op, "dtype": rng.choice(["f16", "bf16", "f32"]), "rows": rows, "cols": _log(rng, 64, max(64, min(32768, (1 << 27) // rows)))}
    eight = op.startswith("i8")
    unit = rng.choice([1, 16, 64]) if eight else rng.choice([1, 8, 64])     # of M and K: most layers' widths are round, some are not
    width = lambda hi: max(unit, _log(rng, 128, hi) // unit * unit)  # noqa: E731
    dtype = rng.choice(["f16", "bf16"])
    if op == "i8":
        M, K = width(16384), width(16384)
        return {"op": op, "dtype": dtype, "M": M, "N": _log(rng, 1, max(1, min(8192, 270_000_000_000 // (M * K)))), "K": K}
    E = _log(rng, 2, 64)
    M = width(8192)
    K = width(max(128, min(8192, (1 << 28) // (E * M))))
    T = _log(rng, 1, max(1, min(16384, 500_000_000_000 // (M * K))))
    return {"op": op, "dtype": dtype, "E": E, "active": min(E, T, rng.choice([E, E, max(1, E - 1), max(1, E // 4)])), "T": T, "M": M, "K": K}


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

    def codes(*shape):      # what a quantiser leaves of normal values: the row's largest at 127, most within 40
        return (torch.randn(*shape, generator=g, device=dev) * 36).round_().clamp_(-127, 127).to(torch.int8)

    def scales(*shape):
        return (0.5 + torch.rand(*shape, generator=g, device=dev)) * 2.0 ** -9

    if op == "quant":
        x = normal(case["rows"], case["cols"])
        x *= torch.exp(torch.randn(case["rows"], 1, generator=g, device=dev)).to(dtype)     # tokens differ in size
        return {"case": case, "x": x}
    if op == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"case": case, "A": codes(M, K), "Bt": codes(N, K), "scale_a": scales(M), "scale_b": scales(N)}

    E, T, M, K = case["E"], case["T"], case["M"], case["K"]
    counts = _counts(case, np.random.RandomState(seed & 0x7FFFFFFF))
    ends = np.cumsum(counts)
    s = {"case": case, "offsets": torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32, device=dev)}
    # the same plan as rows of a padded batch: row p of active expert j is token slots[j, p] (where held[j, p]), token t is row back[t] of the batch
    which = np.flatnonzero(counts)
    longest = int(counts.max())
    at = np.arange(longest)[None, :]
    held = at < counts[which][:, None]
    start = (ends - counts)[which][:, None]
    s["active"] = torch.tensor(which, device=dev)
    s["slots"] = torch.tensor(np.where(held, start + at, 0), device=dev)
    s["held"] = torch.tensor(held, device=dev)
    s["back"] = torch.tensor(np.flatnonzero(held.reshape(-1)), device=dev)
    if op == "i8_grouped":
        return s | {"A": codes(E, M, K), "Bt": codes(T, K), "scale_a": scales(E, M), "scale_b": scales(T)}
    if op != "grad_a":
        s["A"] = normal(E, M, K, scale=K ** -0.5)
    if op != "grad_b":
        s["Bt"] = normal(T, K)
    if op != "grouped":
        s["dCt"] = normal(T, M)
    return s


def _own(s):
    import dense_gemm_tn_gb300 as tn
    op, dtype = s["case"]["op"], TYPES[s["case"]["dtype"]]
    if op == "grouped":
        return tn.tn_grouped(s["A"], s["Bt"], s["offsets"])
    if op == "grad_b":
        return tn.tn_grouped_grad_b(s["A"], s["dCt"], s["offsets"])
    if op == "grad_a":
        return tn.tn_grouped_grad_a(s["dCt"], s["Bt"], s["offsets"])
    if op == "i8":
        return tn.i8_tn(s["A"], s["Bt"], s["scale_a"], s["scale_b"], dtype=dtype)
    if op == "i8_grouped":
        return tn.i8_tn_grouped(s["A"], s["Bt"], s["scale_a"], s["scale_b"], s["offsets"], dtype=dtype)
    return tn.quantize_i8_rows(s["x"])


def run(s):
    if own:
        return _own(s)
    op, dtype = s["case"]["op"], TYPES[s["case"]["dtype"]]
    if op == "quant":
        x = s["x"].double()             # a value next to the border of two codes needs more than 32 bits
        top = x.abs().amax(1, keepdim=True)
        q = torch.where(top > 0, (x * 127 / top).round(), torch.zeros_like(x))
        return q.to(torch.int8), (top[:, 0] / 127).float()
    if op == "i8":
        return (s["Bt"].float() @ s["A"].float().t() * s["scale_a"] * s["scale_b"][:, None]).to(dtype)
    if op == "grouped":
        y = s["Bt"].float()[s["slots"]] @ s["A"][s["active"]].float().transpose(1, 2)
        return y.flatten(0, 1)[s["back"]].to(dtype)
    if op == "grad_b":
        y = s["dCt"].float()[s["slots"]] @ s["A"][s["active"]].float()
        return y.flatten(0, 1)[s["back"]].to(dtype)
    if op == "grad_a":
        rows = s["dCt"].float()[s["slots"]] * s["held"][..., None]
        dA = torch.zeros(s["case"]["E"], s["case"]["M"], s["case"]["K"], dtype=dtype, device=rows.device)
        dA[s["active"]] = (rows.transpose(1, 2) @ s["Bt"].float()[s["slots"]]).to(dtype)
        return dA
    y = s["Bt"].float()[s["slots"]] @ s["A"][s["active"]].float().transpose(1, 2) * s["scale_a"][s["active"]][:, None, :]
    return (y.flatten(0, 1)[s["back"]] * s["scale_b"][:, None]).to(dtype)


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (TYPES[case["dtype"]].itemsize + 1) + 4 * case["rows"], "flops": 3 * n}
    if op == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * (M + N), "flops": 2 * M * N * K}
    E, a, T, M, K = (case[k] for k in ("E", "active", "T", "M", "K"))
    weights, tokens, results = a * M * K, T * K, T * M
    size = {"grad_a": 2 * (tokens + results + E * M * K), "i8_grouped": weights + tokens + 2 * results + 4 * (a * M + T)}
    return {"bytes": size.get(op, 2 * (weights + tokens + results)) + 4 * (E + 1), "flops": 2 * T * M * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        codes, scale = [], []
        for x in s["x"].split(2048):
            x = x.double()
            top = x.abs().max(dim=1).values
            scale.append(top / 127.0)
            ratio = 127.0 * x / torch.clamp(top, min=torch.finfo(torch.float64).tiny)[:, None]
            codes.append(torch.round(ratio).to(torch.int8))
        return torch.cat(codes), torch.cat(scale)
    if op == "i8":
        out = torch.empty(case["N"], case["M"], dtype=torch.float64, device="cuda")
        A = s["A"].double()
        for n in range(0, case["N"], 1024):
            out[n:n + 1024] = torch.einsum("nk,mk->nm", s["Bt"][n:n + 1024].double(), A)
        return out * torch.outer(s["scale_b"].double(), s["scale_a"].double())
    bounds = s["offsets"].tolist()
    T, M, K = case["T"], case["M"], case["K"]
    out = torch.zeros(*{"grad_a": (case["E"], M, K), "grad_b": (T, K)}.get(op, (T, M)), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        if op == "grad_a":
            out[e] = torch.einsum("tm,tk->mk", s["dCt"][lo:hi].double(), s["Bt"][lo:hi].double())
        elif op == "grad_b":
            out[lo:hi] = torch.einsum("tm,mk->tk", s["dCt"][lo:hi].double(), s["A"][e].double())
        else:
            out[lo:hi] = torch.einsum("tk,mk->tm", s["Bt"][lo:hi].double(), s["A"][e].double())
            if op == "i8_grouped":
                out[lo:hi] *= torch.outer(s["scale_b"][lo:hi].double(), s["scale_a"][e].double())
    return out
