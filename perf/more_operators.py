"""The operators of decoding from 4-bit weights and of mixture-of-experts layers that are
measured: quantisation of weights to 4 bits with a scale (and a zero point) for each group
of a row and the values that such weights stand for, the product of a few rows with them,
and a whole mixture-of-experts layer for a few tokens: the router, its choice of experts,
their gated FFNs (weights in bf16 or in 4 bits) and the weighted sum.

Each case names one operator and its sizes.  `prepare` makes what a program holds before
the call, `run` makes one call, in elementary torch operations (`own` false) or through
the package (`own` true), and `exact` gives the same outputs in 64 bits.

A row of K weights in 4 bits is stored in blocks of 128 columns, 64 bytes each: column
32 i + 8 c + 2 n + o of a block (i, c, n < 4, o < 2) is nibble n (from the lowest) of the
16 bits at byte 8 (2 c + o) + 2 i.  A weight is (code - zero) * scale, with zero 8 where
there are no zero points; the columns behind K hold the zero point, the scales of groups
behind K are 0.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
BLOCK = 128


# ----------------------------------------------------------------------- cases


def listed():
    return [
        # a checkpoint's projection on its way into 4 bits, and back for a prompt's product
        {"name": "quantise: 8192 x 2048", "op": "quant", "N": 8192, "K": 2048, "w": "bf16",
         "group": 128, "zero": False, "out": "bf16"},
        # a matrix of odd sizes in fp32, small groups with zero points
        {"name": "quantise: 1001 x 1999, zero points", "op": "quant", "N": 1001, "K": 1999,
         "w": "f32", "group": 32, "zero": True, "out": "f32"},
        # a decode step of one sequence through one projection
        {"name": "4-bit product: 1 x 8192 x 2048", "op": "gemv", "T": 1, "N": 8192, "K": 2048,
         "group": 128, "zero": False, "out": "bf16"},
        # five drafted tokens through a projection with small groups and zero points
        {"name": "4-bit product: 5 x 2048 x 8192, zero points", "op": "gemv", "T": 5, "N": 2048,
         "K": 8192, "group": 32, "zero": True, "out": "f32"},
        # odd sizes
        {"name": "4-bit product: 13 x 1001 x 1999", "op": "gemv", "T": 13, "N": 1001, "K": 1999,
         "group": 64, "zero": True, "out": "bf16"},
        # a decode step of 64 sequences through an up projection
        {"name": "4-bit product: 64 x 9216 x 2304", "op": "gemv", "T": 64, "N": 9216, "K": 2304,
         "group": 128, "zero": False, "out": "bf16"},
        # a decode step of one sequence: experts with a sparse ReLU gate
        {"name": "experts: 1 token, bf16, sparse ReLU", "op": "moe", "T": 1, "D": 2048,
         "F": 1024, "E": 64, "k": 8, "act": "relu", "density": 0.01, "bits": 16, "out": "f32",
         "routed": False},
        # the same step with a dense activation and the weights in 4 bits
        {"name": "experts: 1 token, 4 bits, SiLU", "op": "moe", "T": 1, "D": 2048, "F": 1024,
         "E": 64, "k": 8, "act": "silu", "density": 0.5, "bits": 4, "group": 128, "zero": False,
         "out": "bf16", "routed": False},
        # a decode batch of eight sequences, sparse ReLU
        {"name": "experts: 8 tokens, bf16, sparse ReLU", "op": "moe", "T": 8, "D": 1536,
         "F": 768, "E": 128, "k": 8, "act": "relu", "density": 0.02, "bits": 16, "out": "f32",
         "routed": False},
        # a padded batch routed by the caller, odd sizes
        {"name": "experts: 13 tokens, routed, 4 bits", "op": "moe", "T": 13, "D": 1000, "F": 200,
         "E": 10, "k": 3, "act": "silu", "density": 0.5, "bits": 4, "group": 64, "zero": True,
         "out": "f32", "routed": True},
        # a decode batch of 64 sequences: every expert has tokens
        {"name": "experts: 64 tokens, 4 bits, ReLU", "op": "moe", "T": 64, "D": 2048, "F": 1024,
         "E": 64, "k": 8, "act": "relu", "density": 0.5, "bits": 4, "group": 128, "zero": False,
         "out": "f32", "routed": False},
        {"name": "experts: 64 tokens, bf16, SiLU", "op": "moe", "T": 64, "D": 2048, "F": 1024,
         "E": 64, "k": 8, "act": "silu", "density": 0.5, "bits": 16, "out": "bf16",
         "routed": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "gemv", "gemv", "moe", "moe", "moe"))
    group, zero = rng.choice((32, 64, 128)), rng.random() < 0.5
    out = rng.choice(("bf16", "f32"))
    if op in ("quant", "gemv"):
        n = _log(rng, 32, 16384)
        k = _log(rng, 32, min(16384, 9216 * 2304 // n))
        k = rng.choice((k, -(-k // 128) * 128))
        if op == "quant":
            return {"op": op, "N": n, "K": k, "w": rng.choice(("bf16", "f32")), "group": group,
                    "zero": zero, "out": out}
        return {"op": op, "T": _log(rng, 1, 64), "N": n, "K": k, "group": group, "zero": zero,
                "out": out}
    e = _log(rng, 4, 128)
    k = rng.randint(1, min(8, e))
    d = 8 * _log(rng, 8, 288)
    t = _log(rng, 1, 64)
    most = 64 * 1024 * 2048
    f = _log(rng, 32, min(2048, most // (d * e), 8 * most // (d * t * k)))
    case = {"op": op, "T": t, "D": d, "F": f, "E": e, "k": k, "act": rng.choice(("relu", "silu")),
            "density": rng.choice((0.01, 0.05, 0.5)), "bits": rng.choice((4, 16)), "out": out,
            "routed": rng.random() < 0.25}
    if case["bits"] == 4:
        case["group"], case["zero"] = group, zero
    return case


# ---------------------------------------------------------------------- inputs


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def _pack(code, fill):
    """Codes [..., K] and the code of a padded column [..., 1] as stored."""
    K = code.shape[-1]
    nb = -(-K // BLOCK)
    full = fill.expand(*code.shape[:-1], nb * BLOCK).clone()
    full[..., :K] = code
    # (i, c, n, o) -> (c, o, i, n), two nibbles a byte
    at = full.reshape(-1, nb, 4, 4, 4, 2).permute(0, 1, 3, 5, 2, 4)
    byte = at[..., 0::2] + 16 * at[..., 1::2]
    return byte.reshape(*code.shape[:-1], nb * 64).contiguous()


def _four_bits(w, group, zero):
    """Weights [..., K] as a checkpoint in 4 bits holds them: (codes, scales, zero points)."""
    *lead, K = w.shape
    n, held = -(-K // group), -(-K // BLOCK) * (BLOCK // group)
    p = torch.zeros((*lead, n * group), device=w.device)
    p[..., :K] = w
    p = p.view(*lead, n, group)
    if zero:
        lo, hi = p.amin(-1).clamp_max(0), p.amax(-1).clamp_min(0)
        s = ((hi - lo) / 15).to(torch.bfloat16)
        z = (-lo / s.float()).round().clamp(0, 15)
    else:
        s = (p.abs().amax(-1) / 7).to(torch.bfloat16)
        z = torch.full_like(s, 8, dtype=torch.float32)
    code = ((p / s.float()[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8)
    scale = torch.zeros((*lead, held), dtype=torch.bfloat16, device=w.device)
    scale[..., :n] = s
    zeros = torch.full((*lead, held), 8, dtype=torch.uint8, device=w.device)
    zeros[..., :n] = z.to(torch.uint8)
    return (_pack(code.view(*lead, n * group)[..., :K], zeros.new_full((*lead, 1), 8)), scale,
            zeros if zero else None)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "quant":
        # rows of different size, some weights far above the rest
        w = _normal(g, case["N"], case["K"]) * torch.exp(0.5 * _normal(g, case["N"], 1))
        w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.002, 8 * w, w)
        s["w"] = (w / math.sqrt(case["K"])).to(TYPES[case["w"]])
        return s
    if op == "gemv":
        s["x"] = _normal(g, case["T"], case["K"]).to(torch.bfloat16)
        s["w"] = _four_bits(_normal(g, case["N"], case["K"]) / math.sqrt(case["K"]),
                            case["group"], case["zero"])
        return s
    T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "k"))
    # features of some mean, against which the gates' weights stand so that a share
    # `density` of the gates is positive
    mean = 0.25
    s["x"] = (_normal(g, T, D) + mean).to(torch.bfloat16)
    shift = math.sqrt(2.0) * float(torch.erfinv(torch.tensor(2.0 * case["density"] - 1.0)))
    shift *= math.sqrt(1 + mean * mean) / (mean * D)
    weights = (_normal(g, E, F, D) / math.sqrt(D) + shift, _normal(g, E, F, D) / math.sqrt(D),
               _normal(g, E, F, D) / math.sqrt(F))
    if case["bits"] == 4:
        s["gate"], s["up"], s["down"] = (_four_bits(w, case["group"], case["zero"])
                                         for w in weights)
    else:
        s["gate"], s["up"], s["down"] = (w.to(torch.bfloat16) for w in weights)
    s["router"] = (1.5 * _normal(g, E, D) / math.sqrt(D)).to(torch.bfloat16)
    if case["routed"]:
        # another program's choice of experts; the last rows of the batch are padding
        order = torch.rand((T, E), generator=g, device="cuda").argsort(1)
        s["ids"] = order[:, :k].to(torch.int32)
        s["ids"][T - T // 4:] = -1
        s["weights"] = torch.rand((T, k), generator=g, device="cuda")
    return s


# ------------------------------------------------------------------------- run


def _values(w, K, group):
    """What weights in 4 bits stand for, in fp32."""
    code, scale, zero = w
    lead, nb = code.shape[:-1], code.shape[-1] // 64
    nibble = torch.stack((code & 15, code >> 4), -1).view(-1, nb, 4, 2, 4, 4)  # (c, o, i, n)
    q = nibble.permute(0, 1, 4, 2, 5, 3).reshape(*lead, nb * BLOCK).float()
    q = q - (8.0 if zero is None else zero.float().repeat_interleave(group, -1))
    return (q * scale.float().repeat_interleave(group, -1))[..., :K]


def _plain_quant(s):
    w, group, K = s["w"].float(), s["group"], s["K"]
    n = -(-K // group)
    p = torch.nn.functional.pad(w, (0, n * group - K)).view(s["N"], n, group)
    if s["zero"]:
        lo, hi = p.amin(-1).clamp_max(0), p.amax(-1).clamp_min(0)
        # (in 64 bits: a product with 1/15 in 32 would round some scales the other way)
        scale = ((hi - lo).double() / 15).float().to(torch.bfloat16)
        z = (-lo.double() / scale.double()).round().clamp(0, 15)
    else:
        scale = (p.abs().amax(-1).double() / 7).float().to(torch.bfloat16)
        z = torch.full_like(scale, 8, dtype=torch.float64)
    # in 64 bits: a quotient next to a border between two codes
    q = ((p.double() / scale.double()[..., None]).round() + z[..., None]).clamp(0, 15)
    v = (q - z[..., None]).float() * scale.float()[..., None]
    out = {"w": v.view(s["N"], n * group)[:, :K].to(TYPES[s["out"]]), "scale": scale}
    if s["zero"]:
        out["zero"] = z.to(torch.uint8)
    return out


def _plain_route(s):
    # the logits in 64 bits: values next to the border between two experts
    logits = s["x"].double() @ s["router"].double().t()
    ids = logits.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    top = logits.gather(1, ids).float()
    p = torch.exp(top - top[:, :1])
    return ids.to(torch.int32), p / p.sum(1, keepdim=True)


def _plain_moe(s):
    x, T, D, F, E, k = s["x"].float(), s["T"], s["D"], s["F"], s["E"], s["k"]
    ids, weights = (s["ids"], s["weights"]) if s["routed"] else _plain_route(s)
    live = ids >= 0
    at = ids.clamp_min(0).long()
    share = torch.where(live, weights, torch.zeros_like(weights))

    def wide(w):
        return _values(w, D, s["group"]) if s["bits"] == 4 else w.float()

    if T * k < E:   # the chosen experts' weights, one by one

        def chosen(w):
            return wide(tuple(None if v is None else v[at] for v in w)
                        if s["bits"] == 4 else w[at])

        z = (chosen(s["gate"]) * x[:, None, None, :]).sum(-1)
        u = (chosen(s["up"]) * x[:, None, None, :]).sum(-1)
    else:           # every expert for every token
        share = torch.zeros((T, E), device=x.device).scatter_add_(1, at, share)
        z = (x @ wide(s["gate"]).view(E * F, D).t()).view(T, E, F)
        u = (x @ wide(s["up"]).view(E * F, D).t()).view(T, E, F)
    a = torch.where(z <= 0, torch.zeros_like(z), z) if s["act"] == "relu" else (
        z / (1 + torch.exp(-z)))
    h = a * u * share[:, :, None]
    if T * k < E:
        y = (h[..., None] * chosen(s["down"])).sum((1, 2))
    else:
        y = h.view(T, E * F) @ wide(s["down"]).view(E * F, D)
    out = {"y": y.to(TYPES[s["out"]])}
    if not s["routed"]:
        out["ids"], out["weights"] = ids, weights
    return out


def _plain(s):
    if s["op"] == "quant":
        return _plain_quant(s)
    if s["op"] == "gemv":
        return (s["x"].float() @ _values(s["w"], s["K"], s["group"]).t()).to(TYPES[s["out"]])
    return _plain_moe(s)


def run(state):
    if not own:
        return _plain(state)
    import activation_sparse_gated_gate_gb300 as tw

    s = state
    if s["op"] == "quant":
        w = tw.twell_quant_int4(s["w"], group=s["group"], zero_points=s["zero"])
        n = -(-s["K"] // s["group"])
        out = {"w": tw.twell_dequant_int4(w, dtype=TYPES[s["out"]]), "scale": w.scale[:, :n]}
        if s["zero"]:
            out["zero"] = w.zero[:, :n]
        return out
    if s["op"] == "gemv":
        return tw.twell_gemv_int4(s["x"], tw.Int4(*s["w"], s["K"], s["group"]),
                                  dtype=TYPES[s["out"]])
    gate, up, down = s["gate"], s["up"], s["down"]
    if s["bits"] == 4:
        gate, up, down = (tw.Int4(*w, s["D"], s["group"]) for w in (gate, up, down))
    if s["routed"]:
        o = tw.twell_moe_decode(s["x"], None, gate, up, down, act=s["act"], ids=s["ids"],
                                weights=s["weights"], dtype=TYPES[s["out"]])
        return {"y": o.y}
    o = tw.twell_moe_decode(s["x"], s["router"], gate, up, down, top_k=s["k"], act=s["act"],
                            dtype=TYPES[s["out"]])
    return {"y": o.y, "ids": o.ids, "weights": o.weights}


# ------------------------------------------------------------------ work, exact


def _row_bytes(K, group, zero):
    return K / 2 + -(-K // group) * (3 if zero else 2)


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["N"] * case["K"]
        packed = case["N"] * _row_bytes(case["K"], case["group"], case["zero"])
        # the weights once, what is stored once; their values once
        return {"bytes": n * (BYTES[case["w"]] + BYTES[case["out"]]) + packed, "flops": 4 * n}
    if op == "gemv":
        T, N, K = case["T"], case["N"], case["K"]
        b = N * _row_bytes(K, case["group"], case["zero"]) + 2 * T * K
        return {"bytes": b + T * N * BYTES[case["out"]], "flops": 2 * T * N * K}
    T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "k"))
    live = T - T // 4 if case["routed"] else T
    row = _row_bytes(D, case["group"], case["zero"]) if case["bits"] == 4 else 2 * D
    hit = E * (1 - (1 - k / E) ** live)                     # experts with some token
    per = live * k / hit if hit else 0.0                    # tokens of such an expert
    p = case["density"] if case["act"] == "relu" else 1.0   # gates that are not zero
    rows = 1 + 2 * (1 - (1 - p) ** per)   # the gate's, and up and down where some token's is not
    b = hit * F * rows * row + T * D * (2 + BYTES[case["out"]]) + 8 * T * k
    flops = 2 * live * k * F * D * (1 + 2 * p)
    if not case["routed"]:
        b, flops = b + 2 * E * D, flops + 2 * T * E * D
    return {"bytes": b, "flops": flops}


def _column(K, dev):
    """Byte and nibble of each column of a row in 4 bits."""
    j = torch.arange(K, device=dev)
    r = j % 128
    o, n, c, i = r % 2, r // 2 % 4, r // 8 % 4, r // 32
    return j // 128 * 64 + 8 * (2 * c + o) + 2 * i + n // 2, 4 * (n % 2)


def _wide(w, K, group):
    """The weights in 64 bits that codes, scales and zero points stand for."""
    code, scale, zero = w
    byte, shift = _column(K, code.device)
    q = (code[..., byte].to(torch.int64) >> shift) & 15
    at = torch.arange(K, device=code.device) // group
    z = 8 if zero is None else zero[..., at].to(torch.int64)
    return (q - z).to(torch.float64) * scale[..., at].to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "quant":
        w, group = s["w"].to(f64), case["group"]
        scales, zeros, values = [], [], []
        for k0 in range(0, case["K"], group):
            v = w[:, k0:k0 + group]
            if case["zero"]:
                top = torch.maximum(v.max(1).values, torch.zeros((), dtype=f64, device=v.device))
                low = torch.minimum(v.min(1).values, torch.zeros((), dtype=f64, device=v.device))
                # the scale is defined by its rounding: to fp32, to bf16
                sc = ((top - low).to(torch.float32).to(f64) / 15)
            else:
                top, low, sc = None, None, v.abs().max(1).values / 7
            sc = sc.to(torch.float32).to(torch.bfloat16).to(f64)
            z = (torch.round(-low / sc).clamp(0, 15) if case["zero"]
                 else torch.full_like(sc, 8.0))
            code = (torch.round(v / sc[:, None]) + z[:, None]).clamp(0, 15)
            values.append((code - z[:, None]) * sc[:, None])
            scales.append(sc)
            zeros.append(z)
        out = {"w": torch.cat(values, 1), "scale": torch.stack(scales, 1)}
        if case["zero"]:
            out["zero"] = torch.stack(zeros, 1).to(torch.uint8)
        return out
    if op == "gemv":
        return torch.einsum("tk,nk->tn", s["x"].to(f64), _wide(s["w"], case["K"], case["group"]))
    T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "k"))
    x, out = s["x"].to(f64), {}
    if case["routed"]:
        ids, weights = s["ids"].long(), s["weights"].to(f64)
    else:
        prob = torch.softmax(torch.einsum("td,ed->te", x, s["router"].to(f64)), 1)
        ids = torch.argsort(prob, dim=1, descending=True, stable=True)[:, :k]
        weights = torch.take_along_dim(prob, ids, 1)
        weights = weights / weights.sum(1, keepdim=True)
        out["ids"], out["weights"] = ids.to(torch.int32), weights

    def of(w, e):
        if case["bits"] == 16:
            return w[e].to(f64)
        return _wide(tuple(None if v is None else v[e] for v in w), D, case["group"])

    y = torch.zeros((T, D), dtype=f64, device=x.device)
    for e in range(E):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        z = torch.einsum("td,fd->tf", x[t], of(s["gate"], e))
        u = torch.einsum("td,fd->tf", x[t], of(s["up"], e))
        a = torch.relu(z) if case["act"] == "relu" else z * torch.sigmoid(z)
        y.index_add_(0, t, torch.einsum("tf,fd->td", a * u * weights[t, slot][:, None],
                                        of(s["down"], e)))
    return {"y": y, **out}
