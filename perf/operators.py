"""The operators around the sparse FFN that are measured: residual addition with
root-mean-square norm (forward and backward), quantisation to 8-bit floating point
(e4m3) with a scale for each block of 128, the matrix product of such operands, and
the sparse FFN whose gate is such a product.

Each case names one operator and its sizes.  `prepare` makes what a program holds
before the call, `run` makes one call, in elementary torch operations (`own` false) or
through the package (`own` true), and `exact` gives the same outputs in 64 bits.
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -64   # a block of smaller magnitude is scaled as if it reached this
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ----------------------------------------------------------------------- cases


def listed():
    return [
        # a decode step of four sequences: the projection's output joins the residual
        # stream, its norm goes to the FFN (bf16) and to the gate (8 bits)
        {"name": "norm: decode, 4 x 2048", "op": "norm", "T": 4, "D": 2048, "x": "bf16",
         "r": "bf16", "w": "bf16", "fp8": True, "rstd": False},
        # a prompt: the FFN's fp32 output joins an fp32 stream, both kinds of output
        {"name": "norm: prompt, 8192 x 1536", "op": "norm", "T": 8192, "D": 1536, "x": "f32",
         "r": "f32", "w": "f32", "fp8": True, "rstd": False},
        # a training step's forward: fp32 stream, bf16 output, statistics kept
        {"name": "norm: training, 16384 x 2304", "op": "norm", "T": 16384, "D": 2304, "x": "f32",
         "r": "f32", "w": "f32", "fp8": False, "rstd": True},
        # fine-tuning on a ragged batch of short texts; rows of an odd length
        {"name": "norm gradient: 777 x 1001", "op": "norm_bwd", "T": 777, "D": 1001, "x": "bf16",
         "dy": "bf16", "w": "bf16"},
        # a training step's backward, the stream's own gradient added
        {"name": "norm gradient: training, 16384 x 2304", "op": "norm_bwd", "T": 16384, "D": 2304,
         "x": "f32", "dy": "bf16", "w": "f32"},
        # activations of a prompt on their way into an 8-bit product
        {"name": "quantise: prompt, 8192 x 2048", "op": "quant", "R": 8192, "C": 2048, "x": "bf16",
         "block": 1, "both": False},
        # a training step's output gradient, along both axes (for dX and for dW)
        {"name": "quantise: both ways, 16384 x 2304", "op": "quant", "R": 16384, "C": 2304,
         "x": "bf16", "block": 1, "both": True},
        # a decode step of four sequences through one dense projection
        {"name": "product: decode, 4 x 8192 x 2048", "op": "gemm", "M": 4, "N": 8192, "K": 2048,
         "b_block": 128, "out": "bf16"},
        # a prompt through the same kind of projection
        {"name": "product: prompt, 8192 x 6144 x 1536", "op": "gemm", "M": 8192, "N": 6144,
         "K": 1536, "b_block": 128, "out": "bf16"},
        # a weight gradient: sums over the tokens, scales along them on both sides, fp32
        {"name": "product: dW, 9216 x 2304 x 16384", "op": "gemm", "M": 9216, "N": 2304,
         "K": 16384, "b_block": 1, "out": "f32"},
        # sparse FFN with an 8-bit gate, a decode batch
        {"name": "gate: decode, 16 x 2048 x 8192", "op": "gate", "T": 16, "D": 2048, "F": 8192,
         "density": 0.005},
        # sparse FFN with an 8-bit gate, a prompt
        {"name": "gate: prompt, 8192 x 1536 x 6144", "op": "gate", "T": 8192, "D": 1536,
         "F": 6144, "density": 0.01},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "quant", "gemm", "gate"))
    if op in ("norm", "norm_bwd", "quant"):
        # widths of the models the library is used for, and odd ones; rows within the
        # largest listed case's
        wide = rng.choice((0, 0, 1))
        d = _log(rng, 64, 9216) if wide else 8 * _log(rng, 8, 512)
        t = _log(rng, 1, max(1, min(16384, 16384 * 2304 // d)))
        if op == "norm":
            return {"op": op, "T": t, "D": d, "x": rng.choice(("bf16", "f32")),
                    "r": rng.choice(("bf16", "f32")), "w": rng.choice(("bf16", "f32")),
                    "fp8": rng.random() < 0.5, "rstd": rng.random() < 0.5}
        if op == "norm_bwd":
            return {"op": op, "T": t, "D": d, "x": rng.choice(("bf16", "f32")),
                    "dy": rng.choice(("bf16", "f32")), "w": rng.choice(("bf16", "f32"))}
        block = rng.choice((1, 1, 128))
        return {"op": op, "R": t, "C": d, "x": rng.choice(("bf16", "f32")), "block": block,
                "both": rng.random() < 0.5}
    if op == "gemm":
        m, n = _log(rng, 1, 16384), 8 * _log(rng, 16, 1152)
        k = _log(rng, 64, min(16384, int(9216 * 2304 * 16384 / (m * n))))
        block = rng.choice((128, 128, 1))
        return {"op": op, "M": m, "N": n, "K": k, "b_block": block,
                "out": rng.choice(("bf16", "bf16", "f32"))}
    d = 64 * rng.randint(2, 36)
    f = 128 * rng.randint(8, 72)
    t = _log(rng, 1, min(8192, int(8192 * 1536 * 6144 / (d * f))))
    return {"op": op, "T": t, "D": d, "F": f, "density": rng.choice((0.005, 0.01, 0.02))}


# ---------------------------------------------------------------------- inputs


def _quantised(x, block):
    """e4m3 values and scales of x [R][C], a block of `block` rows by 128 columns each
    (how a checkpoint or the operator before this one left them)."""
    R, C = x.shape
    nr, nc = -(-R // block), -(-C // BLOCK)
    p = torch.zeros((nr * block, nc * BLOCK), dtype=torch.float32, device=x.device)
    p[:R, :C] = x
    p = p.view(nr, block, nc, BLOCK)
    amax = p.abs().amax(dim=(1, 3)).clamp_min(AMAX_MIN)
    q = (p * (E4M3_MAX / amax)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.view(nr * block, nc * BLOCK)[:R, :C].to(torch.float8_e4m3fn)
    # rows on 16-byte boundaries
    held = torch.zeros((R, -(-C // 16) * 16), dtype=torch.uint8, device=x.device)
    held[:, :C] = q.view(torch.uint8)
    return held.view(torch.float8_e4m3fn)[:, :C], amax / E4M3_MAX


def _stream(g, T, D):
    """Rows as they stand in a residual stream: a few features far above the rest, and
    rows of different size."""
    dev = g.device
    feature = torch.ones(D, device=dev)
    feature[torch.randint(0, D, (max(1, D // 200),), generator=g, device=dev)] = 20.0
    row = torch.exp(0.5 * torch.randn((T, 1), generator=g, device=dev))
    return torch.randn((T, D), generator=g, device=dev) * feature * row


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dev = case["op"], "cuda"
    s = dict(case)
    if op == "norm":
        T, D = case["T"], case["D"]
        s["x"] = _normal(g, T, D).to(TYPES[case["x"]])
        s["r"] = _stream(g, T, D).to(TYPES[case["r"]])
        s["w"] = (1 + 0.1 * _normal(g, D)).to(TYPES[case["w"]])
        s["y"] = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
        s["total"] = torch.empty_like(s["r"])
        s["rstd"] = torch.empty(T, device=dev) if case["rstd"] else None
        s["q"] = s["scale"] = None
        if case["fp8"]:
            s["q"] = torch.empty((T, -(-D // 16) * 16), dtype=torch.float8_e4m3fn,
                                 device=dev)[:, :D]
            s["scale"] = torch.empty((T, -(-D // BLOCK)), device=dev)
    elif op == "norm_bwd":
        T, D = case["T"], case["D"]
        s["x"] = _stream(g, T, D).to(TYPES[case["x"]])
        s["w"] = (1 + 0.1 * _normal(g, D)).to(TYPES[case["w"]])
        s["rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt()
        s["dy"] = (0.01 * _normal(g, T, D)).to(TYPES[case["dy"]])
        s["dtotal"] = (0.01 * _normal(g, T, D)).to(s["x"].dtype)
    elif op == "quant":
        s["x"] = _stream(g, case["R"], case["C"]).to(TYPES[case["x"]])
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["a_scale"] = _quantised(_stream(g, M, K), 1)
        s["b"], s["b_scale"] = _quantised(_normal(g, N, K) / math.sqrt(K), case["b_block"])
    else:
        T, D, F, p = case["T"], case["D"], case["F"], case["density"]
        x = _normal(g, T, D)
        x[:, -1] = 1.0
        wg = _normal(g, F, D) / math.sqrt(D)
        # the threshold that leaves a share p of the gates positive
        wg[:, -1] = -math.sqrt(2.0) * float(torch.erfinv(torch.tensor(1.0 - 2.0 * p)))
        s["x"] = x.to(torch.bfloat16)
        s["xq"], s["x_scale"] = _quantised(s["x"].float(), 1)
        s["wq"], s["w_scale"] = _quantised(wg, BLOCK)
        s["wu"] = (_normal(g, F, D) / math.sqrt(D)).to(torch.bfloat16)
        s["wd"] = (_normal(g, F, D) / math.sqrt(F)).to(torch.bfloat16)
        s["y"] = torch.empty((T, D), device=dev)
    return s


# ------------------------------------------------------------------------- run


def _blocks(x, block):
    """|x|'s maximum over each block of `block` rows by 128 columns, and 448 over it
    spread back over x."""
    R, C = x.shape
    nr, nc = -(-R // block), -(-C // BLOCK)
    p = torch.nn.functional.pad(x, (0, nc * BLOCK - C, 0, nr * block - R))
    amax = p.view(nr, block, nc, BLOCK).abs().amax(dim=(1, 3)).clamp_min(AMAX_MIN)
    return amax, _spread(E4M3_MAX / amax, block, R, C)


def _spread(s, block, R, C):
    if block > 1:
        s = s.repeat_interleave(block, 0)[:R]
    return s.repeat_interleave(BLOCK, 1)[:, :C]


def _e4m3(x, block):
    amax, inv = _blocks(x, block)
    q = (x * inv).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, amax * (1.0 / E4M3_MAX)


def _plain(s):
    op = s["op"]
    if op == "norm":
        total = s["x"].float() + s["r"].float()
        rstd = (total.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = total * rstd * s["w"].float()
        out = {"total": total.to(s["r"].dtype), "y": y.to(torch.bfloat16)}
        if s["fp8"]:
            out["q"], out["scale"] = _e4m3(y, 1)
        if s["rstd"] is not None:
            out["rstd"] = rstd[:, 0]
        return out
    if op == "norm_bwd":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        n = x * rstd
        dn = dy * s["w"].float()
        dx = (dn - n * (dn * n).mean(1, keepdim=True)) * rstd + s["dtotal"].float()
        return {"dx": dx.to(s["x"].dtype), "dw": (dy * n).sum(0)}
    if op == "quant":
        x, block = s["x"].float(), s["block"]
        out = {}
        out["q"], out["scale"] = _e4m3(x, block)
        if s["both"]:
            out["qt"], out["scale_t"] = _e4m3(x.t().contiguous(), block)
        return out
    if op == "gemm":
        M, N, K = s["M"], s["N"], s["K"]
        a = s["a"].float() * _spread(s["a_scale"], 1, M, K)
        b = s["b"].float() * _spread(s["b_scale"], s["b_block"], N, K)
        return (a @ b.t()).to(TYPES[s["out"]])
    T, D, F = s["T"], s["D"], s["F"]
    x = s["xq"].float() * _spread(s["x_scale"], 1, T, D)
    wg = s["wq"].float() * _spread(s["w_scale"], BLOCK, F, D)
    h = (x @ wg.t()).clamp_min(0)
    return (h * (s["x"].float() @ s["wu"].float().t())) @ s["wd"].float()


def run(state):
    if not own:
        return _plain(state)
    import activation_sparse_gated_gate_gb300 as tw

    s, op = state, state["op"]
    if op == "norm":
        o = tw.twell_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, y=s["y"],
                              total=s["total"], rstd=s["rstd"], q=s["q"], scale=s["scale"])
        out = {"total": o.total, "y": o.y}
        if s["fp8"]:
            out["q"], out["scale"] = o.q, o.scale
        if s["rstd"] is not None:
            out["rstd"] = o.rstd
        return out
    if op == "norm_bwd":
        dx, dw = tw.twell_rms_norm_bwd(s["x"], s["w"], s["rstd"], s["dy"], dtotal=s["dtotal"])
        return {"dx": dx, "dw": dw}
    if op == "quant":
        o = tw.twell_quant_fp8(s["x"], block_rows=s["block"], transposed=s["both"])
        out = {"q": o.q, "scale": o.scale}
        if s["both"]:
            out["qt"], out["scale_t"] = o.qt, o.scale_t
        return out
    if op == "gemm":
        return tw.twell_gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"],
                                 dtype=TYPES[s["out"]])
    if "h" not in s:  # the gate's buffers, which a program keeps from step to step
        s["h"] = tw.TwELL(s["T"], s["F"], 8)
    tw.twell_gate_pack_fp8(s["xq"], s["x_scale"], s["wq"], s["w_scale"], s["h"])
    return tw.twell_ffn_fwd(s["x"], s["h"], s["wu"], s["wd"], y=s["y"])


# ------------------------------------------------------------------ work, exact


def work(case):
    op = case["op"]
    if op == "norm":
        n, nb = case["T"] * case["D"], case["T"] * -(-case["D"] // BLOCK)
        b = n * (BYTES[case["x"]] + 2 * BYTES[case["r"]] + 2) + case["D"] * BYTES[case["w"]]
        if case["fp8"]:
            b += n + 4 * nb
        if case["rstd"]:
            b += 4 * case["T"]
        return {"bytes": b, "flops": 5 * n}
    if op == "norm_bwd":
        n = case["T"] * case["D"]
        b = n * (3 * BYTES[case["x"]] + BYTES[case["dy"]]) + 4 * case["T"]
        return {"bytes": b + case["D"] * (BYTES[case["w"]] + 4), "flops": 10 * n}
    if op == "quant":
        R, C, block = case["R"], case["C"], case["block"]
        b = R * C * (BYTES[case["x"]] + 1) + 4 * -(-R // block) * -(-C // BLOCK)
        if case["both"]:
            b += R * C + 4 * -(-C // block) * -(-R // BLOCK)
        return {"bytes": b, "flops": (4 if case["both"] else 2) * R * C}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        nk = -(-K // BLOCK)
        b = (M + N) * K + 4 * nk * (M + -(-N // case["b_block"])) + M * N * BYTES[case["out"]]
        return {"bytes": b, "flops": 2 * M * N * K}
    T, D, F, p = case["T"], case["D"], case["F"], case["density"]
    active = F * (1.0 - (1.0 - p) ** T)   # neurons with some active token
    b = (T + F) * D + 4 * -(-D // BLOCK) * (T + F // BLOCK) + 6 * T * D + 4 * active * D
    return {"bytes": b, "flops": 2 * T * D * F + 4 * p * T * F * D}


def _wide(q, scale, block, like):
    """The values that e4m3 codes and their scales stand for, in 64 bits."""
    R, C = like
    rows = torch.arange(R, device=q.device) // block
    cols = torch.arange(C, device=q.device) // BLOCK
    return q.to(torch.float32).to(torch.float64) * scale.to(torch.float64)[rows][:, cols]


def _exact_scaled(v, block):
    """v over its block's scale (before the rounding to e4m3), and the scales."""
    R, C = v.shape
    rows = torch.arange(R, device=v.device) // block
    cols = torch.arange(C, device=v.device) // BLOCK
    key = (rows[:, None] * (-(-C // BLOCK)) + cols[None, :]).reshape(-1)
    n = -(-R // block) * -(-C // BLOCK)
    top = torch.full((n,), AMAX_MIN, dtype=torch.float64, device=v.device)
    top.scatter_reduce_(0, key, v.abs().reshape(-1), "amax")
    scale = (top / 448).view(-(-R // block), -(-C // BLOCK))
    return v / scale[rows][:, cols], scale


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "norm":
        t = s["x"].to(f64) + s["r"].to(f64)
        inv = 1 / torch.sqrt((t ** 2).sum(1) / case["D"] + EPS)
        y = torch.einsum("td,t,d->td", t, inv, s["w"].to(f64))
        out = {"total": t, "y": y}
        if case["fp8"]:
            out["q"], out["scale"] = _exact_scaled(y, 1)
        if case["rstd"]:
            out["rstd"] = inv
        return out
    if op == "norm_bwd":
        x, w, inv, dy = (s[k].to(f64) for k in ("x", "w", "rstd", "dy"))
        g = dy * w
        c = (g * x).sum(1) * inv ** 3 / case["D"]
        dx = g * inv[:, None] - x * c[:, None] + s["dtotal"].to(f64)
        return {"dx": dx, "dw": torch.einsum("td,td,t->d", dy, x, inv)}
    if op == "quant":
        v, out = s["x"].to(f64), {}
        out["q"], out["scale"] = _exact_scaled(v, case["block"])
        if case["both"]:
            out["qt"], out["scale_t"] = _exact_scaled(v.t(), case["block"])
        return out
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a = _wide(s["a"], s["a_scale"], 1, (M, K))
        return torch.einsum("mk,nk->mn", a, _wide(s["b"], s["b_scale"], case["b_block"], (N, K)))
    T, D, F = case["T"], case["D"], case["F"]
    z = torch.einsum("td,fd->tf", _wide(s["xq"], s["x_scale"], 1, (T, D)),
                     _wide(s["wq"], s["w_scale"], BLOCK, (F, D)))
    u = torch.einsum("td,fd->tf", s["x"].to(f64), s["wu"].to(f64))
    return torch.einsum("tf,fd->td", torch.where(z > 0, z * u, torch.zeros_like(z)),
                        s["wd"].to(f64))
