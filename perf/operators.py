"""Cases and plain forms of the operators around a decode or verify step's routed experts:

  norm   the norms after one block and before the next, with the block's gate and residual scale
  route  the router: which experts a token goes to, and with what weights
  moe    a whole mixture-of-experts layer over FP4 experts for a few tokens
  int4   matrix-vector products with 4-bit weights and a scale (and zero point) per group of columns

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, calls the library; ``exact`` gives the definition's values in 64 bits.
"""
import math

import torch

own = False

MXFP4, NVFP4 = 0, 1
SOFTMAX, SIGMOID, SQRT_SOFTPLUS = 0, 1, 2
EPS = 1e-6


def listed():
    return [
        # One token between two blocks of a decode step, and a 16-row verify panel at a larger width, rows gated one by one.
        {"name": "norm_1x4096", "op": "norm", "N": 1, "cols": 4096, "resid": "bf16", "gate": "cols", "post": True, "scale": 0.5},
        {"name": "norm_16x7168_rowgate", "op": "norm", "N": 16, "cols": 7168, "resid": "f32", "gate": "rows", "post": True, "scale": 1.0},
        # The same step over a prefill panel of 8192 tokens.
        {"name": "norm_8192x4096", "op": "norm", "N": 8192, "cols": 4096, "resid": "bf16", "gate": "cols", "post": True, "scale": 1.0},
        # Decode, verify panel, and the router of a 2048-token prefill panel.
        {"name": "route_1_256x4096", "op": "route", "M": 1, "E": 256, "cols": 4096, "K": 8, "score": SQRT_SOFTPLUS, "bias": True, "norm": True},
        {"name": "route_13_160x2064", "op": "route", "M": 13, "E": 160, "cols": 2064, "K": 6, "score": SIGMOID, "bias": True, "norm": True},
        {"name": "route_2048_256x4096", "op": "route", "M": 2048, "E": 256, "cols": 4096, "K": 8, "score": SOFTMAX, "bias": False, "norm": False},
        # One decode token over 8 of 64 NVFP4 experts of 4096 x 2048; a small odd layer; a 16-row verify panel.
        {"name": "moe_nv_1_8of64", "op": "moe", "fmt": NVFP4, "M": 1, "E": 64, "K": 8, "H": 4096, "I": 2048, "limit": 0.0, "base": True},
        {"name": "moe_mx_3_4of32_odd", "op": "moe", "fmt": MXFP4, "M": 3, "E": 32, "K": 4, "H": 1440, "I": 736, "limit": 7.0, "base": False},
        {"name": "moe_mx_16_8of128", "op": "moe", "fmt": MXFP4, "M": 16, "E": 128, "K": 8, "H": 4096, "I": 2048, "limit": 10.0, "base": False},
        # A decode projection, an odd small panel with fine groups, and an output head read by a verify panel.
        {"name": "int4_1_4096x4096_g128", "op": "int4", "M": 1, "rows": 4096, "cols": 4096, "group": 128, "zeros": True},
        {"name": "int4_5_2001x2080_g32", "op": "int4", "M": 5, "rows": 2001, "cols": 2080, "group": 32, "zeros": False},
        {"name": "int4_16_129280x4096_g64", "op": "int4", "M": 16, "rows": 129280, "cols": 4096, "group": 64, "zeros": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "route", "moe", "int4"))
    if op == "norm":
        cols = _log(rng, 256, 8192, 16)
        return {"op": op, "N": _log(rng, 1, 8192 * 4096 // cols), "cols": cols, "resid": rng.choice(("f32", "bf16")),
                "gate": rng.choice(("none", "cols", "rows")), "post": rng.random() < 0.7, "scale": rng.choice((0.25, 0.5, 1.0))}
    if op == "route":
        E, cols = _log(rng, 8, 256), _log(rng, 256, 4096, 16)
        return {"op": op, "M": _log(rng, 1, 2048), "E": E, "cols": cols, "K": rng.randint(1, min(16, E)),
                "score": rng.choice((SOFTMAX, SIGMOID, SQRT_SOFTPLUS)), "bias": rng.random() < 0.5, "norm": rng.random() < 0.5}
    if op == "moe":
        E = _log(rng, 4, 128)
        return {"op": op, "fmt": rng.choice((MXFP4, NVFP4)), "M": rng.randint(1, 16), "E": E, "K": rng.randint(1, min(8, E)),
                "H": _log(rng, 256, 4096, 32), "I": _log(rng, 256, 2048, 32), "limit": rng.choice((0.0, 7.0)), "base": rng.random() < 0.5}
    group = rng.choice((32, 64, 128))
    cols = _log(rng, 256, 8192, group)
    return {"op": op, "M": rng.randint(1, 16), "rows": _log(rng, 64, min(129280, 129280 * 4096 // cols)), "cols": cols, "group": group,
            "zeros": rng.random() < 0.5}


def work(c):
    if c["op"] == "norm":
        r = 4 if c["resid"] == "f32" else 2
        gate = {"none": 0, "cols": c["cols"], "rows": c["N"] * c["cols"]}[c["gate"]]
        n = c["N"] * c["cols"]
        return {"bytes": n * (4 + r + r + 2) + 2 * gate + 2 * c["cols"] * (1 + c["post"]), "flops": 9 * n}
    if c["op"] == "route":
        return {"bytes": 2 * (c["M"] + c["E"]) * c["cols"] + 8 * c["M"] * c["K"] + 4 * c["E"] * c["bias"],
                "flops": 2 * c["M"] * c["E"] * c["cols"]}
    if c["op"] == "moe":
        block = 32 if c["fmt"] == MXFP4 else 16
        experts = c["E"] * (1 - (1 - c["K"] / c["E"]) ** c["M"])  # distinct ones that M tokens choose, on average
        n = c["H"] * c["I"]
        return {"bytes": experts * 3 * n * (0.5 + 1 / block) + c["M"] * (c["H"] * (2 + 4 + 4 * c["base"]) + 8 * c["K"]),
                "flops": 6 * c["M"] * c["K"] * n}
    groups = c["rows"] * (c["cols"] // c["group"])
    return {"bytes": c["rows"] * c["cols"] // 2 + groups * (2 + c["zeros"]) + c["M"] * (2 * c["cols"] + 4 * c["rows"]),
            "flops": 2 * c["M"] * c["rows"] * c["cols"]}


# --- inputs --------------------------------------------------------------------

def _fp4_slab(g, fmt, E, rows, cols, dev):
    """Stacked codes and block scales whose products with N(0, 1) inputs are of order 1."""
    codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=dev, dtype=torch.uint8)
    if fmt == MXFP4:
        top = 127 - round(math.log2(3 * math.sqrt(cols)))
        return codes, torch.randint(top - 2, top + 1, (E, rows, cols // 32), generator=g, device=dev, dtype=torch.uint8), None
    scales = torch.randint(0x28, 0x58, (E, rows, cols // 16), generator=g, device=dev, dtype=torch.uint8)
    return codes, scales, (0.5 + torch.rand(E, generator=g, device=dev)) / (15 * math.sqrt(cols))


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(c)
    if c["op"] == "norm":
        N, cols = c["N"], c["cols"]
        s["resid"] = (4 * normal(N, cols)).to(torch.float32 if c["resid"] == "f32" else torch.bfloat16)
        s["y"] = 2 * normal(N, cols)
        s["post_w"] = (1 + 0.1 * normal(cols)).bfloat16() if c["post"] else None
        s["pre_w"] = (1 + 0.1 * normal(cols)).bfloat16()
        s["gate"] = None if c["gate"] == "none" else torch.sigmoid(normal(N if c["gate"] == "rows" else 1, cols)).bfloat16()
        s["resid_out"] = torch.empty_like(s["resid"])
        s["x_next"] = torch.empty(N, cols, dtype=torch.bfloat16, device=dev)
    elif c["op"] == "route":
        M, E, cols, K = c["M"], c["E"], c["cols"], c["K"]
        s["x"] = normal(M, cols).bfloat16()
        s["w"] = (normal(E, cols) * (1.5 / math.sqrt(cols))).bfloat16()
        s["bias"] = 0.1 * normal(E) if c["bias"] else None
        s["ids"] = torch.empty(M, K, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(M, K, device=dev)
        if own:
            import block_scaled_fp8_fp8blk_amd as fb
            s["ws"] = torch.empty(fb.fp8blk_workspace_bytes(fb.OP_MOE_ROUTE, E, cols, M), dtype=torch.uint8, device=dev)
    elif c["op"] == "moe":
        M, E, K, H, I = c["M"], c["E"], c["K"], c["H"], c["I"]
        s["gate"], s["up"], s["down"] = (_fp4_slab(g, c["fmt"], E, r, k, dev) for r, k in ((I, H), (I, H), (H, I)))
        s["x"] = normal(M, H).bfloat16()
        order = torch.rand(M, E, generator=g, device=dev).argsort(dim=1)
        s["ids"] = order[:, :K].to(torch.int32).contiguous()
        s["weights"] = torch.softmax(normal(M, K), dim=1)
        s["base"] = normal(M, H) if c["base"] else None
        s["y"] = torch.empty(M, H, device=dev)
        if own:
            import block_scaled_fp8_fp8blk_amd as fb
            s["layer"] = fb.fp4_moe_weights(c["fmt"], *s["gate"], *s["up"], *s["down"], limit=c["limit"])
            s["ws"] = torch.empty(fb.fp4_moe_bytes(I, M, K), dtype=torch.uint8, device=dev)
    else:
        M, rows, cols, G = c["M"], c["rows"], c["cols"], c["group"]
        s["codes"] = torch.randint(0, 256, (rows, cols // 2), generator=g, device=dev, dtype=torch.uint8)
        s["scales"] = (torch.exp(0.3 * normal(rows, cols // G)) / (4.6 * math.sqrt(cols))).bfloat16()
        s["zeros"] = torch.randint(5, 11, (rows, cols // G), generator=g, device=dev, dtype=torch.uint8) if c["zeros"] else None
        s["x"] = normal(M, cols).bfloat16()
        s["y"] = torch.empty(M, rows, device=dev)
    return s


# --- one pass ------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "route": _route, "moe": _moe, "int4": _int4}[s["op"]](s)


def _own(s):
    import block_scaled_fp8_fp8blk_amd as fb
    if s["op"] == "norm":
        fb.fp8blk_block_norm(s["resid"], s["y"], s["post_w"], s["gate"], s["scale"], s["resid_out"], s["pre_w"], EPS, s["x_next"])
        return s["resid_out"], s["x_next"]
    if s["op"] == "route":
        fb.fp8blk_moe_route(s["w"], s["bias"], s["x"], s["score"], s["norm"], 2.5, s["ids"], s["weights"], s["ws"])
        return s["ids"], s["weights"]
    if s["op"] == "moe":
        fb.fp4_moe(s["layer"], s["x"], s["ids"], s["weights"], s["base"], s["y"], s["ws"])
        return s["y"]
    fb.int4_gemv(s["codes"], s["scales"], s["zeros"], s["group"], s["x"], s["y"])
    return s["y"]


def _norm(s):
    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w.float()

    d = s["y"] if s["post_w"] is None else rms(s["y"], s["post_w"])
    if s["gate"] is not None:
        d = s["gate"].float() * d
    r = s["resid"].float() + s["scale"] * d
    return r.to(s["resid"].dtype), rms(r, s["pre_w"]).bfloat16()


def _route(s):
    logits = s["x"].double() @ s["w"].double().t()
    if s["score"] == SOFTMAX:
        e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
        score = e / e.sum(dim=1, keepdim=True)
    elif s["score"] == SIGMOID:
        score = 1 / (1 + torch.exp(-logits))
    else:
        score = torch.sqrt(torch.log1p(torch.exp(-logits.abs())) + logits.clamp(min=0))
    choice = score if s["bias"] is None else score + s["bias"]
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :s["K"]]
    weights = score.gather(1, ids)
    if s["norm"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (2.5 * weights).float()


def _fp4_rows(slab, fmt, ids):
    """The chosen experts' weights in f32, [len(ids), rows, cols]."""
    codes, scales, top = slab
    dev = codes.device
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=dev)
    c = codes[ids]
    w = torch.stack((values[(c & 15).int()], values[(c >> 4).int()]), dim=-1)
    sc = scales[ids]
    if fmt == MXFP4:
        sc = torch.exp2(sc.float() - 127)
    else:
        sc = sc.view(torch.float8_e4m3fn).float() * top[ids][:, None, None]
    block = 32 if fmt == MXFP4 else 16
    return (w.reshape(*sc.shape, block) * sc[..., None]).reshape(c.shape[0], c.shape[1], -1)


def _moe(s):
    M, K = s["M"], s["K"]
    ids = s["ids"].reshape(-1).long()
    x = s["x"].float().repeat_interleave(K, dim=0)[:, :, None]
    g = torch.bmm(_fp4_rows(s["gate"], s["fmt"], ids), x)
    u = torch.bmm(_fp4_rows(s["up"], s["fmt"], ids), x)
    if s["limit"] > 0:
        g, u = g.clamp(max=s["limit"]), u.clamp(-s["limit"], s["limit"])
    h = g / (1 + torch.exp(-g)) * u
    y = torch.bmm(_fp4_rows(s["down"], s["fmt"], ids), h)[:, :, 0]
    y = (y.view(M, K, -1) * s["weights"][:, :, None]).sum(dim=1)
    return y if s["base"] is None else s["base"] + y


def _int4(s):
    c = s["codes"]
    q = torch.stack((c & 15, c >> 4), dim=-1).float().reshape(*s["scales"].shape, s["group"])
    z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((q - z) * s["scales"].float()[..., None]).reshape(c.shape[0], -1)
    return s["x"].float() @ w.t()


# --- the definitions in 64 bits --------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _norm64, "route": _route64, "moe": _moe64, "int4": _int464}[c["op"]](s)


def _norm64(s):
    def unit(v):
        return v / (v.square().sum(dim=-1, keepdim=True) / v.shape[-1] + EPS).sqrt()

    block = s["y"].double()
    if s["post_w"] is not None:
        block = unit(block).mul_(s["post_w"].double())
    if s["gate"] is not None:
        block = block.mul_(s["gate"].double())
    total = s["resid"].double().add_(block, alpha=s["scale"])
    return total, unit(total).mul_(s["pre_w"].double())


def _route64(s):
    w = s["w"].double()
    ids, weights = [], []
    for row in s["x"].double():
        logit = (w * row).sum(dim=1)
        if s["score"] == SOFTMAX:
            score = torch.softmax(logit, dim=0)
        elif s["score"] == SIGMOID:
            score = torch.sigmoid(logit)
        else:
            score = torch.nn.functional.softplus(logit, threshold=1000.0).sqrt()
        left = score.clone() if s["bias"] is None else score + s["bias"].double()
        chosen = []
        for _ in range(s["K"]):
            best = left.argmax()
            chosen.append(best)
            left[best] = -math.inf
        chosen = torch.stack(chosen)
        p = score[chosen]
        ids.append(chosen)
        weights.append(2.5 * (p / p.sum() if s["norm"] else p))
    return torch.stack(ids).to(torch.int32), torch.stack(weights)


def _fp4_one(slab, fmt, e):
    """Expert e's weights in 64 bits from the codes' bit fields: sign, 2 exponent bits, 1 mantissa bit."""
    codes, scales, top = (None if t is None else t[e] for t in slab)
    nibbles = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int32, device=codes.device)
    nibbles[:, 0::2] = codes.int() % 16
    nibbles[:, 1::2] = codes.int() // 16
    exponent, mantissa = nibbles // 2 % 4, (nibbles % 2).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.pow(2.0, (exponent - 1).double()))
    w = torch.where(nibbles >= 8, -size, size)
    code = scales.int()
    if fmt == MXFP4:
        scale = torch.pow(2.0, (code - 127).double())
    else:
        field, frac = code // 8, (code % 8).double()
        scale = torch.where(field == 0, frac / 8 * 2.0 ** -6, (1 + frac / 8) * torch.pow(2.0, (field - 7).double())) * top.double()
    return w * scale.repeat_interleave(w.shape[1] // scale.shape[1], dim=1)


def _moe64(s):
    y = torch.zeros(s["M"], s["H"], dtype=torch.float64, device=s["x"].device)
    if s["base"] is not None:
        y += s["base"]
    x = s["x"].double()
    for e in s["ids"].unique().tolist():
        token, place = (s["ids"] == e).nonzero(as_tuple=True)
        g = x[token] @ _fp4_one(s["gate"], s["fmt"], e).t()
        u = x[token] @ _fp4_one(s["up"], s["fmt"], e).t()
        if s["limit"] > 0:
            g, u = torch.minimum(g, torch.full_like(g, s["limit"])), u.clamp(min=-s["limit"]).clamp(max=s["limit"])
        h = g * torch.sigmoid(g) * u
        y.index_add_(0, token, s["weights"][token, place].double()[:, None] * (h @ _fp4_one(s["down"], s["fmt"], e).t()))
    return y


def _int464(s):
    rows, half = s["codes"].shape
    w = torch.empty(rows, 2 * half, dtype=torch.float64, device=s["codes"].device)
    w[:, 0::2] = s["codes"] % 16
    w[:, 1::2] = s["codes"] // 16
    w -= 8 if s["zeros"] is None else s["zeros"].double().repeat_interleave(s["group"], dim=1)
    w *= s["scales"].double().repeat_interleave(s["group"], dim=1)
    return s["x"].double() @ w.t()
