"""Cases and plain forms of the operators between a layer's q and kv linears and its o linear:

  append  rotary positions on q and k, and the new keys and values written into a paged cache
  attn    attention of new tokens (one, a verify panel, a prompt's chunk) over a paged cache
  latent  the same over a cache of one shared latent row a token, whose first columns are the values

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, calls the library; ``exact`` gives the definition's values in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
LATENT = 512
E4M3_MAX = 448.0
K_SCALE, V_SCALE = 0.021, 0.017  # of 8-bit caches: values of a few units reach a third of e4m3's range


def listed():
    return [
        # One decode token between the 4096 x 4096 q and the 1024 x 4096 kv linear: 32 and 4 heads of 128, all of them rotated.
        {"name": "append_1", "op": "append", "N": 1, "heads": 32, "kv": 4, "pass": 0, "rot": 128, "v": 128, "type": "f32", "cache": "bf16",
         "page": 64, "interleaved": False, "rot_first": True, "norm": "none", "far": 4000, "factor": 1.0, "pad": 0},
        # Tokens of 13 sequences into a latent cache, far into a long context, 3 of 16 rows only there to fill the panel.
        {"name": "append_latent_16", "op": "append", "N": 16, "heads": 16, "kv": 1, "pass": 512, "rot": 64, "v": 0, "type": "f32", "cache": "bf16",
         "page": 64, "interleaved": True, "rot_first": False, "norm": "pass", "far": 900000, "factor": 32.0, "pad": 3},
        # A prompt of 8191 tokens with normalised heads, half of each rotated, into an 8-bit cache.
        {"name": "append_8191_e4m3", "op": "append", "N": 8191, "heads": 32, "kv": 4, "pass": 64, "rot": 64, "v": 128, "type": "f32", "cache": "e4m3",
         "page": 16, "interleaved": False, "rot_first": True, "norm": "whole", "far": 0, "factor": 4.0, "pad": 0},
        # One sequence decoding: 32 heads that share 4.
        {"name": "attn_1x4096", "op": "attn", "S": 1, "T": 1, "L": 4096, "heads": 32, "kv": 4, "k": 128, "v": 128, "cache": "bf16", "page": 64,
         "causal": True, "window": 0, "sinks": False, "ragged": False, "pad": 0},
        # 32 sequences decoding at their own lengths up to 16384, and as many of an 8-bit cache with small pages.
        {"name": "attn_32x16384", "op": "attn", "S": 32, "T": 1, "L": 16384, "heads": 32, "kv": 4, "k": 128, "v": 128, "cache": "bf16", "page": 64,
         "causal": True, "window": 0, "sinks": False, "ragged": True, "pad": 0},
        {"name": "attn_32x16384_e4m3", "op": "attn", "S": 32, "T": 1, "L": 16384, "heads": 32, "kv": 4, "k": 128, "v": 128, "cache": "e4m3", "page": 16,
         "causal": True, "window": 0, "sinks": False, "ragged": True, "pad": 0},
        # A verify panel: up to 6 drafted tokens of 5 sequences through a layer with a sliding window and sinks, rows behind them unused.
        {"name": "attn_verify_5x6_window", "op": "attn", "S": 5, "T": 6, "L": 5000, "heads": 64, "kv": 8, "k": 64, "v": 64, "cache": "bf16", "page": 16,
         "causal": True, "window": 128, "sinks": True, "ragged": True, "pad": 3},
        # The last chunk of a prompt of 8192 tokens, and chunks of three prompts at once, heads of 256.
        {"name": "attn_2048_of_8192", "op": "attn", "S": 1, "T": 2048, "L": 8192, "heads": 32, "kv": 4, "k": 128, "v": 128, "cache": "bf16", "page": 64,
         "causal": True, "window": 0, "sinks": False, "ragged": False, "pad": 0},
        {"name": "attn_3x777_of_2999_k256", "op": "attn", "S": 3, "T": 777, "L": 2999, "heads": 16, "kv": 2, "k": 256, "v": 256, "cache": "bf16", "page": 32,
         "causal": True, "window": 0, "sinks": True, "ragged": True, "pad": 0},
        # Latent attention: a prompt in its expanded form (keys of 128 + 64 columns, values of 128, every head its own), one sequence decoding with all
        # 128 heads, and a verify panel of 16 sequences with the 16 heads that one of eight ranks holds.
        {"name": "attn_2000_expanded", "op": "attn", "S": 1, "T": 2000, "L": 2000, "heads": 16, "kv": 16, "k": 192, "v": 128, "cache": "bf16", "page": 64,
         "causal": True, "window": 0, "sinks": False, "ragged": False, "pad": 0},
        {"name": "latent_1x8192_128", "op": "latent", "S": 1, "T": 1, "L": 8192, "heads": 128, "rot": 64, "page": 64, "causal": True, "window": 0,
         "sinks": False, "ragged": False, "pad": 0},
        {"name": "latent_16x2_16", "op": "latent", "S": 16, "T": 2, "L": 16384, "heads": 16, "rot": 64, "page": 64, "causal": True, "window": 0,
         "sinks": False, "ragged": True, "pad": 1},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        scores = 0 if c["op"] == "append" else c["S"] * c["T"] * c["L"] * c["heads"]
        if max(w["bytes"], w["flops"] / 50) < 4e9 and scores < 5e8:
            return c


def _draw(rng):
    op = rng.choice(("append", "attn", "attn", "latent"))
    if op == "append":
        c = {"op": op, "N": _log(rng, 1, 8192), "heads": rng.choice((1, 5, 8, 12, 16, 32)), "kv": rng.choice((1, 2, 3, 4)), "type": rng.choice(("f32", "bf16")),
             "page": rng.choice((1, 8, 16, 64, 256)), "interleaved": rng.random() < 0.5, "rot_first": rng.random() < 0.5,
             "far": rng.choice((0, 1000, 100000)), "factor": rng.choice((1.0, 8.0)), "pad": 0}
        c["pad"] = rng.randint(0, c["N"] // 4)
        if rng.random() < 0.3:
            return {**c, "kv": 1, "pass": LATENT, "rot": rng.choice((32, 64)), "v": 0, "cache": "bf16", "norm": rng.choice(("none", "pass"))}
        cols = rng.choice((64, 128, 256))
        rot = rng.choice((cols, cols // 2, 24))
        return {**c, "pass": cols - rot, "rot": rot, "v": cols, "cache": rng.choice(("bf16", "e4m3")), "norm": rng.choice(("none", "whole"))}
    T = rng.choice((1, 1, rng.randint(2, 16), _log(rng, 17, 2048)))
    c = {"op": op, "S": _log(rng, 1, 32), "T": T, "L": _log(rng, max(T, 16), 16384), "page": rng.choice((1, 8, 16, 64, 256)), "causal": rng.random() < 0.85,
         "window": rng.choice((0, 0, _log(rng, 16, 4096))), "sinks": rng.random() < 0.4, "ragged": rng.random() < 0.7, "pad": rng.randint(0, 2)}
    if op == "latent":
        return {**c, "heads": rng.choice((1, 8, 12, 16, 32, 64, 128)), "rot": rng.choice((0, 64))}
    kv = rng.choice((1, 2, 4, 8))
    k, v = rng.choice(((64, 64), (128, 128), (256, 256), (192, 128)))
    return {**c, "heads": kv * rng.choice((1, 3, 4, 5, 8, 16)), "kv": kv, "k": k, "v": v, "cache": rng.choice(("bf16", "e4m3"))}


def _batch(c):
    """Tokens in the cache (the new ones among them) and new tokens of every sequence."""
    S = c["S"]
    if not c["ragged"]:
        return [c["L"]] * S, [c["T"]] * S
    new = [max(1, c["T"] * (5 * i % S + 1) // S) for i in range(S)]
    return [max(n, c["L"] * ((7 * i + 3) % S + 1) // S) for i, n in enumerate(new)], new


def _widths(c):
    """Key and value columns, key heads, bytes of a cached value and of a token's cached rows."""
    if c["op"] == "latent":
        return LATENT + c["rot"], LATENT, 1, 2, 2 * (LATENT + c["rot"])
    b = 1 if c["cache"] == "e4m3" else 2
    return c["k"], c["v"], c["kv"], b, b * c["kv"] * (c["k"] + c["v"])


def work(c):
    if c["op"] == "append":
        cols, live, size = c["pass"] + c["rot"], c["N"] - c["pad"], 4 if c["type"] == "f32" else 2
        stored = 1 if c["cache"] == "e4m3" else 2
        q, kv = c["N"] * c["heads"] * cols, live * c["kv"] * (cols + c["v"])
        return {"bytes": (size + 2) * q + (size + stored) * kv + 8 * c["N"], "flops": 6 * (q + kv)}
    k, v, _, _, row = _widths(c)
    seen, pairs = 0, 0
    for length, new in zip(*_batch(c)):
        first = length - new  # the first new token's position
        lo = max(0, first - c["window"] + 1) if c["window"] else 0
        seen += length - lo
        for at in range(first, length):
            pairs += (at + 1 if c["causal"] else length) - (max(0, at - c["window"] + 1) if c["window"] else 0)
    n = sum(_batch(c)[1])
    return {"bytes": seen * row + 2 * n * c["heads"] * (k + v), "flops": 2 * pairs * c["heads"] * (k + v)}


# --- inputs --------------------------------------------------------------------

def _freqs(rot, factor, dev):
    """Radians a position of each pair: turns that fit an original context of 4096 more than 32 times stay, those that fit less than once are
    divided by factor, those between in between."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    keep = ((f * 4096 / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f * (keep + (1 - keep) / factor)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def order(n):
        return torch.rand(n, generator=g, device=dev).argsort()

    return (_prepare_append if c["op"] == "append" else _prepare_attn)(c, dict(c), dev, g, normal, order)


def _prepare_append(c, s, dev, g, normal, order):
    N, H, h, P, R, V = c["N"], c["heads"], c["kv"], c["pass"], c["rot"], c["v"]
    cols, kind = P + R, torch.float32 if c["type"] == "f32" else torch.bfloat16
    if V:  # q and kv as two linears write them
        q, kv = (2 * normal(N, H, cols)).to(kind), (2 * normal(N, h * (cols + V))).to(kind)
        k, s["v_new"] = kv[:, :h * cols].view(N, h, cols), kv[:, h * cols:].view(N, h, V)
        at = (slice(R, cols), slice(0, R)) if c["rot_first"] else (slice(0, P), slice(P, cols))
        s["q"], s["k_new"] = tuple(tuple(t[..., a] if a.stop > a.start else None for a in at) for t in (q, k))
    else:  # the latent row from one linear; q's first part head by head out of the products with the keys' weights, its second part beside others
        q_all, kv = (2 * normal(N, H, 128 + R)).to(kind), (2 * normal(N, 1, cols)).to(kind)
        s["q"] = normal(H, N, P).to(kind).transpose(0, 1), q_all[..., 128:]
        s["k_new"], s["v_new"] = (kv[..., :P], kv[..., P:]), None
    normed = {"none": 0, "pass": P, "whole": cols}[c["norm"]]
    s["k_norm"] = (1 + 0.1 * normal(normed)).bfloat16() if normed else None
    s["q_norm"] = (1 + 0.1 * normal(cols)).bfloat16() if c["norm"] == "whole" else None
    s["freqs"], s["mscale"] = _freqs(R, c["factor"], dev), 1 + 0.1 * math.log(c["factor"])
    page, t = c["page"], torch.arange(N, device=dev)
    if N <= 16:  # each token belongs to a sequence of its own
        pages = 64
        slots = order(pages)[:N] * page + torch.randint(0, page, (N,), generator=g, device=dev)
        positions = c["far"] + torch.randint(0, 1000, (N,), generator=g, device=dev)
    else:
        pages = N // page + 3
        slots = order(pages)[(t + page // 2) // page] * page + (t + page // 2) % page
        positions = c["far"] + t
    if c["pad"]:
        slots[N - c["pad"]:] = -1
    s["slots"], s["positions"] = slots.int(), positions.int()
    stored = torch.float8_e4m3fn if c["cache"] == "e4m3" else torch.bfloat16
    s["cache_k"] = torch.zeros(pages, page, h, cols, device=dev).to(stored)
    s["cache_v"] = torch.zeros(pages, page, h, V, device=dev).to(stored) if V else None
    s["scales"] = (K_SCALE, V_SCALE) if c["cache"] == "e4m3" else (1.0, 1.0)
    s["q_out"] = torch.zeros(N, H, cols, dtype=torch.bfloat16, device=dev)
    if own:
        import block_scaled_fp8_fp8blk_amd as fb
        s["rope"] = fb.fp8blk_rope(s["freqs"], interleaved=c["interleaved"], rot_first=c["rot_first"], mscale=s["mscale"])
        s["cache"] = fb.fp8blk_cache(s["cache_k"], s["cache_v"], k_scale=s["scales"][0], v_scale=s["scales"][1])
    return s


def _prepare_attn(c, s, dev, g, normal, order):
    k, v, h, _, _ = _widths(c)
    lens, new = _batch(c)
    S, page = c["S"], c["page"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    ids, at = order(pages).int(), 0
    table = torch.full((S, max(need) + 1), -1, dtype=torch.int32, device=dev)
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["starts"] = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32, device=dev)
    s["most"], s["scale"] = max(lens), 1 / math.sqrt(k)
    eight = c["op"] == "attn" and c["cache"] == "e4m3"
    stored, s["scales"] = (torch.float8_e4m3fn, (K_SCALE, V_SCALE)) if eight else (torch.bfloat16, (1.0, 1.0))
    s["cache_k"] = (normal(pages, page, h, k) / s["scales"][0]).to(stored)
    s["cache_v"] = (normal(pages, page, h, v) / s["scales"][1]).to(stored) if c["op"] == "attn" else None
    N = sum(new) + c["pad"]
    s["q"] = (1.5 * normal(N, c["heads"], k)).bfloat16()
    s["sink"] = normal(c["heads"]) if c["sinks"] else None
    s["out"] = torch.zeros(N, c["heads"], v, dtype=torch.bfloat16, device=dev)
    if own:
        import block_scaled_fp8_fp8blk_amd as fb
        s["cache"] = fb.fp8blk_cache(s["cache_k"], s["cache_v"], k_scale=s["scales"][0], v_scale=s["scales"][1], **({} if c["op"] == "attn" else {"v_cols": v}))
        s["ws"] = torch.empty(fb.fp8blk_attn_bytes(s["cache"], c["heads"], S, c["T"], s["most"], c["window"]), dtype=torch.uint8, device=dev)
    return s


# --- one pass ------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return _append(s) if s["op"] == "append" else _attn(s)


def _own(s):
    import block_scaled_fp8_fp8blk_amd as fb
    if s["op"] == "append":
        fb.fp8blk_rope_append(s["rope"], s["positions"], s["q"], s["q_out"], s["k_new"], s["v_new"], s["cache"], s["slots"],
                              q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return s["q_out"], s["cache_k"], s["cache_v"]
    attend = fb.fp8blk_paged_attn if s["op"] == "attn" else fb.fp8blk_latent_attn
    attend(s["cache"], s["q"], s["table"], s["lens"], s["starts"], s["T"], s["most"], s["scale"], s["out"], s["ws"],
           causal=s["causal"], window=s["window"], sinks=s["sink"])
    return s["out"]


def _rotated(s, parts, norm):
    """[N, heads, cols] in f32: normalised, rotated, the parts in their order."""
    first, rot = (None if t is None else t.float() for t in parts)
    if norm is not None and first is not None and norm.numel() == first.shape[-1]:
        first = first * torch.rsqrt(first.square().mean(-1, keepdim=True) + EPS) * norm.float()
    elif norm is not None:
        total = rot.square().sum(-1, keepdim=True) + (0 if first is None else first.square().sum(-1, keepdim=True))
        unit = torch.rsqrt(total / norm.numel() + EPS)
        R = rot.shape[-1]
        w_rot, w_first = (norm[:R], norm[R:]) if s["rot_first"] else (norm[-R:], norm[:-R])
        rot = rot * unit * w_rot.float()
        first = None if first is None else first * unit * w_first.float()
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((s["mscale"] * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    a, b = (rot[..., 0::2], rot[..., 1::2]) if s["interleaved"] else rot.chunk(2, dim=-1)
    x, y = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack((x, y), dim=-1).flatten(-2) if s["interleaved"] else torch.cat((x, y), dim=-1)
    if first is None:
        return rot
    return torch.cat((rot, first) if s["rot_first"] else (first, rot), dim=-1)


def _append(s):
    s["q_out"].copy_(_rotated(s, s["q"], s["q_norm"]).bfloat16())
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    for cache, rows, scale in ((s["cache_k"], _rotated(s, s["k_new"], s["k_norm"]), s["scales"][0]), (s["cache_v"], s["v_new"], s["scales"][1])):
        if cache is not None:
            rows = rows[live].float()
            if cache.dtype == torch.float8_e4m3fn:
                rows = (rows / scale).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype).view(torch.uint8)
                cache.view(torch.uint8).view(-1, *cache.shape[2:])[slots] = rows
            else:
                cache.view(-1, *cache.shape[2:])[slots] = rows.bfloat16()
    return s["q_out"], s["cache_k"], s["cache_v"]


def _attn(s):
    S, T, L, H, dev = s["S"], s["T"], s["most"], s["heads"], s["q"].device
    starts, lens, N = s["starts"].long(), s["lens"].long(), s["q"].shape[0]
    new, t = starts[1:] - starts[:-1], torch.arange(T, device=dev)
    q = s["q"][(starts[:-1, None] + t).clamp(max=N - 1)].float()
    pages = s["table"][:, :-(-L // s["page"])].clamp(min=0).long()

    def rows(cache, scale):
        return cache.view(torch.uint8 if cache.dtype.itemsize == 1 else cache.dtype)[pages].view(cache.dtype).flatten(1, 2)[:, :L].float() * scale

    k = rows(s["cache_k"], s["scales"][0])
    v = k[..., :LATENT] if s["op"] == "latent" else rows(s["cache_v"], s["scales"][1])
    h = k.shape[2]
    G = H // h
    q = q.view(S, T, h, G, -1).permute(0, 2, 1, 3, 4).reshape(S, h, T * G, -1)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(S, h, T, G, L)
    at, j = (lens - new)[:, None, None] + t[:, None], torch.arange(L, device=dev)
    hidden = j >= lens[:, None, None]
    if s["causal"]:
        hidden = hidden | (j > at)
    if s["window"]:
        hidden = hidden | (j <= at - s["window"])
    score = score.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, h, 1, G, 1)
        top = torch.maximum(top, sink)
    top = top.masked_fill(top == -math.inf, 0)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - top)
    out = torch.matmul(e.view(S, h, T * G, L), v.transpose(1, 2)).view(S, h, T, G, -1) / total.masked_fill(total == 0, 1)
    out = out.permute(0, 2, 1, 3, 4).reshape(S, T, H, -1).bfloat16()
    n = torch.arange(N, device=dev)
    seq = torch.searchsorted(starts, n, right=True).sub(1).clamp(max=S - 1)
    s["out"].copy_(torch.where((n < starts[-1])[:, None, None], out[seq, (n - starts[seq]).clamp(max=T - 1)], s["out"]))
    return s["out"]


# --- the definitions in 64 bits --------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return _append64(s) if c["op"] == "append" else _attn64(s)


def _row64(s, parts, norm):
    first, rot = parts
    R = rot.shape[-1]
    rot = rot.double().clone()
    first = rot[..., :0] if first is None else first.double().clone()
    if norm is not None:
        w = norm.double()
        if norm.numel() == first.shape[-1]:
            first *= w / (first.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        else:
            rms = (torch.cat((first, rot), -1).pow(2).mean(-1, keepdim=True) + EPS).sqrt()
            first *= (w[R:] if s["rot_first"] else w[:w.numel() - R]) / rms
            rot *= (w[:R] if s["rot_first"] else w[w.numel() - R:]) / rms
    turn = torch.polar(torch.full_like(s["freqs"], s["mscale"]), s["freqs"] * s["positions"].double()[:, None])[:, None]
    if s["interleaved"]:
        z = torch.view_as_complex(rot.view(*rot.shape[:-1], R // 2, 2)) * turn
        rot = torch.view_as_real(z).reshape(rot.shape)
    else:
        z = torch.complex(rot[..., :R // 2], rot[..., R // 2:]) * turn
        rot = torch.cat((z.real, z.imag), -1)
    return torch.cat((rot, first) if s["rot_first"] else (first, rot), -1)


def _append64(s):
    caches = []
    for cache, rows, scale in ((s["cache_k"], _row64(s, s["k_new"], s["k_norm"]), s["scales"][0]), (s["cache_v"], s["v_new"], s["scales"][1])):
        if cache is None:
            caches.append(None)
            continue
        flat = torch.zeros(cache.shape[0] * cache.shape[1], *cache.shape[2:], dtype=torch.float64, device=cache.device)
        rows = rows.double() / scale
        limit = E4M3_MAX if cache.dtype == torch.float8_e4m3fn else math.inf
        for n, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                flat[slot] = rows[n].clamp(-limit, limit)
        caches.append(flat.view(cache.shape))
    return _row64(s, s["q"], s["q_norm"]), caches[0], caches[1]


def _attn64(s):
    page, starts, dev = s["page"], s["starts"].tolist(), s["q"].device
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    G = s["heads"] // s["cache_k"].shape[2]
    for i, length in enumerate(s["lens"].tolist()):
        lo, hi = starts[i], starts[i + 1]
        j = torch.arange(length, device=dev)
        page_ids = s["table"][i].long()[j // page]
        at = torch.arange(length - (hi - lo), length, device=dev)[:, None]
        seen = torch.ones(hi - lo, length, dtype=torch.bool, device=dev)
        if s["causal"]:
            seen &= j <= at
        if s["window"]:
            seen &= j > at - s["window"]
        for head in range(s["heads"]):
            k = s["cache_k"][page_ids, j % page, head // G].double() * s["scales"][0]
            v = k[:, :LATENT] if s["cache_v"] is None else s["cache_v"][page_ids, j % page, head // G].double() * s["scales"][1]
            z = s["scale"] * (s["q"][lo:hi, head].double() @ k.t())
            z[~seen] = -math.inf
            if s["sink"] is not None:
                z = torch.cat((z, s["sink"][head].double().expand(hi - lo, 1)), 1)
            p = torch.softmax(z, dim=1).nan_to_num(0.0)
            out[lo:hi, head] = p[:, :length] @ v
    return out
