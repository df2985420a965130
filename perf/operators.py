"""The operators behind the engram sub-layer, as cases to measure: the residual
addition with RMS norm and an 8-bit output, the append of rotated keys and
values to a paged 8-bit cache, and the attention that reads that cache.

`own` false: elementary torch operations in 32 bits, rounded once at the end.
`own` true: the calls a program makes of libengram.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu


# ---------------------------------------------------------------- cases ----

def _norm(name, rows, dim, x, res, out, block):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "x": x, "res": res, "out": out, "block": block}


def _kv(name, op, batch, q_lo, q_hi, pre_lo, pre_hi, heads, kv_heads, head_dim, page, dtype, **more):
    """Sequences of pre_lo..pre_hi tokens in the cache, each with q_lo..q_hi new ones."""
    return {"name": name, "op": op, "batch": batch, "q_lo": q_lo, "q_hi": q_hi, "pre_lo": pre_lo, "pre_hi": pre_hi,
            "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "dtype": dtype, **more}


def listed():
    return [
        # one token's highway row before its attention: launch latency
        _norm("norm_one_token", 1, 4096, "bf16", "f32", "e8m0", 32),
        # four highway streams of a 4096-token prompt: DRAM bandwidth
        _norm("norm_prompt_streams", 16384, 4096, "bf16", "f32", "e8m0", 32),
        # a ragged batch of a wider model with a 16-bit residual and 128-column scales
        _norm("norm_ragged_16bit", 1537, 5120, "f16", "bf16", "fp8", 128),
        # single-token decode of one sequence after the 2048-token prefix
        _kv("append_one_token", "append", 1, 1, 1, 2048, 2048, 32, 8, 128, 64, "bf16", rot=128, pairs="halves"),
        # decode step of many sequences of unlike lengths, small pages
        _kv("append_decode_batch", "append", 64, 1, 1, 150, 1500, 32, 8, 128, 16, "bf16", rot=128, pairs="halves"),
        # a whole prompt into an empty cache
        _kv("append_prompt", "append", 1, 4096, 4096, 0, 0, 32, 8, 128, 64, "bf16", rot=128, pairs="halves"),
        # chunks of unlike lengths that begin inside pages; 64-wide heads, partly rotated, adjacent pairs, 32-bit input
        _kv("append_ragged_chunks", "append", 9, 1, 700, 0, 900, 12, 4, 64, 32, "f32", rot=32, pairs="adjacent"),
        # single-token decode of one sequence: latency, the cache split over the SMs
        _kv("attention_one_token", "attention", 1, 1, 1, 2048, 2048, 32, 8, 128, 64, "bf16", window=0),
        # decode of a full batch of unlike lengths: DRAM bandwidth
        _kv("attention_decode_batch", "attention", 64, 1, 1, 500, 8191, 32, 8, 128, 16, "bf16", window=0),
        # one very long sequence
        _kv("attention_long_context", "attention", 1, 1, 1, 200000, 200000, 32, 8, 128, 128, "bf16", window=0),
        # the second half of an 8192-token prompt: tensor cores
        _kv("attention_prompt", "attention", 1, 4096, 4096, 4096, 4096, 32, 8, 128, 64, "bf16", window=0),
        # mixed batch: single tokens beside chunks, 64-wide heads shared by 8, sliding window
        _kv("attention_mixed_window", "attention", 12, 1, 600, 100, 5000, 16, 2, 64, 32, "f16", window=1024),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(("norm", "append", "attention", "attention"))
    if op == "norm":
        block = rng.choice((16, 32, 64, 128))
        dim = block * _log(rng, 512 // block, 8192 // block)
        if dim == 3072:
            dim += block
        rows = min(_log(rng, 1, 16384), 50_000_000 // dim)
        return {k: v for k, v in _norm("", rows, dim, rng.choice(("bf16", "f16", "f32")), rng.choice(("f32", "bf16")),
                                       rng.choice(("e8m0", "fp8", "bf16")), block).items() if k != "name"}
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 4, 5, 8))
    if (heads + 2 * kv_heads) * head_dim == 3072:
        heads += kv_heads
    page = rng.choice((16, 32, 64, 128))
    if rng.random() < 0.5:                                   # decode steps
        batch = _log(rng, 1, 64)
        q_lo, q_hi = (1, 1) if rng.random() < 0.7 else (1, 4)
    else:                                                    # prompts and chunks
        batch = _log(rng, 1, 8)
        q_hi = _log(rng, 16, min(4096, 131072 // heads) // batch)
        q_lo = rng.randint(max(1, q_hi // 8), q_hi)
    if op == "append":
        pre = _log(rng, 1, 1500)
        c = _kv("", op, batch, q_lo, q_hi, rng.randint(0, pre), pre, heads, kv_heads, head_dim, page,
                rng.choice(("bf16", "f16", "f32")), rot=rng.choice((0, head_dim // 2, head_dim, head_dim)),
                pairs=rng.choice(("halves", "adjacent")))
    else:
        pre = _log(rng, 16, min(200000, 262144 // batch) if q_hi <= 4 else 4096)
        c = _kv("", op, batch, q_lo, q_hi, rng.randint(pre // 4, pre), pre, heads, kv_heads, head_dim, page,
                rng.choice(("bf16", "f16")), window=rng.choice((0, 0, 0, _log(rng, 16, 2048))))
    c["lens"] = rng.randrange(1 << 20)
    del c["name"]
    return c


def _lens(case):
    """(new tokens, tokens in the cache with them) of each sequence: by the case alone."""
    rng = random.Random(1000 + case.get("lens", 0))
    new, kv = [], []
    for _ in range(case["batch"]):
        n, p = rng.randint(case["q_lo"], case["q_hi"]), rng.randint(case["pre_lo"], case["pre_hi"])
        new.append(n)
        kv.append(n + p)
    return new, kv


def work(case):
    if case["op"] == "norm":
        n, res = case["rows"] * case["dim"], SIZE[case["res"]]
        out = 2 * n if case["out"] == "bf16" else n + n // case["block"] * (4 if case["out"] == "fp8" else 1)
        return {"bytes": n * (SIZE[case["x"]] + 2 * res) + 4 * case["dim"] + out, "flops": 6 * n}
    new, kv = _lens(case)
    H, KH, D, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    rows = sum(new)
    if case["op"] == "append":
        pages = sum((b - 1) // page - (b - a) // page + 1 for a, b in zip(new, kv))
        el = SIZE[case["dtype"]]
        return {"bytes": rows * D * (el * (2 * H + 2 * KH) + 2 * KH) + pages * KH * 2 + rows * case["rot"] * 4,
                "flops": rows * (H + KH) * case["rot"] * 3 + rows * KH * D * 4}
    pairs = read = 0
    w = case["window"]
    for a, b in zip(new, kv):
        first = b - a                                          # the first row's position
        if not w:
            pairs += a * first + a * (a + 1) // 2
            read += b
        else:
            pairs += sum(min(w, p + 1) for p in range(first, b))
            read += b - max(0, first - w + 1)
    return {"bytes": 2 * read * KH * D + 2 * (read + page - 1) // page * KH + rows * H * (2 * 2 * D + 4),
            "flops": 4 * pairs * H * D}


# --------------------------------------------------------------- inputs ----

def _scale_exp(amax):
    """The exponent e of the smallest power of two with amax <= 448 * 2^e (at least -126)."""
    m, e = torch.frexp(amax)                                   # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    s = dict(case)
    if case["op"] == "norm":
        rows, dim, block = case["rows"], case["dim"], case["block"]
        s["x_dtype"], s["res_dtype"] = case["x"], case["res"]
        s["x"], s["res"] = randn(rows, dim, dtype=DT[case["x"]]), randn(rows, dim, dtype=DT[case["res"]]) * 3
        s["w"] = 1 + 0.2 * randn(dim)
        s["res_out"] = torch.empty_like(s["res"])
        if case["out"] == "bf16":
            s["y"], s["scales"] = torch.empty((rows, dim), dtype=torch.bfloat16, device=DEV), None
        else:
            s["y"] = torch.empty((rows, dim), dtype=torch.uint8, device=DEV).view(F8)
            s["scales"] = (torch.empty((rows, dim // block), device=DEV) if case["out"] == "fp8" else
                           torch.empty((rows, dim // block), dtype=torch.uint8, device=DEV).view(E8))
    else:
        new, kv = _lens(case)
        B, H, KH, D, page, dt = (case["batch"], case["heads"], case["kv_heads"], case["head_dim"], case["page"],
                                 DT[case["dtype"]])
        rows = sum(new)
        per = [-(-n // page) for n in kv]
        n_pages = sum(per) + 3                                 # a few pages belong to nobody
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        s["page_table"] = torch.zeros((B, max(per)), dtype=torch.int32, device=DEV)
        owner = torch.arange(max(per), device=DEV)[None, :] < torch.tensor(per, device=DEV)[:, None]
        s["page_table"][owner] = order[: sum(per)]
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        s["row_start"] = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV)
        s["rows"], s["n_max"], s["pages_of"] = rows, max(new), max(per)
        for name in ("k", "v"):
            codes = torch.empty((n_pages, KH, page, D), dtype=torch.uint8, device=DEV)
            scales = torch.empty((n_pages, KH), dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 28) // (KH * page * D))
            for i in range(0, n_pages, step):
                # heads of unlike size, now and then a large token
                x = randn(min(step, n_pages - i), KH, page, D)
                x *= torch.exp(0.5 * randn(1, KH, 1, 1)) * torch.exp(0.3 * randn(x.shape[0], 1, page, 1))
                e = _scale_exp(x.abs().amax((2, 3)))
                codes[i:i + step] = torch.ldexp(x, -e[:, :, None, None]).to(F8).view(torch.uint8)
                scales[i:i + step] = (e + 127).to(torch.uint8)
            s[name + "_cache"], s[name + "_scales"] = codes.view(F8), scales.view(E8)
        # q, k and v as the projection leaves them: side by side in one row
        qkv = randn(rows, (H + 2 * KH) * D, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, : H * D], qkv[:, H * D: (H + KH) * D], qkv[:, (H + KH) * D:]
        s["out"] = torch.empty((rows, H * D), dtype=dt, device=DEV)
        if case["op"] == "append":
            at = torch.arange(max(kv), device=DEV, dtype=torch.float64)
            f = 10000.0 ** (-torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64) / max(1, case["rot"] // 2))
            s["rope"] = torch.stack([(at[:, None] * f).cos(), (at[:, None] * f).sin()], -1).float().contiguous()
        else:
            s["lse"] = torch.empty((rows, H), device=DEV)
            s["scale"] = D ** -0.5
    if own:
        s.update(_handles(s))
    return s


def _handles(s):
    """What a program keeps beside its tensors: the descriptors of its cache and batch, and the attention's workspace."""
    from deepseek_v4_engram_hash_gb300 import _lib as E
    types = {"bf16": E.ENGRAM_T_BF16, "f16": E.ENGRAM_T_F16, "f32": E.ENGRAM_T_F32}
    h = {"E": E}
    if s["op"] == "norm":
        h["x_type"], h["res_type"] = types[s["x_dtype"]], types[s["res_dtype"]]
        h["fmt"] = {"fp8": E.ENGRAM_FMT_FP8, "e8m0": E.ENGRAM_FMT_FP8_E8M0, "bf16": E.ENGRAM_FMT_BF16}[s["out"]]
        return h
    h["type"], h["stride"] = types[s["dtype"]], s["q"].stride(0)
    h["cache"] = E.KvCache(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["k_cache"].shape[0],
                           s["kv_heads"], s["page"], s["head_dim"])
    h["plan"] = E.KvBatch(s["page_table"], s["kv_len"], s["row_start"], s["batch"], s["pages_of"], s["rows"],
                          s["n_max"])
    if s["op"] == "attention":
        h["attn"] = E.Attention()
    else:
        h["turn"] = E.Rope(s["rope"], s["rope"].shape[0], s["rot"], s["pairs"] == "adjacent") if s["rot"] else None
    return h


# ------------------------------------------------------------ the passes ----

def run(s):
    if s["op"] == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    if s["op"] == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_attention(s) if own else _plain_attention(s)


def _norm_outputs(s, res, y, scales):
    return {"res": res, "y": y} if scales is None else {"res": res, "y": y, "scales": scales}


def _own_norm(s):
    s["E"].engram_residual_norm(s["x"], s["x_type"], s["res"], s["res_type"], s["res_out"], s["w"], s["rows"], s["dim"],
                                EPS, s["fmt"], s["block"], s["y"], s["scales"])
    return _norm_outputs(s, s["res_out"], s["y"], s["scales"])


def _plain_norm(s):
    r = s["res"].float() + s["x"].float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w"]
    res = r.to(s["res"].dtype)
    if s["out"] == "bf16":
        return _norm_outputs(s, res, y.to(torch.bfloat16), None)
    y = y.view(s["rows"], -1, s["block"])
    e = _scale_exp(y.abs().amax(2))
    codes = torch.ldexp(y, -e[:, :, None]).to(F8).view(s["rows"], s["dim"])
    if s["out"] == "fp8":
        return _norm_outputs(s, res, codes, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e))
    return _norm_outputs(s, res, codes, (e + 127).to(torch.uint8).view(E8))


def _cache_outputs(s, q):
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _own_append(s):
    s["E"].engram_kv_append(s["cache"], s["plan"], s["type"], s["k"], s["stride"], s["v"], s["stride"], s["q"], s["stride"],
                            s["out"], 0, s["heads"], s["turn"])
    return _cache_outputs(s, s["out"])


def _row_places(s):
    """Of every row: its sequence, its number in the sequence's new tokens and its position."""
    start = s["row_start"].long()
    r = torch.arange(s["rows"], device=start.device)
    b = torch.searchsorted(start, r, right=True) - 1
    i = r - start[b]
    return b, i, s["kv_len"].long()[b] - (start[b + 1] - start[b]) + i


def _rotate(x, cs, rot, pairs):
    """x [rows, heads, D] in 32 bits, cs [rows, 1, rot / 2, 2]."""
    if not rot:
        return x
    c, sn = cs[..., 0], cs[..., 1]
    if pairs == "adjacent":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _store(s, x, codes, scales, b, pos, n_new):
    """x [rows, KH, D] in 32 bits into the pages of its rows' positions."""
    codes, scales = codes.view(torch.uint8), scales.view(torch.uint8)
    page, KH, D = s["page"], s["kv_heads"], s["head_dim"]
    first = s["kv_len"].long() - n_new                         # tokens already there
    span = (s["n_max"] + page - 2) // page + 1                 # pages that a sequence can touch
    u = first[:, None] // page + torch.arange(span, device=x.device)
    touched = u * page < s["kv_len"].long()[:, None]
    at = s["page_table"].long().gather(1, u.clamp(max=s["pages_of"] - 1))
    held = codes[at].view(F8).float()                          # [B, span, KH, page, D]
    where = u[..., None] * page + torch.arange(page, device=x.device)
    old = where < first[:, None, None]                         # [B, span, page]
    fresh = torch.zeros_like(held)
    fresh[b, pos // page - first[b] // page, :, pos % page] = x
    e_new = _scale_exp(fresh.abs().amax((3, 4)))
    e_old = torch.where(old.any(2)[..., None], scales[at].int() - 127, torch.full_like(e_new, -126))
    e = torch.maximum(e_new, e_old)
    kept = torch.ldexp(held, (e_old - e)[..., None, None]).to(F8)
    put = torch.ldexp(fresh, -e[..., None, None]).to(F8)
    is_new = (~old & (where < s["kv_len"].long()[:, None, None]))[:, :, None, :, None]
    now = torch.where(is_new, put.view(torch.uint8), torch.where(old[:, :, None, :, None], kept.view(torch.uint8), codes[at]))
    codes[at[touched]] = now[touched]
    scales[at[touched]] = (e + 127).to(torch.uint8)[touched]


def _plain_append(s):
    D = s["head_dim"]
    b, _, pos = _row_places(s)
    n_new = (s["row_start"][1:] - s["row_start"][:-1]).long()
    cs = s["rope"][pos][:, None]
    k = _rotate(s["k"].float().view(s["rows"], -1, D), cs, s["rot"], s["pairs"])
    q = _rotate(s["q"].float().view(s["rows"], -1, D), cs, s["rot"], s["pairs"])
    _store(s, k, s["k_cache"], s["k_scales"], b, pos, n_new)
    _store(s, s["v"].float().view(s["rows"], -1, D), s["v_cache"], s["v_scales"], b, pos, n_new)
    return _cache_outputs(s, q.flatten(1).to(s["q"].dtype))


def _own_attention(s):
    s["E"].engram_attention(s["attn"], s["cache"], s["plan"], s["type"], s["q"], s["stride"], s["heads"], s["scale"],
                            s["window"], s["out"], 0, s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attention(s):
    B, H, KH, D, page = s["batch"], s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    b, i, pos = _row_places(s)
    pt = s["page_table"].long()

    def tokens(codes, scales):                                 # [B, KH, L, D]
        x = codes.view(torch.uint8)[pt].view(F8).float()
        x *= torch.exp2(scales.view(torch.uint8)[pt].float() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, KH, -1, D)

    k, v = tokens(s["k_cache"], s["k_scales"]), tokens(s["v_cache"], s["v_scales"])
    n, L = s["n_max"], k.shape[2]
    q = torch.zeros((B, n, H, D), device=k.device)
    q[b, i] = s["q"].float().view(-1, H, D)
    at = torch.full((B, n), -1, device=k.device)
    at[b, i] = pos
    q = q.view(B, n, KH, H // KH, D).permute(0, 2, 3, 1, 4).reshape(B, KH, -1, D)
    sc = (q @ k.transpose(2, 3)).view(B, H, n, L) * s["scale"]
    j = torch.arange(L, device=k.device)
    seen = j <= at[..., None]
    if s["window"]:
        seen &= j > at[..., None] - s["window"]
    sc.masked_fill_(~seen[:, None], -math.inf)
    m = sc.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp_(sc.sub_(m))
    total = p.sum(3, keepdim=True)
    o = (p.view(B, KH, -1, L) @ v).view(B, H, n, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).view(B, H, n)
    return {"out": o.permute(0, 2, 1, 3)[b, i].flatten(1).to(s["q"].dtype), "lse": lse.permute(0, 2, 1)[b, i]}


# ----------------------------------------------------- from the definition ----

def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)


def _e4m3(y):
    """The nearest e4m3 value (ties to even) of y in 64 bits, |y| <= 448."""
    _, e = torch.frexp(y.abs())
    step = _pow2((e - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _code_values():
    c = torch.arange(256, device=DEV)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * _pow2(e - 7), m / 8 * 2.0 ** -6)
    return torch.where(c >= 128, -v, v)


def _block_scale(amax):
    """The smallest power of two that is at least amax / 448, and at least 2^-126."""
    m, e = torch.frexp(amax / 448)
    return torch.where(amax > 0, _pow2(torch.where(m == 0.5, e - 1, e)), torch.zeros_like(amax)).clamp(min=2.0 ** -126)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "append": _exact_append, "attention": _exact_attention}[case["op"]](s)


def _exact_norm(s):
    r = s["res"].double() + s["x"].double()
    y = r / torch.sqrt(r.square().sum(1, keepdim=True) / s["dim"] + EPS) * s["w"].double()
    if s["out"] == "bf16":
        return {"res": r, "y": y}
    y = y.view(s["rows"], s["dim"] // s["block"], s["block"])
    sc = _block_scale(y.abs().amax(2))
    return {"res": r, "y": _e4m3(y / sc[..., None]).view(s["rows"], s["dim"]), "scales": sc}


def _exact_append(s):
    D, page, rot = s["head_dim"], s["page"], s["rot"]
    start, kv, table = s["row_start"].tolist(), s["kv_len"].tolist(), s["page_table"].tolist()
    value = _code_values()

    def turned(x, at):
        x = x.double().view(x.shape[0], -1, D).clone()
        z = torch.view_as_complex(s["rope"].double())[at][:, None]
        if not rot:
            return x
        if s["pairs"] == "adjacent":
            w = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2)) * z
            x[..., :rot] = torch.view_as_real(w).flatten(2)
        else:
            w = torch.complex(x[..., : rot // 2], x[..., rot // 2: rot]) * z
            x[..., :rot] = torch.cat([w.real, w.imag], -1)
        return x

    out = {"q": torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)}
    for name in ("k", "v"):
        codes = value[s[name + "_cache"].view(torch.uint8).long()]
        scales = _pow2(s[name + "_scales"].view(torch.uint8).int() - 127)
        for b, n in enumerate(kv):
            rows = slice(start[b], start[b + 1])
            old = n - (start[b + 1] - start[b])
            at = torch.arange(old, n, device=DEV)
            if name == "k":
                out["q"][rows] = turned(s["q"][rows], at).flatten(1)
            x = turned(s["k"][rows], at) if name == "k" else s["v"][rows].double().view(n - old, -1, D)
            for p in range(old // page, (n - 1) // page + 1):
                lo, hi = max(old, p * page), min(n, (p + 1) * page)
                have, g = lo - p * page, table[b][p]
                part = x[lo - old: hi - old].transpose(0, 1)       # [KH, tokens, D]
                sc = _block_scale(part.abs().amax((1, 2)))
                if have:
                    sc = torch.maximum(sc, scales[g])
                    codes[g, :, :have] = _e4m3(codes[g, :, :have] * (scales[g] / sc)[:, None, None])
                codes[g, :, have: have + hi - lo] = _e4m3(part / sc[:, None, None])
                scales[g] = sc
        out[name], out[name + "_scales"] = codes, scales
    return out


def _exact_attention(s):
    D, page, H, KH, w = s["head_dim"], s["page"], s["heads"], s["kv_heads"], s["window"]
    start, kv, table = s["row_start"].tolist(), s["kv_len"].tolist(), s["page_table"].long()
    value = _code_values()
    out = torch.empty((s["rows"], H, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["rows"], H), dtype=torch.float64, device=DEV)
    for b, n in enumerate(kv):
        pages = table[b, : -(-n // page)]
        at = torch.arange(start[b], start[b + 1], device=DEV) - start[b + 1] + n
        j = torch.arange(n, device=DEV)
        hide = j[None, :] > at[:, None]
        if w:
            hide |= at[:, None] - j[None, :] >= w
        for kh in range(KH):
            k, v = ((value[s[c + "_cache"].view(torch.uint8)[pages, kh].long()]
                     * _pow2(s[c + "_scales"].view(torch.uint8)[pages, kh].int() - 127)[:, None, None])
                    .reshape(-1, D)[:n] for c in ("k", "v"))
            for h in range(kh * (H // KH), (kh + 1) * (H // KH)):
                q = s["q"][start[b]: start[b + 1], h * D: (h + 1) * D].double()
                z = ((q @ k.T) * s["scale"]).masked_fill(hide, -math.inf)
                lse[start[b]: start[b + 1], h] = torch.logsumexp(z, 1)
                out[start[b]: start[b + 1], h] = torch.softmax(z, 1) @ v
    return {"out": out.flatten(1), "lse": lse}
