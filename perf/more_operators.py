"""The operators of the experts' sub-layer, as cases to measure: routing of tokens
to experts, the product of e4m3 rows with e4m3 weights (a scale for each block of
128), the gated pair of such products with an 8-bit output, and the weighted sum
of the experts' outputs.

`own` false: elementary torch operations in 32 bits (scores that decide a choice
in 64), rounded once at the end.  `own` true: the calls a program makes of libengram.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu
B = 128                                                        # values a scale block


# ---------------------------------------------------------------- cases ----

def _route(name, tokens, experts, k, dtype, score, bias, groups, top_groups, best, renorm):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "k": k, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "top_groups": top_groups, "best": best, "renorm": renorm}


def _dense(name, op, rows, K, N, xfmt, wfmt, out):
    """One matrix for all rows; op "project" (out: element type) or "glu" (N: values a row of the output; out: its scales)."""
    return {"name": name, "op": op, "tokens": rows, "K": K, "N": N, "xfmt": xfmt, "wfmt": wfmt, "out": out, "experts": 0,
            "k": 1, "limit": 0.0}


def _experts(name, op, tokens, k, experts, K, N, xfmt, wfmt, out):
    """A matrix (pair) for each expert, k experts a token."""
    return {**_dense(name, op, tokens, K, N, xfmt, wfmt, out), "experts": experts, "k": k}


def _combine(name, tokens, k, dim, dtype, add, out):
    return {"name": name, "op": "combine", "tokens": tokens, "k": k, "dim": dim, "dtype": dtype, "add": add, "out": out}


def listed():
    return [
        # the router of one decoded token: launch latency
        _route("route_one_token", 1, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True),
        # a long prompt's tokens at once
        _route("route_prompt", 16384, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True),
        # query, key and value projection of one decoded token: the weight is read once, its latency counts
        _dense("project_one_token", "project", 1, 4096, 6144, "e8m0", "e8m0", "bf16"),
        # the same kind of product for a prompt: tensor cores
        _dense("project_prompt", "project", 8192, 4096, 6144, "e8m0", "e8m0", "bf16"),
        # a wider model's batch of odd size onto a narrow, odd output in 32 bits, weights with scales that are no powers of two
        _dense("project_ragged", "project", 777, 5120, 1000, "fp8", "fp8", "f32"),
        # the gated half of a token's eight experts: DRAM bandwidth
        _experts("glu_one_token", "glu", 1, 8, 256, 4096, 2048, "e8m0", "e8m0", "e8m0"),
        # a decode batch that touches most experts with a row or two each
        _experts("glu_decode_batch", "glu", 64, 8, 256, 4096, 2048, "e8m0", "e8m0", "e8m0"),
        # a prompt through its experts: tensor cores on unlike row counts
        _experts("glu_prompt", "glu", 4096, 8, 64, 4096, 1024, "e8m0", "fp8", "e8m0"),
        # the second product of the decode batch
        _experts("down_decode_batch", "project", 64, 8, 256, 2048, 4096, "e8m0", "e8m0", "bf16"),
        # the second product of the prompt
        _experts("down_prompt", "project", 4096, 8, 64, 1024, 4096, "e8m0", "fp8", "bf16"),
        # a decode batch's outputs summed onto the shared expert's
        _combine("combine_decode_batch", 64, 8, 4096, "bf16", True, "bf16"),
        # a prompt's
        _combine("combine_prompt", 4096, 8, 4096, "bf16", False, "bf16"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(("route", "project", "project", "glu", "glu", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        k = min(rng.randint(1, 12), experts // groups * top_groups)
        c = _route("", min(_log(rng, 1, 16384), 4194304 // experts), experts, k, rng.choice(("f32", "bf16", "f16")),
                   rng.choice(("sigmoid", "softmax")), rng.random() < 0.6, groups, top_groups, rng.choice((1, 2)),
                   rng.random() < 0.7)
    elif op == "combine":
        dim, k = 8 * _log(rng, 32, 1024), rng.randint(1, 12)
        c = _combine("", min(_log(rng, 1, 4096), 134217728 // (dim * k)), k, dim, rng.choice(("bf16", "f16", "f32")),
                     rng.random() < 0.5, rng.choice(("bf16", "f16", "f32")))
    else:
        K, N = 16 * _log(rng, 16, 400), _log(rng, 64, 8192)
        if op == "glu":
            N = max(16, N // 32 * 16)
        wide = N * (2 if op == "glu" else 1)
        fmts = rng.choice(("e8m0", "fp8")), rng.choice(("e8m0", "fp8"))
        out = rng.choice(("bf16", "f16", "f32")) if op == "project" else rng.choice(("e8m0", "fp8"))
        most = 2 ** 37 // (K * wide)                           # rows that cost half of the largest listed case
        if rng.random() < 0.5:
            c = _dense("", op, min(_log(rng, 1, 8192), most), K, N, *fmts, out)
        else:
            experts = min(_log(rng, 4, 256), 2 ** 32 // (K * wide))
            k = min(rng.randint(1, 8), experts)
            c = _experts("", op, min(_log(rng, 1, 4096), most // k), k, experts, K, N, *fmts, out)
        if op == "glu" and rng.random() < 0.3:
            c["limit"] = 1.5
    del c["name"]
    c["lists"] = rng.randrange(1 << 20)
    return c


def _choices(case):
    """[tokens, k] experts of each token, some experts more popular than others: by the case alone."""
    g = torch.Generator().manual_seed(1000 + case.get("lists", 0))
    z = torch.randn(case["tokens"], case["experts"], generator=g) + 0.5 * torch.randn(case["experts"], generator=g)
    return torch.topk(z, case["k"]).indices


def work(case):
    T, k = case["tokens"], case["k"]
    if case["op"] == "route":
        n = T * case["experts"]
        return {"bytes": n * SIZE[case["dtype"]] + 4 * case["experts"] * (1 + case["bias"]) + 12 * T * k, "flops": 8 * n}
    if case["op"] == "combine":
        D = case["dim"]
        return {"bytes": T * (k * (D * SIZE[case["dtype"]] + 4) + D * SIZE[case["out"]] * (1 + case["add"])),
                "flops": 2 * T * k * D}
    K, N = case["K"], case["N"]
    KB, NB = -(-K // B), -(-N // B)
    pairs, glu = T * k, case["op"] == "glu"
    used = len(torch.unique(_choices(case))) if case["experts"] else 1
    sx, sw = (1 if case[f] == "e8m0" else 4 for f in ("xfmt", "wfmt"))
    rows = T if glu or not case["experts"] else pairs          # rows of x
    out = pairs * (N + NB * (1 if case["out"] == "e8m0" else 4)) if glu else pairs * N * SIZE[case["out"]]
    wide = 2 if glu else 1
    return {"bytes": rows * (K + KB * sx) + used * wide * (N * K + NB * KB * sw) + out, "flops": 2 * wide * pairs * N * K}


# --------------------------------------------------------------- inputs ----

def _scale_exp(amax):
    """The exponent e of the smallest power of two with amax <= 448 * 2^e (at least -126)."""
    m, e = torch.frexp(amax)                                   # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def _as_scales(e, fmt):
    """The powers of two of the exponents e as a program holds them."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e) if fmt == "fp8" else (e + 127).to(torch.uint8).view(E8)


def _quantise_rows(y, fmt):
    """Codes [rows, K] and scales [rows, ceil(K / 128)] of y in 32 bits: a power of two for each block of a row."""
    rows, K = y.shape
    y = torch.nn.functional.pad(y, (0, -K % B)).view(rows, -1, B)
    e = _scale_exp(y.abs().amax(2))
    codes = torch.ldexp(y, -e[:, :, None]).to(F8).view(rows, -1)[:, :K].contiguous()
    return codes, _as_scales(e, fmt)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)

    s = dict(case)
    T, k = case["tokens"], case["k"]
    if case["op"] == "route":
        E = case["experts"]
        s["logits"] = (1.5 * randn(T, E)).to(DT[case["dtype"]])
        s["b"] = 0.1 * randn(E) if case["bias"] else None
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((T, k), device=DEV)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["pairs"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        s["factor"] = 2.5
    elif case["op"] == "combine":
        D = case["dim"]
        s["y"] = randn(T * k, D).to(DT[case["dtype"]])
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["added"] = randn(T, D).to(DT[case["out"]]) if case["add"] else None
        s["result"] = torch.empty((T, D), dtype=DT[case["out"]], device=DEV)
    else:
        _prepare_product(s, randn)
    if own:
        s.update(_handles(s))
    return s


def _prepare_product(s, randn):
    T, k, K, N, E, glu = s["tokens"], s["k"], s["K"], s["N"], s["experts"], s["op"] == "glu"
    pairs = T * k
    KB, NB = -(-K // B), -(-N // B)
    rows = T if glu or not E else pairs
    # rows as a norm leaves them, a few channels larger than the others
    x = randn(rows, K) * torch.exp(0.4 * randn(K))
    s["x"], s["x_scales"] = _quantise_rows(x, s["xfmt"])
    # weights of unlike size from block to block
    n_mats = max(1, E) * (2 if glu else 1)
    codes = torch.empty((n_mats, N, K), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n_mats, NB, KB), dtype=torch.float32 if s["wfmt"] == "fp8" else torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for i in range(0, n_mats, step):
        n = min(step, n_mats - i)
        w = randn(n, N, K) * (K ** -0.5 * (2.0 if glu else 1.0))
        w = torch.nn.functional.pad(w, (0, -K % B, 0, -N % B)).view(n, NB, B, KB, B)
        w *= torch.exp(0.3 * randn(n, NB, 1, KB, 1))
        amax = w.abs().amax((2, 4))
        if s["wfmt"] == "fp8":
            scales[i: i + n] = amax / 448
            w = w / scales[i: i + n, :, None, :, None]
        else:
            e = _scale_exp(amax)
            scales[i: i + n] = (e + 127).to(torch.uint8)
            w = torch.ldexp(w, -e[:, :, None, :, None])
        codes[i: i + n] = w.to(F8).view(torch.uint8).view(n, NB * B, KB * B)[:, :N, :K]
    s["w"], s["w_scales"] = codes.view(F8), scales if s["wfmt"] == "fp8" else scales.view(E8)
    if E:
        ids = _choices(s).flatten()
        order = torch.argsort(ids, stable=True)
        counts = torch.bincount(ids, minlength=E)
        s["pairs"] = order.to(torch.int32).to(DEV)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(torch.int32).to(DEV)
        s["most"] = int(counts.max())
    if glu:
        s["codes"] = torch.empty((pairs, N), dtype=torch.uint8, device=DEV).view(F8)
        s["scales"] = (torch.empty((pairs, NB), device=DEV) if s["out"] == "fp8" else
                       torch.empty((pairs, NB), dtype=torch.uint8, device=DEV).view(E8))
    else:
        s["result"] = torch.empty((pairs, N), dtype=DT[s["out"]], device=DEV)


def _handles(s):
    """What a program keeps beside its tensors: descriptors of its weights and lists, the router's workspace."""
    from deepseek_v4_engram_hash_gb300 import _lib as E
    types = {"bf16": E.ENGRAM_T_BF16, "f16": E.ENGRAM_T_F16, "f32": E.ENGRAM_T_F32}
    fmts = {"fp8": E.ENGRAM_FMT_FP8, "e8m0": E.ENGRAM_FMT_FP8_E8M0}
    h = {"L": E}
    if s["op"] == "route":
        h["type"] = types[s["dtype"]]
        h["router"] = E.Router(s["experts"], s["k"], E.ENGRAM_SCORE_SIGMOID if s["score"] == "sigmoid" else
                               E.ENGRAM_SCORE_SOFTMAX, s["groups"], s["top_groups"], s["best"], s["renorm"], s["factor"])
        h["lists"] = E.ExpertLists(s["offsets"], s["pairs"], s["experts"], s["k"], s["tokens"])
        h["ws_bytes"] = E.engram_route_workspace_bytes(s["experts"], s["tokens"])
        h["ws"] = torch.empty(h["ws_bytes"], dtype=torch.uint8, device=DEV)
    elif s["op"] == "combine":
        h["type"], h["out_type"] = types[s["dtype"]], types[s["out"]]
    else:
        h["weight"] = E.Fp8Weight(s["w"], s["w_scales"], fmts[s["wfmt"]], max(1, s["experts"]), s["N"], s["K"],
                                  s["op"] == "glu")
        h["x_format"] = fmts[s["xfmt"]]
        h["lists"] = E.ExpertLists(s["offsets"], s["pairs"], s["experts"], s["k"], s["tokens"]) if s["experts"] else None
        h["out_kind"] = fmts[s["out"]] if s["op"] == "glu" else types[s["out"]]
    return h


# ------------------------------------------------------------ the passes ----

def run(s):
    return {"route": _own_route if own else _plain_route, "combine": _own_combine if own else _plain_combine,
            "project": _own_project if own else _plain_project, "glu": _own_glu if own else _plain_glu}[s["op"]](s)


def _own_route(s):
    s["L"].engram_route(s["router"], s["type"], s["logits"], 0, s["b"], s["tokens"], s["ids"], s["weights"], s["lists"],
                        s["ws"], s["ws_bytes"])
    return {"ids": s["ids"], "weights": s["weights"], "offsets": s["offsets"], "pairs": s["pairs"]}


def _own_project(s):
    s["L"].engram_project_fp8(s["x"], 0, s["x_scales"], s["x_format"], s["x"].shape[0], s["weight"], s["lists"],
                              s["out_kind"], s["result"], 0)
    return {"out": s["result"]}


def _own_glu(s):
    s["L"].engram_glu_fp8(s["x"], 0, s["x_scales"], s["x_format"], s["x"].shape[0], s["weight"], s["lists"], s["limit"],
                          s["out_kind"], s["codes"], s["scales"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_combine(s):
    s["L"].engram_combine(s["y"], s["type"], 0, s["weights"], s["tokens"], s["k"], s["dim"], s["added"], s["out_type"], 0,
                          s["out_type"], s["result"], 0)
    return {"out": s["result"]}


def _best(c, k):
    """The k largest of each row, ties to the lower index."""
    return torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s):
    T, E, k, G = s["tokens"], s["experts"], s["k"], s["groups"]
    z = s["logits"].double()
    if s["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
    else:
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    c = z if s["b"] is None else p + s["b"].double()
    if s["top_groups"] < G:
        of = c if s["best"] == 1 or s["b"] is not None else p
        group = torch.sort(of.view(T, G, E // G), dim=2, descending=True).values[:, :, : s["best"]].sum(2)
        keep = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, _best(group, s["top_groups"]), True)
        c = c.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    ids = _best(c, k)
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    flat = ids.flatten()
    counts = (flat[:, None] == torch.arange(E, device=z.device)).sum(0)
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)])
    return {"ids": ids.int(), "weights": (w * s["factor"]).float(), "offsets": offsets.int(),
            "pairs": torch.sort(flat, stable=True).indices.int()}


def _scales32(t):
    """Scales in 32 bits."""
    return t if t.dtype == torch.float32 else torch.exp2(t.view(torch.uint8).float() - 127)


def _rows32(s):
    x = s["x"].float()
    return x * _scales32(s["x_scales"]).repeat_interleave(B, 1)[:, : s["K"]]


def _weights32(s, mats):
    """Matrices `mats` (all: None) in 32 bits."""
    w, sc = (s["w"], s["w_scales"]) if mats is None else (s["w"].view(torch.uint8)[mats].view(F8),
                                                          s["w_scales"].view(s["w_scales"].dtype if s["wfmt"] == "fp8"
                                                                             else torch.uint8)[mats])
    sc = _scales32(sc).repeat_interleave(B, 1)[:, : s["N"]]
    return w.float().mul_(sc.repeat_interleave(B, 2)[:, :, : s["K"]])


def _products32(s):
    """x W^T of every pair in the lists' order: [pairs, N], for "glu" [pairs, 2, N]."""
    K, N, E = s["K"], s["N"], s["experts"]
    m = 2 if s["op"] == "glu" else 1
    x = _rows32(s)
    if not E:
        return (x @ _weights32(s, None).view(m * N, K).T).view(-1, m, N)
    n = s["pairs"].numel()
    at = torch.arange(n, device=x.device)
    e = torch.searchsorted(s["offsets"].long(), at, right=True) - 1
    if s["op"] == "glu":
        x = x[s["pairs"].long() // s["k"]]
    if n <= E:
        mats = (e[:, None] * m + torch.arange(m, device=x.device)).flatten()
        return torch.bmm(_weights32(s, mats).view(n, m * N, K), x[:, :, None]).view(n, m, N)
    within = at - s["offsets"].long()[e]
    padded = torch.zeros((E, s["most"], K), device=x.device)
    padded[e, within] = x
    return torch.bmm(padded, _weights32(s, None).view(E, m * N, K).transpose(1, 2))[e, within].view(n, m, N)


def _plain_project(s):
    y = _products32(s)[:, 0].to(DT[s["out"]])
    if s["experts"]:
        back = torch.empty_like(y)
        back[s["pairs"].long()] = y
        y = back
    return {"out": y}


def _plain_glu(s):
    g, u = _products32(s).unbind(1)
    if s["limit"]:
        g, u = g.clamp(max=s["limit"]), u.clamp(-s["limit"], s["limit"])
    codes, scales = _quantise_rows(g / (1 + torch.exp(-g)) * u, s["out"])
    return {"codes": codes, "scales": scales}


def _plain_combine(s):
    y = s["y"].float().view(s["tokens"], s["k"], s["dim"])
    w = s["weights"][:, :, None]
    o = torch.where(w == 0, torch.zeros_like(y), y * w).sum(1)
    return {"out": (o if s["added"] is None else o + s["added"].float()).to(DT[s["out"]])}


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
    if case["op"] in ("project", "glu") and work(case)["flops"] > 1e13:
        return None                                            # 64-bit products of that size take minutes
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "combine": _exact_combine, "project": _exact_product, "glu": _exact_product}[s["op"]](s)


def _exact_route(s):
    z = s["logits"].double().cpu()
    T, E, G, k = s["tokens"], s["experts"], s["groups"], s["k"]
    p = torch.sigmoid(z) if s["score"] == "sigmoid" else torch.softmax(z, 1)
    b = None if s["b"] is None else s["b"].double().cpu()
    c = z if b is None else p + b
    if s["top_groups"] < G:
        of = (p if b is None and s["best"] == 2 else c).view(T, G, E // G)
        g = of.topk(min(s["best"], E // G), 2).values.sum(2)
        for _ in range(G - s["top_groups"]):
            # the worst of the groups that are left, of equal ones the last
            worst = G - 1 - g.flip(1).argmin(1)
            g[torch.arange(T), worst] = math.inf
            c = c.clone()
            c.view(T, G, E // G)[torch.arange(T), worst] = -math.inf
    ids = torch.empty((T, k), dtype=torch.int64)
    c = c.clone()
    for j in range(k):
        ids[:, j] = c.argmax(1)
        c[torch.arange(T), ids[:, j]] = -math.inf
    w = torch.stack([p[torch.arange(T), ids[:, j]] for j in range(k)], 1)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    flat = ids.flatten()
    of_expert = [torch.nonzero(flat == e).flatten() for e in range(E)]
    offsets = [0]
    for m in of_expert:
        offsets.append(offsets[-1] + len(m))
    return {"ids": ids.int().to(DEV), "weights": (w * s["factor"]).to(DEV),
            "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV), "pairs": torch.cat(of_expert).int().to(DEV)}


def _exact_product(s):
    K, N, E, glu = s["K"], s["N"], s["experts"], s["op"] == "glu"
    value = _code_values()
    m = 2 if glu else 1

    def scale(t):
        return t.double() if t.dtype == torch.float32 else _pow2(t.view(torch.uint8).int() - 127)

    def spread(sc, n):
        return sc[..., torch.arange(n, device=DEV) // B]

    x = value[s["x"].view(torch.uint8).long()] * spread(scale(s["x_scales"]), K)
    n = s["tokens"] * s["k"]
    out = torch.empty((n, m, N), dtype=torch.float64, device=DEV)
    w8, wsc = s["w"].view(torch.uint8), s["w_scales"] if s["wfmt"] == "fp8" else s["w_scales"].view(torch.uint8)
    starts = s["offsets"].tolist() if E else [0, n]
    for e in range(max(1, E)):
        lo, hi = starts[e], starts[e + 1]
        if lo == hi:
            continue
        rows = torch.arange(lo, hi, device=DEV)
        mine = x[rows] if not E or not glu else x[s["pairs"][lo:hi].long() // s["k"]]
        for i in range(m):
            w = value[w8[e * m + i].long()]
            sc = scale(wsc[e * m + i] if s["wfmt"] == "fp8" else wsc[e * m + i].view(E8))
            w *= spread(sc[torch.arange(N, device=DEV) // B], K)
            out[lo:hi, i] = mine @ w.T
    if not glu:
        y = out[:, 0]
        if E:
            back = torch.empty_like(y)
            back[s["pairs"].long()] = y
            y = back
        return {"out": y}
    gate, up = out[:, 0], out[:, 1]
    if s["limit"]:
        gate, up = torch.minimum(gate, torch.full_like(gate, s["limit"])), up.clamp(-s["limit"], s["limit"])
    a = torch.nn.functional.pad(torch.sigmoid(gate) * gate * up, (0, -N % B)).view(n, -1, B)
    sc = _block_scale(a.abs().amax(2))
    return {"codes": _e4m3(a / sc[..., None]).view(n, -1)[:, :N], "scales": sc}


def _exact_combine(s):
    w = s["weights"].double()
    o = torch.einsum("tk,tkd->td", w, s["y"].double().view(s["tokens"], s["k"], s["dim"]))
    return {"out": o if s["added"] is None else o + s["added"].double()}
