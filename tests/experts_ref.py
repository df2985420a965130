"""The experts' sub-layer's operators from their definitions in 64 bits (tests
only): plain torch and Python, no code of the CUDA path."""
import math

import torch

import sublayer_ref as R

B = 128


def scale_values(s):
    """Scales in 64 bits: f32, or e8m0 bytes (255: NaN)."""
    if s.dtype == torch.float32:
        return s.double()
    v = R.pow2(s.view(torch.uint8).int() - 127)
    return torch.where(s.view(torch.uint8) == 255, torch.full_like(v, math.nan), v)


def rows64(codes, scales):
    """codes [rows, K] u8 with scales [rows, ceil(K / 128)]."""
    at = torch.arange(codes.shape[-1], device=codes.device) // B
    return R.e4m3_values().to(codes.device)[codes.long()] * scale_values(scales)[:, at]


def weight64(codes, scales):
    """codes [N, K] u8 with scales [ceil(N / 128), ceil(K / 128)]."""
    n, k = (torch.arange(m, device=codes.device) // B for m in codes.shape)
    return R.e4m3_values().to(codes.device)[codes.long()] * scale_values(scales)[n][:, k]


def product(x, w):
    """x W^T of 64-bit rows and weights, and the sum of the products' sizes."""
    return x @ w.T, x.abs() @ w.abs().T


def sum_error(K):
    """The relative bound (of the products' sizes) on a sum of K exact products that is added up in f32, each addition cut off or
    rounded (2^-23 of a partial sum): blocks of 128 in any order, the factor sx sw (2^-24) and one FMA a block (2^-24); or 32 products
    in any order at a time onto the running sum (power-of-two factors are exact).  Up to 8 partial sums are then added."""
    return (max(B + 1 + (K + B - 1) // B, 32 + (K + 31) // 32) + 8) * 2.0 ** -23


def glu(g, u, limit):
    if limit:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1 + torch.exp(-g)) * u


def route(logits, bias, k, score="sigmoid", groups=1, top_groups=1, best=2, renorm=True, scale=1.0):
    """ids [T, k] and weights [T, k] of logits [T, E]; every row in Python's 64-bit floats."""
    T, E = logits.shape
    rows = logits.double().cpu().tolist()
    b = None if bias is None else bias.double().cpu().tolist()
    ids, weights = [], []
    for z in rows:
        nan = any(math.isnan(x) or (score == "softmax" and x == math.inf) for x in z)
        live = [e for e in range(E) if not math.isnan(z[e]) and z[e] != -math.inf]
        s = {}
        if score == "softmax" and live:
            top = max(z[e] for e in live)
            part = {e: math.exp(z[e] - top) if top < math.inf else math.nan for e in live}
            total = math.fsum(part.values())
            s = {e: v / total for e, v in part.items()}
        else:
            s = {e: 1 / (1 + math.exp(-z[e])) if z[e] > -700 else 0.0 for e in live}
        c = {e: z[e] if b is None else s[e] + b[e] for e in live}
        if top_groups < groups:
            size, rank = E // groups, []
            of = s if b is None and best == 2 else c
            for g in range(groups):
                inside = sorted((of[e] for e in live if e // size == g), reverse=True)[:best]
                if inside:
                    rank.append((-sum(inside), g))
            kept = {g for _, g in sorted(rank)[:top_groups]}
            live = [e for e in live if e // size in kept]
        chosen = sorted(live, key=lambda e: (-c[e], e))[:k]
        w = [s[e] for e in chosen]
        if renorm:
            total = math.fsum(w) + 1e-20
            w = [x / total for x in w]
        more = k - len(chosen)
        ids.append(chosen + [-1] * more)
        weights.append([math.nan] * k if nan else [x * scale for x in w] + [0.0] * more)
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64)


def lists(ids, E):
    """offsets [E + 1] and pairs (in the lists' order) of ids [T, k]."""
    flat = ids.flatten().tolist()
    by = [[p for p, e in enumerate(flat) if e == x] for x in range(E)]
    offsets = [0]
    for x in by:
        offsets.append(offsets[-1] + len(x))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(sum(by, []), dtype=torch.int32)
