"""The attention sub-layer's operators from their definitions in 64 bits
(tests only): plain torch, no code of the CUDA path."""
import math

import torch


def pow2(e):
    """2^e of a tensor of whole numbers, exactly (exp2 and ldexp on the GPU go through pow, which is not)."""
    return torch.tensor([2.0 ** i for i in range(-1022, 1024)], dtype=torch.float64, device=e.device)[e.long() + 1022]


def e4m3_values():
    """The value of each of the 256 e4m3 codes (127 and 255 NaN)."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        x = math.nan if (c & 127) == 127 else x
        v.append(-x if c >= 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def scale_byte(amax: float) -> int:
    """The e8m0 byte of a block: the smallest 2^e >= amax / 448, e >= -126; 255 where a value is not finite."""
    if not math.isfinite(amax):
        return 255
    if amax == 0:
        return 1
    m, e = math.frexp(amax / 448)
    return max(1, (e - 1 if m == 0.5 else e) + 127)


def scale_bytes(amax):
    return torch.tensor([scale_byte(a) for a in amax.flatten().tolist()], dtype=torch.int64).view(amax.shape)


def e4m3_step(y):
    """The spacing of e4m3 values at |y| (64-bit tensor)."""
    _, e = torch.frexp(y.abs())
    return pow2((e - 1).clamp(min=-6) - 3)


def e4m3_round(y):
    s = e4m3_step(y)
    return torch.round(y / s) * s


def dequant(codes, scales):
    """codes [pages, heads, tokens, dim] u8, scales [pages, heads] u8 -> 64 bits."""
    return e4m3_values().to(codes.device)[codes.long()] * pow2(scales.int() - 127)[..., None, None]


def rotate(x, table, pos, dim, interleaved):
    """x [rows, heads, D] in 64 bits at positions pos, table [positions, dim / 2, 2]."""
    if not dim:
        return x
    c, s = (table.double()[pos][:, None, :, i] for i in (0, 1))
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:dim:2], x[..., 1:dim:2]
        y[..., 0:dim:2], y[..., 1:dim:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., : dim // 2], x[..., dim // 2: dim]
        y[..., : dim // 2], y[..., dim // 2: dim] = a * c - b * s, b * c + a * s
    return y


def attention(q, k, v, positions, scale, window):
    """q [n, H, D], k, v [L, KH, D] in 64 bits -> out, lse, and what the bounds need: sum p |v|, the largest sum |q k|, max |v|."""
    n, H, D = q.shape
    L, KH = k.shape[0], k.shape[1]
    j = torch.arange(L, device=q.device)
    seen = j[None] <= positions[:, None]
    if window:
        seen &= j[None] > positions[:, None] - window
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    reach, big = torch.zeros(n, H, dtype=torch.float64, device=q.device), torch.zeros(n, H, dtype=torch.float64, device=q.device)
    some = seen.any(1)
    for h in range(H):
        kk, vv = k[:, h // (H // KH)], v[:, h // (H // KH)]
        z = (q[:, h] @ kk.T * scale).masked_fill(~seen, -math.inf)
        p = torch.softmax(z, 1)
        p = torch.where(seen, p, torch.zeros_like(p))
        p[~some] = 0
        lse[some, h] = torch.logsumexp(z[some], 1)
        out[:, h] = p @ vv
        mass[:, h] = p @ vv.abs()
        if L:
            reach[:, h] = ((q[:, h].abs() @ kk.abs().T) * abs(scale)).masked_fill(~seen, 0).amax(1)
            big[:, h] = torch.where(seen, vv.abs().amax(1)[None], torch.zeros_like(z)).amax(1)
    return out, lse, mass, reach, big
