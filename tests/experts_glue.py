"""Inputs and calls for the experts' sub-layer's GPU tests."""
import pytest
import torch

import sublayer_ref as R

TYPES = {"bf16": (torch.bfloat16, 0), "f16": (torch.float16, 1), "f32": (torch.float32, 2)}
# half a step of a value's size, and half the least step near zero (f32: what the sums' bound has)
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25), "f32": (2.0 ** -24, 2.0 ** -149)}


@pytest.fixture(scope="module")
def E():
    import __graft_entry__
    __graft_entry__.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    assert torch.cuda.is_available()
    return _lib


def fmt(E, name):
    return {"fp8": E.ENGRAM_FMT_FP8, "e8m0": E.ENGRAM_FMT_FP8_E8M0}[name]


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape, spread=60.0):
    """Finite e4m3 codes of normal values."""
    x = torch.randn(shape, generator=g, device="cuda") * spread
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def scales(g, kind, *shape):
    """Scales around 2^-7, as bytes or as f32 that are no powers of two."""
    if kind == "e8m0":
        return (120 + torch.randint(-3, 4, shape, generator=g, device="cuda")).to(torch.uint8)
    return torch.exp(torch.randn(shape, generator=g, device="cuda")) * 2.0 ** -7


def blocks(n):
    return -(-n // 128)


def random_lists(E, g, tokens, k, n_experts, skew=0.0):
    """ids [tokens, k] and their lists on the GPU (through torch)."""
    z = torch.rand((tokens, n_experts), generator=g, device="cuda") + skew * torch.rand(n_experts, generator=g, device="cuda")
    ids = torch.topk(z, k).indices
    flat = ids.flatten()
    pairs = torch.sort(flat, stable=True).indices.int()
    counts = torch.bincount(flat, minlength=n_experts)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), counts.cumsum(0)]).int()
    return ids, offsets, pairs, E.ExpertLists(offsets, pairs, n_experts, k, tokens)


def check_codes(got, byte_or_f32, want, error):
    """Codes [rows, N] and scales [rows, blocks] against 64-bit values `want` that are known to `error` (absolute)."""
    n = want.shape[1]
    pad = -n % 128
    w = torch.nn.functional.pad(want, (0, pad)).view(want.shape[0], -1, 128)
    err = torch.nn.functional.pad(error, (0, pad)).view(w.shape)
    sc = torch.where(byte_or_f32 == 255, float("nan"), R.pow2(byte_or_f32.int() - 127)) if byte_or_f32.dtype == torch.uint8 \
        else byte_or_f32.double()
    finite = torch.isfinite(w).all(2)
    assert torch.equal(torch.isfinite(sc), finite)
    # the scale is the rule's for the largest value, or its neighbour's where that is within the error of a border
    lo, hi = ((w.abs() + s * err).amax(2).clamp(min=0) for s in (-1, 1))
    bytes_lo, bytes_hi = (R.scale_bytes(torch.where(finite, x, torch.zeros_like(x))).to(w.device) for x in (lo, hi))
    have = torch.log2(torch.where(finite, sc, torch.ones_like(sc))).round().long() + 127
    assert ((have >= bytes_lo) & (have <= bytes_hi) | ~finite).all()
    assert torch.equal(R.pow2(have - 127)[finite], sc[finite])
    y = R.e4m3_values().to(w.device)[torch.nn.functional.pad(got, (0, pad)).view(w.shape).long()]
    assert not torch.isnan(y).any()
    s = sc[..., None]
    off = (y * s - w).abs()
    limit = err + 0.5 * R.e4m3_step(torch.maximum(y.abs(), (w / s).abs().nan_to_num())) * s * (1 + 1e-6)
    assert (off <= limit)[finite].all()
    assert (y[~finite] == 0).all()
