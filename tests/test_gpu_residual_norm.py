"""engram_residual_norm against its definition in 64 bits.

Bounds, from the arithmetic: the residual is one f32 addition (and one rounding
to its type), so it is exact there.  y's relative error before its own rounding
is at most that of the sum of squares (under 32 sequential f32 additions a
thread and a tree above: 20 x 2^-24 after the root's halving), the root, the
reciprocal and two products: together under 40 x 2^-24 < 2.5e-6.  Codes are
then within half a step of y / scale, bf16 (8 significant bits) within 2^-8.
"""
import math

import pytest
import torch

import sublayer_ref as R

pytestmark = pytest.mark.gpu
Y_REL = 2.5e-6


@pytest.fixture(scope="module")
def E():
    import __graft_entry__
    __graft_entry__.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    assert torch.cuda.is_available()
    return _lib


TYPES = {"bf16": (torch.bfloat16, 0), "f16": (torch.float16, 1), "f32": (torch.float32, 2)}


def _fmt(E, fmt):
    return {"bf16": E.ENGRAM_FMT_BF16, "fp8": E.ENGRAM_FMT_FP8, "e8m0": E.ENGRAM_FMT_FP8_E8M0}[fmt]


def _call(E, x, res, w, fmt, block, eps=1e-6, in_place=False, write_res=True):
    rows, dim = res.shape
    y = torch.empty((rows, dim), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device="cuda")
    sc = None
    if fmt != "bf16":
        sc = torch.empty((rows, dim // block), dtype=torch.uint8 if fmt == "e8m0" else torch.float32, device="cuda")
    out = (res if in_place else torch.empty_strided(res.size(), res.stride(), dtype=res.dtype, device="cuda")) if write_res else None
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    E.engram_residual_norm(x, code[x.dtype] if x is not None else 0, res, code[res.dtype], out, w, rows, dim, eps,
                           _fmt(E, fmt), block, y, sc, x_stride=x.stride(0) if x is not None and rows > 1 else 0,
                           res_stride=res.stride(0) if rows > 1 else 0)
    assert E.engram_check() == 0
    return out, y, sc


def _check(x, res, w, fmt, block, out, y, sc, eps=1e-6):
    r32 = res.float() + (x.float() if x is not None else 0)
    if out is not None:
        assert torch.equal(out, r32.to(res.dtype))
    r = r32.double()
    want = r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * (w.double() if w is not None else 1)
    if fmt == "bf16":
        assert ((y.double() - want).abs() <= (2.0 ** -8 + Y_REL) * want.abs()).all()
        return
    rows, dim = want.shape
    want = want.view(rows, -1, block)
    byte = R.scale_bytes(want.abs().amax(2).cpu()).to(y.device)
    scale = R.pow2(byte - 127)
    assert torch.equal(sc.double() if fmt == "fp8" else sc.long(), scale if fmt == "fp8" else byte)
    got = R.e4m3_values().to(y.device)[y.long()].view(rows, -1, block) * scale[..., None]
    tol = 0.5 * R.e4m3_step(want / scale[..., None]) * scale[..., None] * (1 + 1e-9) + Y_REL * want.abs()
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("rows,dim,xt,rt,fmt,block", [
    (1, 4096, "bf16", "f32", "e8m0", 32),
    (3, 16, "f32", "f32", "fp8", 16),
    (5, 8, "bf16", "bf16", "bf16", 0),
    (2, 48, "f16", "f32", "e8m0", 48),            # block of 6 chunks: the shared-memory maxima
    (7, 1040, "f16", "bf16", "fp8", 80),
    (4, 2048, "bf16", "f32", "fp8", 512),         # a block wider than a warp
    (3, 4096, "f32", "bf16", "e8m0", 4096),       # one scale a row
    (129, 4096, "bf16", "f32", "bf16", 0),
    (33, 5120, "f16", "f32", "e8m0", 128),
    (9, 8200, "f32", "f32", "bf16", 0),
    (3, 16384, "f32", "f32", "fp8", 256),
    (2, 16384, "bf16", "bf16", "e8m0", 16),
    (1537, 1504, "bf16", "bf16", "e8m0", 16),
])
def test_matches_the_definition(E, rows, dim, xt, rt, fmt, block):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + dim)
    x = torch.randn(rows, dim, generator=g, device="cuda").to(TYPES[xt][0])
    res = (3 * torch.randn(rows, dim, generator=g, device="cuda")).to(TYPES[rt][0])
    w = 1 + 0.3 * torch.randn(dim, generator=g, device="cuda")
    out, y, sc = _call(E, x, res, w, fmt, block)
    _check(x, res, w, fmt, block, out, y, sc)


def test_without_x_weight_or_residual_output(E):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randn(6, 256, generator=g, device="cuda") for _ in range(2))
    w = torch.randn(256, generator=g, device="cuda")
    for xx, ww, wr in ((None, w, True), (x, None, True), (x, w, False), (None, None, False)):
        out, y, sc = _call(E, xx, res, ww, "e8m0", 32, write_res=wr)
        _check(xx, res, ww, "e8m0", 32, out, y, sc)


def test_in_place_equals_out_of_place(E):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, res = torch.randn(17, 4096, generator=g, device="cuda").bfloat16(), torch.randn(17, 4096, generator=g, device="cuda")
    a = _call(E, x, res.clone(), None, "fp8", 64)
    mine = res.clone()
    b = _call(E, x, mine, None, "fp8", 64, in_place=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and b[0] is mine


def test_strided_rows(E):
    """Rows that are slices of wider ones; what lies between them stays."""
    g = torch.Generator(device="cuda").manual_seed(3)
    xw = torch.randn(11, 300 * 8, generator=g, device="cuda").half()
    rw = torch.randn(11, 2 * 512, generator=g, device="cuda")
    x, res = xw[:, 64:64 + 512], rw[:, :512]
    keep = rw.clone()
    w = torch.randn(512, generator=g, device="cuda")
    before = res.clone()
    out, y, sc = _call(E, x, res, w, "e8m0", 32, in_place=True)
    _check(x, before, w, "e8m0", 32, out, y, sc)
    assert torch.equal(rw[:, 512:], keep[:, 512:])


@pytest.mark.parametrize("mag", [0.0, 1e-30, 1e-18, 1e15])
def test_magnitudes(E, mag):
    """Zero rows (scale 2^-126, zero codes), rows whose squares are tiny beside eps, and large ones."""
    g = torch.Generator(device="cuda").manual_seed(4)
    res = torch.randn(4, 512, generator=g, device="cuda") * mag
    out, y, sc = _call(E, None, res, None, "e8m0", 32)
    _check(None, res, None, "e8m0", 32, out, y, sc)
    if mag == 0.0:
        assert (sc == 1).all() and (y & 127 == 0).all()


def test_non_finite_rows_are_nan_and_alone(E):
    """A NaN anywhere makes its row NaN (NaN scales, zero codes); an infinity makes 0 elsewhere and NaN in its own block."""
    g = torch.Generator(device="cuda").manual_seed(5)
    res = torch.randn(4, 256, generator=g, device="cuda")
    clean = _call(E, None, res, None, "e8m0", 32)
    bad = res.clone()
    bad[1, 40] = math.nan
    bad[2, 70] = math.inf
    _, y, sc = _call(E, None, bad, None, "e8m0", 32)
    assert (sc[1] == 255).all() and (y[1] == 0).all()
    assert sc[2, 2] == 255 and (sc[2, [0, 1, 3, 4, 5, 6, 7]] == 1).all() and (y[2] & 127 == 0).all()
    for r in (0, 3):
        assert torch.equal(y[r], clean[1][r]) and torch.equal(sc[r], clean[2][r])
    _, y, sc = _call(E, None, bad, None, "fp8", 32)
    assert sc[1].isnan().all() and sc[2, 2].isnan()


def test_rows_read_by_the_table_gather(E):
    """The output is an engram table: engram_rows_fp8(_e8m0) turns it into bf16."""
    g = torch.Generator(device="cuda").manual_seed(6)
    rows, dim, block = 21, 256, 32
    res = torch.randn(rows, dim, generator=g, device="cuda")
    ids = torch.arange(rows, device="cuda", dtype=torch.int64)
    got = []
    for fmt, call in (("fp8", E.engram_rows_fp8), ("e8m0", E.engram_rows_fp8_e8m0)):
        _, y, sc = _call(E, None, res, None, fmt, block)
        x = torch.empty((rows, dim), dtype=torch.bfloat16, device="cuda")
        call(y, sc, rows, dim, block, ids, rows, 1, 1, x)
        got.append(x)
    assert E.engram_check() == 0
    want = res.double() / torch.sqrt(res.double().square().mean(1, keepdim=True) + 1e-6)
    assert torch.equal(got[0], got[1])
    assert ((got[0].double() - want).abs() <= want.abs() / 16 + 2.0 ** -10 * want.abs().amax(1, keepdim=True) / 448 * 2).all()


def test_zero_rows_and_another_stream(E):
    empty = torch.empty(0, 64, device="cuda")
    E.engram_residual_norm(None, 0, None, 2, None, None, 0, 64, 1e-6, E.ENGRAM_FMT_BF16, 0, None, None)
    s = torch.cuda.Stream()
    x = torch.ones(3, 64, device="cuda")
    torch.cuda.synchronize()
    y = torch.empty(3, 64, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(s):
        E.engram_residual_norm(None, 0, x, 2, None, None, 3, 64, 0.0, E.ENGRAM_FMT_BF16, 0, y, None)
    assert E.engram_check(s) == 0
    assert (y == 1).all() and empty.numel() == 0
