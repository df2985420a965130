"""engram_project_fp8 and engram_glu_fp8 against their definitions in 64 bits.

Bounds, from the arithmetic: a product of codes is exact; a sum of K of them is
within experts_ref.sum_error(K) of the sum of their sizes, and an output within
half a step of its type more.  The gated value a = g / (1 + e^-g) u moves by at
most 1.1 |u| dg + |g s(g)| du with the errors of g and u (|d/dg g s(g)| < 1.1) and by
2^-20 of itself (exp to 2 ulp, a sum, a quotient and a product); its codes are then within half a step.
"""
import math

import pytest
import torch

import experts_ref as X
from experts_glue import HALF, TYPES, E, blocks, check_codes, codes, fmt, random_lists, rng, scales  # noqa: F401

pytestmark = pytest.mark.gpu


def _rows(g, rows, K, kind, stride=0):
    x = codes(g, rows, stride or K)[:, :K]
    return x, scales(g, kind, rows, blocks(K))


def _weight(E, g, mats, N, K, kind, gated=False):
    w, s = codes(g, mats, N, K), scales(g, kind, mats, blocks(N), blocks(K))
    n = mats // 2 if gated else mats
    return w, s, E.Fp8Weight(w, s, fmt(E, kind), n, N, K, gated)


def _near(got, want, mass, K, out):
    rel, least = HALF[out]
    bound = X.sum_error(K) * mass
    ok = (got.double() - want).abs() <= bound + rel * (want.abs() + bound) + least
    assert ok.all(), (got.double() - want).abs().max()


def _project(E, x, xs, xfmt, weight, lists, out, rows, N, stride=0):
    dt, code = TYPES[out]
    full = torch.full((rows, stride or N), -7.0, dtype=dt, device="cuda")
    E.engram_project_fp8(x, x.stride(0) if rows > 1 else 0, xs, fmt(E, xfmt), rows, weight, lists, code, full, stride)
    assert E.engram_check() == 0
    assert (full[:, N:] == -7).all()
    return full[:, :N]


# rows, K, N: one row and a few, odd ones, tails of every kind, tiles of 32, 64 and 128 rows, K cut over clusters or not
DENSE = [(1, 16, 1), (1, 128, 128), (1, 4096, 256), (1, 1040, 129), (2, 48, 300), (3, 2064, 1000), (16, 512, 512),
         (17, 144, 257), (24, 4096, 640), (25, 256, 100), (33, 1536, 384), (56, 400, 500), (57, 128, 999), (64, 2048, 256),
         (65, 640, 384), (128, 4096, 128), (129, 272, 513), (300, 1024, 1280), (777, 320, 1000), (1025, 160, 2050),
         (2049, 64, 5000)]


@pytest.mark.parametrize("i,shape", list(enumerate(DENSE)))
def test_project_dense(E, i, shape):
    rows, K, N = shape
    xk, wk, out = ("e8m0", "fp8")[i % 2], ("e8m0", "fp8")[i // 2 % 2], ("f32", "bf16", "f16")[i % 3]
    g = rng(i)
    x, xs = _rows(g, rows, K, xk)
    w, ws, weight = _weight(E, g, 1, N, K, wk)
    y = _project(E, x, xs, xk, weight, None, out, rows, N)
    _near(y, *X.product(X.rows64(x, xs), X.weight64(w[0], ws[0])), K, out)


def test_project_is_exact_where_f32_is(E):
    """Small whole numbers: every partial sum is a whole number below 2^24."""
    for rows, K, N in [(1, 4096, 256), (40, 1024, 300), (200, 2048, 384)]:
        g = rng(rows)
        pick = torch.tensor([0x00, 0x38, 0x40, 0x44, 0xB8, 0xC0], dtype=torch.uint8, device="cuda")   # 0 1 2 3 -1 -2
        x, w = (pick[torch.randint(0, 6, s, generator=g, device="cuda")] for s in ((rows, K), (1, N, K)))
        xs = (127 + torch.randint(0, 3, (rows, blocks(K)), generator=g, device="cuda")).to(torch.uint8)
        ws = (127 + torch.randint(0, 2, (1, blocks(N), blocks(K)), generator=g, device="cuda")).to(torch.uint8)
        y = _project(E, x, xs, "e8m0", E.Fp8Weight(w, ws, fmt(E, "e8m0"), 1, N, K), None, "f32", rows, N)
        assert torch.equal(y.double(), X.rows64(x, xs) @ X.weight64(w[0], ws[0]).T)


def test_project_strides_and_scales_at_the_ends(E):
    rows, K, N = 37, 528, 200
    g = rng(5)
    x, xs = _rows(g, rows, K, "e8m0", stride=640)
    w, ws, weight = _weight(E, g, 1, N, K, "fp8")
    xs[3, 1], xs[4, 0] = 255, 1                             # a block that is NaN, one of the least scale
    y = _project(E, x, xs, "e8m0", weight, None, "f32", rows, N, stride=211)
    want, mass = X.product(X.rows64(x, xs), X.weight64(w[0], ws[0]))
    keep = torch.arange(rows, device="cuda") != 3
    assert torch.isnan(y[3]).all()
    _near(y[keep], want[keep], mass[keep], K, "f32")


def test_project_to_the_same_bits_every_time(E):
    g = rng(6)
    for rows, K, N in [(1, 4096, 512), (100, 4096, 384)]:    # cut over a cluster
        x, xs = _rows(g, rows, K, "fp8")
        _, _, weight = _weight(E, g, 1, N, K, "fp8")
        first = _project(E, x, xs, "fp8", weight, None, "f32", rows, N)
        for _ in range(5):
            assert torch.equal(first, _project(E, x, xs, "fp8", weight, None, "f32", rows, N))


# tokens, k, experts, K, N, skew: experts without rows, with one, with nearly all
EXPERTS = [(1, 1, 1, 64, 64, 0), (1, 8, 32, 2048, 512, 0), (3, 2, 300, 128, 80, 0), (16, 4, 8, 400, 272, 0),
           (64, 6, 64, 512, 256, 2.0), (130, 3, 5, 256, 144, 5.0), (200, 8, 16, 384, 640, 1.0), (513, 2, 7, 176, 400, 0),
           (40, 32, 40, 128, 128, 0), (900, 4, 1024, 64, 16, 0)]


@pytest.mark.parametrize("i,shape", list(enumerate(EXPERTS)))
def test_project_experts(E, i, shape):
    tokens, k, n, K, N, skew = shape
    xk, wk, out = ("e8m0", "fp8")[i % 2], ("fp8", "e8m0")[i // 2 % 2], ("bf16", "f32", "f16")[i % 3]
    g = rng(100 + i)
    ids, offsets, pairs, lists = random_lists(E, g, tokens, k, n, skew)
    x, xs = _rows(g, tokens * k, K, xk)
    w, ws, weight = _weight(E, g, n, N, K, wk)
    y = _project(E, x, xs, xk, weight, lists, out, tokens * k, N)
    x64 = X.rows64(x, xs)
    for e in range(n):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if mine.start < mine.stop:
            _near(y[pairs[mine].long()], *X.product(x64[mine], X.weight64(w[e], ws[e])), K, out)


FORMATS = [("e8m0", "e8m0"), ("e8m0", "fp8"), ("fp8", "e8m0"), ("fp8", "fp8")]
# enough rows for tiles of 128 rows and 256 weight rows: K of 1 to 33 blocks, whole and cut off, N with tails of both halves
MANY = [(2600, 1552, 2049, "bf16"), (65, 4096, 300, "f32"), (100, 1568, 1000, "bf16"), (777, 640, 515, "f16"), (128, 8192, 256, "bf16"), (300, 2064, 2100, "f32"), (1300, 1040, 2000, "bf16"), (700, 128, 7000, "f32"), (2500, 528, 1100, "f16"), (1153, 4112, 2177, "f32"), (9000, 16, 300, "bf16"),
        (640, 1664, 4097, "f16")]


@pytest.mark.parametrize("formats", FORMATS)
@pytest.mark.parametrize("i,shape", list(enumerate(MANY)))
def test_project_many_rows(E, i, shape, formats):
    rows, K, N, out = shape
    g = rng(400 + i)
    x, xs = _rows(g, rows, K, formats[0], stride=K + 16 * (i % 2))
    w, ws, weight = _weight(E, g, 1, N, K, formats[1])
    y = _project(E, x, xs, formats[0], weight, None, out, rows, N, stride=(0, N + 3, (N + 31) // 16 * 16)[i % 3])
    _near(y, *X.product(X.rows64(x, xs), X.weight64(w[0], ws[0])), K, out)


def test_many_rows_with_scales_at_the_ends(E):
    """NaN scales of rows and of weights, the least and large ones, powers of two for the tensor cores and in 32 bits alike."""
    rows, K, N = 1500, 640, 2000
    g = rng(21)
    x, xs = _rows(g, rows, K, "e8m0")
    w, ws, _ = _weight(E, g, 1, N, K, "e8m0")
    xs[3, 1], xs[4, 0], xs[5, 2], xs[1400, 4], xs[77] = 255, 1, 247, 255, 0
    ws[0, 2, 1], ws[0, 3, 4], ws[0, 5, 0] = 255, 0, 130
    nan_rows = torch.zeros(rows, dtype=torch.bool, device="cuda")
    nan_rows[[3, 1400]] = True
    nan_cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    nan_cols[256:384] = True
    want, mass = X.product(X.rows64(x, xs.clone()), X.weight64(w[0], ws[0]))
    f32 = [torch.where(s == 255, math.nan, X.scale_values(s)).float() for s in (xs, ws)]
    for xk, wk, a, b in (("e8m0", "e8m0", xs, ws), ("e8m0", "fp8", xs, f32[1]), ("fp8", "fp8", f32[0], f32[1])):
        y = _project(E, x, a, xk, E.Fp8Weight(w, b, fmt(E, wk), 1, N, K), None, "f32", rows, N)
        assert torch.equal(torch.isnan(y), nan_rows[:, None] | nan_cols[None])
        # row 5 reaches 2^120 2^3 448^2 128: beyond f32 where |want| >= 2^128, and anywhere on the way where the sizes' sum is
        ok = ~nan_rows[:, None] & ~nan_cols[None] & (mass < 2.0 ** 127)
        _near(y[ok], want[ok], mass[ok], K, "f32")
        beyond = ~nan_cols[None] & (want.abs().nan_to_num() >= 2.0 ** 128)
        assert not torch.isfinite(y[beyond]).any() and ok[~nan_rows][:, ~nan_cols].float().mean() > 0.99


MANY_EXPERTS = [(150, 1, 2, 2064, 272, 0), (200, 2, 3, 1040, 640, 1.0), (2000, 2, 7, 656, 1200, 1.0), (1500, 4, 9, 144, 2000, 0), (700, 3, 6, 1536, 1792, 3.0)]


@pytest.mark.parametrize("formats", FORMATS)
@pytest.mark.parametrize("i,shape", list(enumerate(MANY_EXPERTS)))
def test_many_rows_of_experts(E, i, shape, formats):
    tokens, k, n, K, N, skew = shape
    g = rng(500 + i)
    ids, offsets, pairs, lists = random_lists(E, g, tokens, k, n, skew)
    x, xs = _rows(g, tokens * k, K, formats[0])
    w, ws, weight = _weight(E, g, n, N, K, formats[1])
    y = _project(E, x, xs, formats[0], weight, lists, "f32", tokens * k, N)
    x64 = X.rows64(x, xs)
    for e in range(n):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if mine.start < mine.stop:
            _near(y[pairs[mine].long()], *X.product(x64[mine], X.weight64(w[e], ws[e])), K, "f32")


def _glu_want(x64, w, ws, e, limit):
    (g, mg), (u, mu) = (X.product(x64, X.weight64(w[2 * e + i], ws[2 * e + i])) for i in (0, 1))
    K = x64.shape[1]
    a = X.glu(g, u, limit)
    dg, du = X.sum_error(K) * mg, X.sum_error(K) * mu
    if limit:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    err = 1.1 * u.abs() * dg + (g * torch.sigmoid(g)).abs() * du + 1.1 * dg * du + 2.0 ** -20 * a.abs()
    return a, err


def _glu(E, x, xs, xk, weight, lists, limit, out, n_out, N):
    c = torch.full((n_out + 3, N), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((n_out + 3, blocks(N)), 9, dtype=torch.uint8 if out == "e8m0" else torch.float32, device="cuda")
    E.engram_glu_fp8(x, x.stride(0) if x.shape[0] > 1 else 0, xs, fmt(E, xk), x.shape[0], weight, lists, limit, fmt(E, out), c, s)
    assert E.engram_check() == 0
    return c, s


GLU_DENSE = [(1, 16, 16), (1, 4096, 128), (5, 400, 144), (31, 1040, 272), (48, 256, 400), (64, 2048, 128), (100, 144, 512),
             (257, 512, 160), (1000, 128, 640)]


@pytest.mark.parametrize("limit", [0.0, 0.75])
@pytest.mark.parametrize("i,shape", list(enumerate(GLU_DENSE)))
def test_glu_dense(E, i, shape, limit):
    rows, K, N = shape
    xk, wk, out = ("e8m0", "fp8")[i % 2], ("e8m0", "fp8")[i // 2 % 2], ("e8m0", "fp8")[(i + 1) % 2]
    g = rng(200 + i)
    x, xs = _rows(g, rows, K, xk)
    w, ws, weight = _weight(E, g, 2, N, K, wk, True)
    c, s = _glu(E, x, xs, xk, weight, None, limit, out, rows, N)
    check_codes(c[:rows], s[:rows], *_glu_want(X.rows64(x, xs), w, ws, 0, limit))
    assert (c[rows:] == 0x55).all() and (s[rows:] == 9).all()


@pytest.mark.parametrize("i,shape", list(enumerate(EXPERTS)))
def test_glu_experts(E, i, shape):
    tokens, k, n, K, N, skew = shape
    N = N // 16 * 16
    xk, wk, out = ("fp8", "e8m0")[i % 2], ("fp8", "e8m0")[i // 2 % 2], ("fp8", "e8m0")[i // 3 % 2]
    g = rng(300 + i)
    ids, offsets, pairs, lists = random_lists(E, g, tokens, k, n, skew)
    x, xs = _rows(g, tokens, K, xk)
    w, ws, weight = _weight(E, g, 2 * n, N, K, wk, True)
    total = tokens * k
    c, s = _glu(E, x, xs, xk, weight, lists, 0.0, out, total, N)
    x64 = X.rows64(x, xs)
    want, err = (torch.empty((total, N), dtype=torch.float64, device="cuda") for _ in "ab")
    for e in range(n):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if mine.start < mine.stop:
            want[mine], err[mine] = _glu_want(x64[pairs[mine].long() // k], w, ws, e, 0.0)
    check_codes(c[:total], s[:total], want, err)
    assert (c[total:] == 0x55).all()


@pytest.mark.parametrize("formats", FORMATS)
@pytest.mark.parametrize("i,shape", [(0, (1500, 272, 1200)), (1, (2600, 1296, 640)), (2, (700, 128, 2064)),
                                     (3, (70, 4096, 80)), (4, (333, 1088, 272)), (5, (128, 2048, 1040)), (6, (2600, 1040, 1040))])
def test_glu_many_rows(E, i, shape, formats):
    rows, K, N = shape
    g, out, limit = rng(600 + i), ("e8m0", "fp8")[i % 2], (0.0, 0.75)[i % 2]
    x, xs = _rows(g, rows, K, formats[0], stride=K + 32)
    w, ws, weight = _weight(E, g, 2, N, K, formats[1], True)
    c, s = _glu(E, x, xs, formats[0], weight, None, limit, out, rows, N)
    check_codes(c[:rows], s[:rows], *_glu_want(X.rows64(x, xs), w, ws, 0, limit))
    assert (c[rows:] == 0x55).all() and (s[rows:] == 9).all()


@pytest.mark.parametrize("formats", FORMATS)
@pytest.mark.parametrize("i,shape", list(enumerate(MANY_EXPERTS)))
def test_glu_many_rows_of_experts(E, i, shape, formats):
    tokens, k, n, K, N, skew = shape
    g = rng(700 + i)
    ids, offsets, pairs, lists = random_lists(E, g, tokens, k, n, skew)
    x, xs = _rows(g, tokens, K, formats[0], stride=K + 48)
    w, ws, weight = _weight(E, g, 2 * n, N, K, formats[1], True)
    total = tokens * k
    c, s = _glu(E, x, xs, formats[0], weight, lists, 0.0, ("fp8", "e8m0")[i % 2], total, N)
    x64 = X.rows64(x, xs)
    want, err = (torch.empty((total, N), dtype=torch.float64, device="cuda") for _ in "ab")
    for e in range(n):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if mine.start < mine.stop:
            want[mine], err[mine] = _glu_want(x64[pairs[mine].long() // k], w, ws, e, 0.0)
    check_codes(c[:total], s[:total], want, err)
    assert (c[total:] == 0x55).all()


@pytest.mark.parametrize("rows,formats", [(20, "fp8"), (2500, "fp8"), (2500, "e8m0")])
def test_glu_of_values_that_are_not_finite(E, rows, formats):
    K, N = 256, 640
    g = rng(9)
    x, xs = _rows(g, rows, K, "e8m0")
    w, ws, weight = _weight(E, g, 2, N, K, formats, True)
    xs[2] = 255                                              # a NaN row
    ws[1, 1] = math.inf if formats == "fp8" else 255         # infinite or NaN values in the second block of all rows
    c, s = _glu(E, x, xs, "e8m0", weight, None, 0.0, "e8m0", rows, N)
    assert (s[2] == 255).all() and (c[2] == 0).all()
    assert (s[:rows, 1] == 255).all() and (c[:rows, 128:256] == 0).all()
    keep = torch.arange(rows, device="cuda") != 2
    ws[1, 1] = 1 if formats == "fp8" else 127
    want, err = _glu_want(X.rows64(x, xs)[keep], w, ws, 0, 0.0)
    for b in (0, 2, 4):
        at = slice(128 * b, 128 * b + 128)
        check_codes(c[:rows][keep][:, at].contiguous(), s[:rows][keep][:, b: b + 1].contiguous(), want[:, at], err[:, at])


def test_rows_in_no_list_stay_as_they_were(E):
    """Masked choices: the lists end before tokens * k."""
    tokens, k, n, K, N = 30, 4, 6, 128, 96
    g = rng(11)
    ids, offsets, pairs, _ = random_lists(E, g, tokens, k, n)
    gone = int(offsets[4])                                   # experts 4 and 5 lose theirs
    offsets[5:] = gone
    pairs[gone:] = 1 << 20                                   # never read
    lists = E.ExpertLists(offsets, pairs, n, k, tokens)
    x, xs = _rows(g, tokens * k, K, "e8m0")
    w, ws, weight = _weight(E, g, n, N, K, "e8m0")
    y = _project(E, x, xs, "e8m0", weight, lists, "f32", tokens * k, N)
    listed = torch.zeros(tokens * k, dtype=torch.bool, device="cuda")
    listed[pairs[:gone].long()] = True
    assert (y[~listed] == -7).all() and not (y[listed] == -7).any()
    w2, ws2, gated = _weight(E, g, 2 * n, N, K, "e8m0", True)
    c, s = _glu(E, x[:tokens], xs[:tokens], "e8m0", gated, lists, 0.0, "e8m0", tokens * k, N)
    assert (c[gone:] == 0x55).all() and (s[gone:] == 9).all() and not (s[:gone] == 9).any()


def test_bad_lists_are_reported_and_read_as_absent(E):
    tokens, k, n, K, N = 16, 2, 4, 128, 64
    g = rng(12)
    ids, offsets, pairs, _ = random_lists(E, g, tokens, k, n)
    x, xs = _rows(g, tokens * k, K, "e8m0")
    w, ws, weight = _weight(E, g, n, N, K, "e8m0")
    out = torch.full((tokens * k, N), -7.0, device="cuda")

    def call(o, p):
        out.fill_(-7)
        E.engram_project_fp8(x, 0, xs, fmt(E, "e8m0"), tokens * k, weight, E.ExpertLists(o, p, n, k, tokens), 2, out, 0)
        return E.engram_check()

    assert call(offsets, pairs) == 0
    good = out.clone()
    bad = offsets.clone()
    bad[4] = tokens * k + 1                                  # the last expert leaves the lists
    assert call(bad, pairs) == -14
    have = torch.zeros(tokens * k, dtype=torch.bool, device="cuda")
    have[pairs[: int(offsets[3])].long()] = True
    assert torch.equal(out[have], good[have]) and (out[~have] == -7).all()
    wrong = pairs.clone()
    wrong[0] = -1
    assert call(offsets, wrong) == -8
    row = int(pairs[0])
    assert (out[row] == -7).all()
    out[row] = good[row]
    assert torch.equal(out, good)


def test_offsets_past_32_bits(E):
    """Weights of more than 2^32 bytes, and x rows more than 2^31 bytes apart."""
    n, N, K = 300, 4096, 4096
    g = rng(13)
    w = torch.full((n, N, K), 0x38, dtype=torch.uint8, device="cuda")
    w[n - 1] = codes(g, N, K)
    ws = scales(g, "e8m0", n, blocks(N), blocks(K))
    offsets = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    offsets[n] = 2
    pairs = torch.arange(2, dtype=torch.int32, device="cuda")
    stride = (1 << 31) + 4096
    x = torch.empty(stride + K, dtype=torch.uint8, device="cuda").as_strided((2, K), (stride, 1))
    x.copy_(codes(g, 2, K))
    xs = scales(g, "e8m0", 2, blocks(K))
    weight = E.Fp8Weight(w, ws, fmt(E, "e8m0"), n, N, K)
    y = _project(E, x, xs, "e8m0", weight, E.ExpertLists(offsets, pairs, n, 2, 1), "f32", 2, N)
    _near(y, *X.product(X.rows64(x, xs), X.weight64(w[n - 1], ws[n - 1])), K, "f32")
