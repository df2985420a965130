"""Lists whose offsets do not rise: experts that begin before the end of one before them count as absent too, and no other
expert's rows, nor a wait, suffer from it."""
import time

import pytest
import torch

import experts_ref as X
from experts_glue import E, blocks, check_codes, fmt, rng  # noqa: F401
from test_gpu_products import _glu_want, _near, _rows, _weight

pytestmark = pytest.mark.gpu


def _alternating(n, experts):
    return [0, n] * ((experts + 1) // 2) + [0] * ((experts + 1) % 2)


# pairs, offsets, experts that count; K, N such that a cluster shares a tile (but the last two: more tiles than SMs)
CASES = [(1, _alternating(1, 4), [0], 4096, 256), (20, _alternating(20, 8), [0], 2048, 272), (20, [0, 7, 3, 12, 20], [0, 3], 1024, 400),
         (300, _alternating(300, 7), [0], 1024, 256), (300, [0, 120, 40, 200, 300], [0, 3], 1536, 128), (300, [0, 50, 309, 80, 300], [0, 3], 1024, 256),
         (300, [0, -3, 100, 300], [2], 2048, 256), (300, [0, 200, 100, 150, 120, 150, 150, 300], [0], 1024, 256),
         (300, [0, 200, 100, 150, 120, 250, 250, 300], [0, 6], 1024, 256),
         (24, _alternating(24, 200), [0], 256, 1040), (2000, _alternating(2000, 9), [0], 128, 2560)]


@pytest.mark.parametrize("formats", [("e8m0", "e8m0"), ("e8m0", "fp8")])
@pytest.mark.parametrize("i,case", list(enumerate(CASES)))
def test_experts_that_begin_before_the_end_of_another(E, i, case, formats):
    n, offsets, live, K, N = case
    experts, g = len(offsets) - 1, rng(i)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    pairs = torch.randperm(n, generator=g, device="cuda").int()
    lists = E.ExpertLists(off, pairs, experts, 1, n)
    x, xs = _rows(g, n, K, formats[0])
    w, ws, weight = _weight(E, g, experts, N, K, formats[1])
    w2, ws2, gated = _weight(E, g, 2 * experts, N, K, formats[1], True)
    out = torch.full((n, N), -7.0, device="cuda")
    c = torch.full((n, N), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((n, blocks(N)), 9, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    began = time.monotonic()
    E.engram_project_fp8(x, 0, xs, fmt(E, formats[0]), n, weight, lists, 2, out, 0)
    assert E.engram_check() == -14                            # ENGRAM_E_LENGTH
    E.engram_glu_fp8(x, 0, xs, fmt(E, formats[0]), n, gated, lists, 0.0, fmt(E, "e8m0"), c, s)
    assert E.engram_check() == -14
    assert time.monotonic() - began < 1                       # a wait that runs out takes two seconds
    x64, there = X.rows64(x, xs), torch.zeros(n, dtype=torch.bool, device="cuda")
    for e in live:
        mine = slice(offsets[e], offsets[e + 1])
        there[mine] = True
        _near(out[pairs[mine].long()], *X.product(x64[mine], X.weight64(w[e], ws[e])), K, "f32")
        check_codes(c[mine], s[mine], *_glu_want(x64[pairs[mine].long()], w2, ws2, e, 0.0))
    assert (out[pairs[~there].long()] == -7).all() and (c[~there] == 0x55).all() and (s[~there] == 9).all()
