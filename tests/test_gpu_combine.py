"""engram_combine against its definition in 64 bits: k FMAs and one addition in f32 are within (k + 1) 2^-24 of the
sum of the terms' sizes, the output half a step of its type from that."""
import math

import pytest
import torch

from experts_glue import HALF, TYPES, E, rng  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, k, dim, y, add, out
CASES = [(1, 1, 8, "f32", None, "f32"), (1, 8, 4096, "bf16", "bf16", "bf16"), (3, 9, 264, "f16", None, "f32"),
         (130, 2, 1000, "f32", "f16", "bf16"), (64, 32, 72, "bf16", "f32", "f16"), (17, 16, 5120, "f16", "f16", "f16"),
         (1000, 8, 128, "bf16", None, "bf16")]


@pytest.mark.parametrize("wide", [0, 24])
@pytest.mark.parametrize("i,case", list(enumerate(CASES)))
def test_combine(E, i, case, wide):
    T, k, dim, yt, at, ot = case
    g = rng(i)
    y = torch.randn((T * k, dim + wide), generator=g, device="cuda").to(TYPES[yt][0])
    w = torch.rand((T, k), generator=g, device="cuda")
    w[torch.rand((T, k), generator=g, device="cuda") < 0.2] = 0
    y[(w == 0).flatten()] = math.nan                         # choices of weight 0 are not read
    add = torch.randn((T, dim + wide), generator=g, device="cuda").to(TYPES[at][0]) if at else None
    out = torch.full((T, dim + wide), -7.0, dtype=TYPES[ot][0], device="cuda")
    st = dim + wide if wide else 0
    E.engram_combine(y, TYPES[yt][1], st, w, T, k, dim, add, TYPES[at][1] if at else 0, st, TYPES[ot][1], out, st)
    assert E.engram_check() == 0
    assert (out[:, dim:] == -7).all()
    terms = torch.where(w[:, :, None] == 0, 0.0, y[:, :dim].double().view(T, k, dim) * w.double()[:, :, None])
    want, mass = terms.sum(1), terms.abs().sum(1)
    if at:
        want, mass = want + add[:, :dim].double(), mass + add[:, :dim].double().abs()
    rel, least = HALF[ot]
    bound = (k + 1) * 2.0 ** -24 * mass
    assert ((out[:, :dim].double() - want).abs() <= bound + rel * (want.abs() + bound) + least).all()


def test_in_place_on_what_is_added(E):
    g = rng(9)
    y, w = torch.randn((40, 64), generator=g, device="cuda"), torch.rand((10, 4), generator=g, device="cuda")
    add = torch.randn((10, 64), generator=g, device="cuda")
    out = torch.empty_like(add)
    E.engram_combine(y, 2, 0, w, 10, 4, 64, add, 2, 0, 2, out, 0)
    E.engram_combine(y, 2, 0, w, 10, 4, 64, add, 2, 0, 2, add, 0)
    assert torch.equal(out, add)
