"""engram_route against its definition in 64 bits: ids and lists are equal, and
weights within 2^-20 of themselves (exp to 2 ulp, a sum of at most 1024 terms in a tree and 32 in
turn for softmax, quotients and products: under 12 x 2^-24) and, for softmax, 2^-24
(l - max) more (the difference's rounding)."""
import math

import pytest
import torch

import experts_ref as X
from experts_glue import TYPES, E, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def _route(E, logits, bias, k, score="sigmoid", groups=1, top_groups=1, best=2, renorm=True, scale=1.0, lists=True, stream=None):
    T, n = logits.shape
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[logits.dtype]
    r = E.Router(n, k, E.ENGRAM_SCORE_SIGMOID if score == "sigmoid" else E.ENGRAM_SCORE_SOFTMAX, groups, top_groups, best, renorm, scale)
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -9.0, device="cuda")
    offsets = torch.full((n + 1,), -9, dtype=torch.int32, device="cuda")
    pairs = torch.full((T * k,), -9, dtype=torch.int32, device="cuda")
    L = E.ExpertLists(offsets, pairs, n, k, T) if lists else None
    need = E.engram_route_workspace_bytes(n, T)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    E.engram_route(r, code, logits, logits.stride(0) if T > 1 else 0, bias, T, ids, w, L, ws, need, stream=stream)
    assert E.engram_check() == 0
    assert (ws[need:] == 0xAB).all()
    return ids, w, offsets, pairs


def _check(E, logits, bias, k, lists=True, times=1, **spec):
    ids, w, offsets, pairs = _route(E, logits.repeat(times, 1) if times > 1 else logits, bias, k, lists=lists, **spec)
    want_ids, want_w = (x.repeat(times, 1) for x in X.route(logits, bias, k, **spec))
    assert torch.equal(ids.cpu(), want_ids)
    got = w.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want_w))
    finite = ~torch.isnan(want_w)
    off = (got - want_w)[finite].abs()
    assert (off <= (2.0 ** -20 + (2.0 ** -18 if spec.get("score") == "softmax" else 0)) * want_w[finite].abs() + 1e-30).all(), off.max()
    if lists:
        o, p = X.lists(want_ids, logits.shape[1])
        assert torch.equal(offsets.cpu(), o) and torch.equal(pairs[: len(p)].cpu(), p)
        assert (pairs[len(p):] == -9).all()


# tokens, experts, k, type, score, bias, groups, top_groups, best, renorm
CASES = [(1, 1, 1, "f32", "sigmoid", False, 1, 1, 2, True), (1, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True),
         (3, 7, 7, "f16", "softmax", True, 1, 1, 1, False), (64, 33, 5, "bf16", "sigmoid", False, 3, 2, 2, True),
         (65, 64, 6, "f32", "softmax", False, 1, 1, 2, True), (200, 160, 6, "bf16", "softmax", False, 8, 3, 1, False),
         (77, 96, 32, "f32", "sigmoid", True, 3, 3, 2, True), (300, 100, 4, "f16", "sigmoid", True, 4, 1, 2, False),
         (129, 300, 12, "f32", "softmax", True, 4, 2, 2, True), (50, 1024, 8, "bf16", "sigmoid", True, 32, 5, 2, True),
         (41, 512, 3, "f32", "sigmoid", False, 16, 7, 2, True), (500, 40, 2, "bf16", "sigmoid", True, 20, 3, 2, True),
         (33, 32, 1, "f32", "softmax", False, 32, 1, 2, True), (1000, 256, 8, "bf16", "sigmoid", False, 8, 4, 2, True),
         (2500, 128, 4, "f32", "sigmoid", True, 4, 2, 1, True), (70, 1000, 16, "f32", "softmax", True, 1, 1, 2, True)]


@pytest.mark.parametrize("i,case", list(enumerate(CASES)))
def test_route(E, i, case):
    T, n, k, dt, score, bias, groups, top_groups, best, renorm = case
    g = rng(i)
    logits = (2 * torch.randn((T, n), generator=g, device="cuda")).to(TYPES[dt][0])
    b = 0.2 * torch.randn(n, generator=g, device="cuda") if bias else None
    _check(E, logits, b, k, score=score, groups=groups, top_groups=top_groups, best=best, renorm=renorm, scale=1.75)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_equal_scores_go_to_the_lower_index(E, score, bias):
    """Few different values, and zeros of both signs: nearly every choice is among equals."""
    g = rng(1)
    logits = torch.randint(-1, 2, (150, 72), generator=g, device="cuda").float() * 0.5
    logits[::2][logits[::2] == 0] = -0.0
    b = torch.randint(0, 2, (72,), generator=g, device="cuda").float() * 0.25 if bias else None
    for groups, top in ((1, 1), (6, 2)):
        _check(E, logits, b, 9, score=score, groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_scores_nearer_than_32_bits_tell(E, score):
    """Logits an ulp apart, where the scores' differences are far under an f32 ulp: the order is that of 64 bits."""
    T, n = 80, 96
    g = rng(2)
    base = torch.rand((T, 1), generator=g, device="cuda") * 4 + 2
    step = torch.randint(0, 40, (T, n), generator=g, device="cuda")
    logits = (base.view(torch.int32) + step.int()).view(torch.float32)
    assert ((1 / (1 + torch.exp(-logits))).sort(1).values.diff(dim=1) == 0).float().mean() > 0.5    # f32 cannot tell
    for bias in (torch.zeros(n, device="cuda"), torch.full((n,), 0.5, device="cuda")):
        _check(E, logits, bias, 8, score=score)
        _check(E, logits, bias, 8, score=score, groups=8, top_groups=3)
    _check(E, logits, None, 8, score=score, groups=8, top_groups=3)
    _check(E, logits, None, 8, score=score)


def _near(T, n, seed):
    g = rng(seed)
    base = torch.rand((T, 1), generator=g, device="cuda") * 4 + 2
    return (base.view(torch.int32) + torch.randint(0, 40, (T, n), generator=g, device="cuda").int()).view(torch.float32)


@pytest.mark.parametrize("T,n,k", [(9, 8, 8), (70, 8, 8), (50, 40, 9), (90, 64, 6), (90, 256, 8)])
def test_near_scores_with_none_behind_the_last(E, T, n, k):
    """As many experts as choices, or that many that are not masked: no score bounds the last choice from below."""
    logits = _near(T, n, n)
    if n > k:
        keep = torch.rand((T, n), generator=rng(n + 1), device="cuda").argsort(1)[:, :k]
        logits = torch.full_like(logits, -math.inf).scatter(1, keep, logits.gather(1, keep))
    for score in ("sigmoid", "softmax"):
        _check(E, logits, torch.full((n,), 0.25, device="cuda"), k, score=score)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,groups", [(64, 1), (64, 8), (128, 4), (256, 1), (256, 2), (256, 8)])
def test_four_tokens_a_warp(E, n, groups, dt):
    """8, 16 and 32 experts a lane: random rows, near and equal scores, masked and non-finite ones, an odd number of
    tokens, 62 times."""
    T, g = 159, rng(n + groups)
    logits = 2 * torch.randn((T, n), generator=g, device="cuda")
    logits[40:80] = _near(40, n, 5)
    logits[80:100] = torch.randint(-1, 2, (20, n), generator=g, device="cuda").float() * 0.5
    logits[100:120][torch.rand((20, n), generator=g, device="cuda") < 0.9] = -math.inf
    logits[120] = -math.inf
    logits[121, 5], logits[122, 9], logits[123, 3] = math.nan, math.inf, -3e4
    logits[124, : n // 2] = -math.inf
    logits = logits.to(TYPES[dt][0])
    biases = [0.2 * torch.randn(n, generator=g, device="cuda"), torch.randint(0, 2, (n,), generator=g, device="cuda") * 0.25]
    for k, b in ((8, biases[0]), (3, biases[1]), (8, torch.zeros(n, device="cuda")), (6, None)):
        for best in (1, 2):
            _check(E, logits, b, k, times=62, groups=groups, top_groups=max(1, groups // 2), best=best, renorm=k != 3)


@pytest.mark.parametrize("n", [48, 256])
def test_group_sums_whose_parts_are_larger(E, n):
    """Biases of +-1000: a group's two largest nearly cancel, and the sums' 32-bit errors are those of the parts."""
    g = rng(n)
    logits = 2 * torch.randn((90, n), generator=g, device="cuda")
    size = n // 8
    bias = torch.full((n,), -1000.0, device="cuda")
    bias[::size] = 1000.0
    for T, times in ((20, 1), (89, 1), (89, 111)):
        _check(E, logits[:T], bias, 2, times=times, groups=8, top_groups=3)


def test_masked_experts_and_rows(E):
    """-inf: never chosen; rows with fewer experts than choices, and with none, are padded with -1 and weight 0."""
    g = rng(3)
    for score in ("sigmoid", "softmax"):
        for bias in (None, 0.1 * torch.randn(48, generator=g, device="cuda")):
            for groups, top in ((1, 1), (6, 2)):
                logits = torch.randn((100, 48), generator=g, device="cuda")
                logits[torch.rand((100, 48), generator=g, device="cuda") < 0.6] = -math.inf
                logits[3, 5:] = -math.inf
                logits[7] = -math.inf
                logits[90:] = -math.inf
                logits[11, :40] = -math.inf
                for renorm in (True, False):
                    _check(E, logits, bias, 6, score=score, groups=groups, top_groups=top, renorm=renorm)


def test_values_that_are_not_finite(E):
    logits = torch.randn((6, 40), generator=rng(4), device="cuda")
    logits[1, 7] = math.nan
    logits[2, :] = math.nan
    logits[3, 9] = math.inf
    logits[4, 2] = 3e38
    logits[5, 3] = -3e38
    _check(E, logits, None, 5)
    _check(E, logits, torch.zeros(40, device="cuda"), 5)
    keep = [0, 1, 2, 4, 5]
    _check(E, logits[keep].contiguous(), None, 5, score="softmax")
    assert torch.isnan(_route(E, logits, None, 5, score="softmax")[1][3]).all()


def test_strides_and_calls_without_lists(E):
    logits = torch.randn((90, 77), generator=rng(5), device="cuda")[:, 3:61]
    for T in (1, 20, 90):
        _check(E, logits[:T], None, 4, lists=False)
        _check(E, logits[:T], None, 4)


def test_no_tokens_leave_empty_lists(E):
    offsets = torch.full((9,), -9, dtype=torch.int32, device="cuda")
    E.engram_route(E.Router(8, 2), 2, None, 0, None, 0, None, None, E.ExpertLists(offsets, None, 8, 2, 0))
    assert E.engram_check() == 0
    assert (offsets == 0).all()


def test_lists_of_many_tokens(E):
    """Against torch's stable sort: more tokens than the Python reference takes."""
    for T, n, k in ((16384, 256, 8), (5000, 1024, 3), (40001, 64, 6)):
        logits = torch.randn((T, n), generator=rng(T), device="cuda")
        ids, w, offsets, pairs = _route(E, logits, None, k)
        assert torch.equal(ids, torch.topk(logits, k).indices.int())      # f32 normal logits: no ties here to speak of
        flat = ids.flatten()
        assert torch.equal(pairs, torch.sort(flat, stable=True).indices.int())
        counts = torch.bincount(flat, minlength=n)
        assert offsets[0] == 0 and torch.equal(offsets[1:], counts.cumsum(0).int())
