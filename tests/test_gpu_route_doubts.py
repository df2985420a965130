"""engram_route where 32-bit scores mislead: choices are those of 64-bit scores all the same."""
import math

import pytest
import torch

import experts_ref as X
from experts_glue import E, TYPES, rng  # noqa: F401
from test_gpu_route import _check, _route

pytestmark = pytest.mark.gpu

ROWS, TIMES = 154, 64                                       # together enough for four tokens a warp


@pytest.mark.parametrize("n", [64, 128, 256])
@pytest.mark.parametrize("border", [1.0, 2.0, 4.0])
def test_two_negative_scores_on_both_sides_of_a_power_of_two(E, n, border):
    """Scores with a bias within 1.5e-7 (of their size) of -1, -2, -4: the unit of the smaller is twice the larger's.  Others are masked."""
    g = rng(int(border) + n)
    bias = -border - 0.1 - 0.8 * torch.rand(n, generator=g, device="cuda")
    pair = torch.rand((16 * ROWS, n), generator=g, device="cuda").argsort(1)[:, :2]
    off = border * 3e-7 * (torch.rand((16 * ROWS, 2), generator=g, device="cuda", dtype=torch.float64) - 0.5)
    s = -border + off - bias.double()[pair]
    logits = torch.full((16 * ROWS, n), -math.inf, device="cuda").scatter(1, pair, torch.log(s / (1 - s)).float())
    if n == 256 and border == 1:
        logits[0] = -math.inf
        bias[0], bias[1] = -1.83829141, -1.79599667          # 64 bits: -0.999999945 and -1.000000020; 32: the other way
        logits[1:][:, :2] = -math.inf
        logits[0, 0], logits[0, 1] = 1.64557028, 1.36145854
    for k in (1, 2):
        _check(E, logits, bias, k, times=TIMES // 16)


def _rows(T, n, k, tied, third, at, seed):
    """k - 1 clear choices, two equal logits for the last choice and the one behind it, a larger one that 32 bits (nearly) cannot tell from
    them at a higher index; the rest masked."""
    g = rng(seed)
    logits = torch.full((T, n), -math.inf, device="cuda")
    bias = torch.zeros(n, device="cuda")
    clear = torch.arange(k - 1, device="cuda") * 2 % (n - 3) if k > 1 else torch.empty(0, dtype=torch.long, device="cuda")
    bias[clear] = 1.0
    logits[:, clear] = 0.25 * torch.arange(k - 1, device="cuda") - 0.5
    free = torch.tensor([e for e in range(n) if e not in clear.tolist()], device="cuda")
    if at == "lane":                                         # neighbours
        first = torch.randint(0, len(free) - 2, (T, 1), generator=g, device="cuda")
        pick = free[first + torch.arange(3, device="cuda")]
    else:
        pick = free[torch.rand((T, len(free)), generator=g, device="cuda").argsort(1)[:, :3].sort(1).values]
    return logits.scatter(1, pick, torch.tensor([tied, tied, third], device="cuda").expand(T, 3)), bias


@pytest.mark.parametrize("T,times", [(1, 1), (20, 1), (300, 1), (ROWS, TIMES)])
@pytest.mark.parametrize("n", [40, 64, 256, 512])
def test_equal_numbers_behind_the_last_choice_and_a_larger_one_behind_those(E, n, T, times):
    two = 2.0 + 2.0 ** -22                                   # the next float
    for i, (tied, third) in enumerate(((30.0, 31.0), (-100.0, -99.0), (2.0, two), (20.0, 25.0))):
        for k in (1, 8):
            for at in ("lane", "anywhere"):
                logits, bias = _rows(T, n, k, tied, third, at, 10 * i + k)
                if tied > -80:
                    _check(E, logits, bias, k, times=times)
                    continue
                # e^-99 is under 2^-126, and a score under that may be 0 as a 32-bit number: over a sum of at least 1e-20 that moves
                # its weight by 2^-126 / 1e-20
                ids, w, offsets, pairs = _route(E, logits.repeat(times, 1), bias, k)
                want_ids, want = (x.repeat(times, 1) for x in X.route(logits, bias, k))
                assert torch.equal(ids.cpu(), want_ids)
                assert ((w.double().cpu() - want).abs() <= 2.0 ** -20 * want + 2.0 ** -126 / 1e-20).all()
                assert all(torch.equal(x.cpu(), y) for x, y in zip((offsets, pairs), X.lists(want_ids, n)))
    logits, bias = _rows(T, n, 8, 2.0, two, "anywhere", 99)
    _check(E, logits, bias, 8, times=times, score="softmax")


def test_equal_numbers_alone(E):
    """Rows whose scores are all equal, or equal but for a few, of every kernel: the lower index, and no third to be found."""
    for T, times in ((20, 1), (300, 1), (ROWS, TIMES)):
        logits = torch.zeros((T, 256), device="cuda")
        logits[1::3, 200] = 1.0
        logits[2::3, 100:103] = -1.0
        for dt in ("f32", "bf16"):
            _check(E, logits.to(TYPES[dt][0]), torch.full((256,), 0.5, device="cuda"), 8, times=times)
            _check(E, logits.to(TYPES[dt][0]), torch.full((256,), 0.5, device="cuda"), 4, times=times, groups=8, top_groups=4)


@pytest.mark.parametrize("T", [1, 100])
def test_a_softmax_whose_sum_loses_its_small_terms(E, T):
    """1024 experts, one of e^0 and the others each too small for the sum where they come to it (36 x 2^-24 in all): the 32-bit score of the
    first is 2.1e-6 too large, and a rival by its bias lies between."""
    t = 2.0 ** -24 * 0.999
    logits = torch.empty((32, 32), dtype=torch.float64)
    logits[0] = math.log(t)
    lane = torch.arange(32)
    for mine in (lane == 16, lane % 16 == 8, lane % 8 == 4, lane % 4 == 2, lane % 2 == 1):
        logits[mine] = math.log(t / 32 / int(mine.sum()))
    logits[0, 0] = 0
    rows = logits.flatten().float().cuda().expand(T, 1024).contiguous()
    for rival in (5, 700):
        for step in range(12):
            bias = torch.full((1024,), -1.0, device="cuda")
            bias[0] = -0.5
            bias[rival] = torch.tensor(0.49999775).view(torch.int32).add(step).view(torch.float32)
            _check(E, rows, bias, 2, score="softmax")
