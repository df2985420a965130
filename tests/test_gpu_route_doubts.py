"""engram_route where 32-bit scores mislead: choices are those of 64-bit scores all the same."""
import math

import pytest
import torch

from experts_glue import E, TYPES, rng  # noqa: F401
from test_gpu_route import _check

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
