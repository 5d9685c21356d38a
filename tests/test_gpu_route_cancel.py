"""moe_route with groups whose two largest keys nearly cancel, so that their sum is small beside what
fp32 keys are off.  Against ffnref.route in float64."""
import numpy as np
import pytest

from gpuutil import say, to_dev
from test_gpu_moe import check_route

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("E,groups,keep,topk", [(8, 2, 1, 2), (64, 8, 3, 6), (60, 4, 2, 8), (256, 8, 4, 8), (200, 8, 2, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_cancel(E, groups, keep, topk, score):
    """A group's two largest keys of either sign: its sum is small, but off by what its keys are."""
    rng = np.random.default_rng(E)
    per = E // groups
    x = to_dev((rng.standard_normal((1500, E)) * 2).astype(np.float32))
    for size in (2.0 ** 12, 2.0 ** 17, 2.0 ** 20, 1e30):
        say(f"moe_route biases of +-{size:g} E={E} groups={groups} {score}")
        bias = np.full(E, -2.0 * size)
        bias[::per], bias[1::per] = size, -size
        check_route(x, topk, bias, score=score, groups=groups, topk_groups=keep, renorm=False)
    # some groups so, some plain, some of masked experts alone
    bias = rng.standard_normal(E) * 0.2
    for g in range(groups):
        if g % 3 == 0:
            bias[g * per:(g + 1) * per] = -1e5
            bias[g * per], bias[g * per + 1] = 4096.0, -4096.0 + 0.75
        elif g % 3 == 1 and g > 1:
            bias[g * per:(g + 1) * per] = -1e9
    check_route(x, topk, bias, score=score, groups=groups, topk_groups=keep)
    # infinite and of the largest finite size: sums that fp32 does not hold
    bias[0], bias[1], bias[per], bias[per + 1] = INF, -1.0, 3e38, 3e38
    check_route(x, topk, bias, score=score, groups=groups, topk_groups=keep)
    bias[0], bias[1] = 3e38, -3e38
    check_route(x, topk, bias, score=score, groups=groups, topk_groups=keep)
