"""moe_route where rows have fewer candidates than slots: id -1 and weight 0 in those, whatever the
others' weights are.  Against ffnref.route in float64."""
import numpy as np
import pytest

from gpuutil import say, to_dev
from test_gpu_moe import check_route

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("renorm", [True, False])
def test_empty_slots_of_rows_that_are_not_finite(renorm):
    """id -1 and weight 0, also where the others' weights are NaN."""
    x = np.full((8, 8), -INF, np.float32)
    x[0, :2] = INF, 0.0
    x[1, :3] = NAN, 1.0, 0.0
    x[2, 5] = INF
    x[3, 5:] = 1.0, INF, NAN
    x[4, :4] = 0.0, 1.0, 2.0, 3.0
    x[5] = NAN
    x[6, :2] = -200.0, -1e30     # finite, but zero beside nothing and as sigmoids
    for topk in (3, 5, 8):
        for groups in (1, 4):
            say(f"moe_route empty slots topk={topk} groups={groups} renorm={renorm}")
            check_route(to_dev(x), topk, groups=groups, topk_groups=groups, renorm=renorm, scale=2.0)
            check_route(to_dev(x), topk, score="sigmoid", groups=groups, topk_groups=groups, renorm=renorm)
            check_route(to_dev(x), topk, np.linspace(0.5, 0.1, 8), groups=groups, topk_groups=groups, renorm=renorm)
    wide = np.full((3, 300), -INF, np.float32)      # more slots than sixteen lanes hold
    wide[0, 250:270], wide[1, :9], wide[2, 7] = 1.0, INF, NAN
    wide[0, 255] = INF
    check_route(to_dev(wide), 33, renorm=renorm)
