"""moe_route with scores next to the least normal fp32 number, below which the hardware's exponential
and reciprocal give zero.  Against ffnref.route in float64."""
import numpy as np
import pytest
import torch

from gpuutil import device, say, to_dev
from test_gpu_moe import check_route, run_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
def test_one_flushed_score_of_two(renorm):
    """Sums of two sigmoids one of which lies below 2^-126 = 1.1755e-38 = e^-87.337."""
    x = np.array([[-87.30, -87.34, -200, -200, -87.25, -200, -200, -200],
                  [-87.2, -87.4, -200, -200, -86.9, -200, -200, -200],
                  [-86.9, -200, -200, -200, -87.2, -87.4, -200, -200],
                  [-87.34, -87.35, -87.33, -300, -86.7, -300, -300, -300]], np.float32)
    say(f"moe_route flushed scores renorm={renorm}")
    for topk in (1, 2):     # with two, equal zeros among the candidates
        check_route(to_dev(x), topk, score="sigmoid", groups=2, topk_groups=1, renorm=renorm)
    top = np.zeros((4, 12), np.float32)             # softmax: the third group holds the largest logit
    top[:, :8], top[:, 8], top[:, 9:] = x, 0.0, -200.0
    for topk in (2, 3):
        check_route(to_dev(top), topk, groups=3, topk_groups=2, renorm=renorm)


# E to a group: whole lanes, parts of lanes, and groups that no lane begins
@pytest.mark.parametrize("E,groups,keep,topk", [(8, 2, 1, 2), (64, 8, 3, 6), (60, 4, 2, 8), (256, 8, 4, 8), (200, 8, 2, 5),
                                                (512, 16, 3, 8), (1024, 64, 5, 20)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_scores_next_to_the_flush(E, groups, keep, topk, group_top):
    say(f"moe_route next to 2^-126 E={E} groups={groups} group_top={group_top}")
    rng = np.random.default_rng(E + group_top)
    x = rng.uniform(-87.6, -87.1, (400, E))
    x[100:200] = rng.uniform(-110.0, -60.0, (100, E))        # 2^-100 = e^-69.3 within
    x[200:300] = np.where(rng.random((100, E)) < 0.9, -150.0, x[200:300])
    x[300:] = rng.uniform(-87.3366, -87.3360, (100, E))      # steps of 2^-17
    check_route(to_dev(x.astype(np.float32)), topk, score="sigmoid", groups=groups, topk_groups=keep, group_top=group_top)
    x[:, 0] = 0.0                                            # softmax: so far below the largest
    check_route(to_dev(x.astype(np.float32)), topk, groups=groups, topk_groups=keep, group_top=group_top)


def test_far_scores_are_still_chosen_in_order():
    """Many rows at once, so that rows of both kinds share a workgroup."""
    say("moe_route rows near and far from the flush side by side")
    g = torch.Generator(device=device()).manual_seed(3)
    x = torch.randn((4001, 64), generator=g, device=device())
    x[::3] = x[::3] * 0.2 - 87.3
    ids, w = run_route(x, 4, score="sigmoid", groups=8, topk_groups=3, renorm=False)
    s = torch.sigmoid(x.double())
    best = s.view(-1, 8, 8).topk(2, 2).values.sum(2)
    kept = torch.zeros_like(best).scatter(1, best.topk(3, 1).indices, 1.0).repeat_interleave(8, 1).bool()
    want = torch.where(kept, s, -1.0).sort(dim=1, descending=True, stable=True)   # equal logits: the lower number
    assert torch.equal(ids.long(), want.indices[:, :4])
    # one fp32 rounding, and two steps of fp64's last bit between two exponentials
    want = want.values[:, :4]
    assert bool(((w.double() - want).abs() <= 2.0 ** -24 * 1.001 * want + 2.0 ** -150).all())
