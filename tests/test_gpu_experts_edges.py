"""GPU tests of the operators around an expert layer where their arithmetic is at its
edge, against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import gpu_helpers as H
from tests.test_gpu_experts import SIGMOID, SOFTMAX, check_route
from tests.test_gpu_grouped import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF, NAN = math.inf, math.nan
LARGEST = torch.finfo(torch.float32).max


# ---- routing -----------------------------------------------------------------------

@pytest.mark.parametrize("size", [1.0, 64.0, 1000.0])
@pytest.mark.parametrize("E,groups,group_top", [(32, 16, 3), (128, 64, 9), (256, 8, 3),
                                                (100, 50, 4)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_groups_whose_two_scores_cancel(gpu_lib, E, groups, group_top, size, score):
    """A group's two largest values are +size and -size and a score: each is rounded by
    2^-24 size, their sum is of the scores' order.  Scores that differ by about that
    rounding."""
    H.say(f"route cancelling groups E={E} groups={groups} size={size} score={score}")
    g = gen(E + int(size))
    bias = torch.full((groups, E // groups), -size)
    bias[:, 0] = size
    steps = size * U * (E if score == SOFTMAX else 4)
    logits = (torch.randn(E, generator=g) * 16 + torch.randn(60, E, generator=g) * 4) * steps
    check_route(logits, 4, bias=bias.reshape(-1), score=score, groups=groups,
                group_top=group_top, group_best=2, what=f"size={size}")
    check_route(logits - logits[:, :1], 4, bias=bias.reshape(-1), score=score, groups=groups,
                group_top=group_top, group_best=2, what=f"equal firsts, size={size}")


@pytest.mark.parametrize("E,groups", [(8, 4), (128, 8), (300, 100)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_groups_of_lowest_biases(gpu_lib, E, groups, score):
    """Biases of the lowest float (a mask): a group of them has a score, though the sum of
    two passes the largest float, and comes before a group in which nothing can be
    chosen; sums that pass it go by their real size."""
    H.say(f"route lowest biases E={E} groups={groups} score={score}")
    size = E // groups
    logits = torch.randn(9, E, generator=gen(E))
    logits[1:, :size] = -INF                 # nothing to choose in group 0
    logits[2, size:2 * size] = NAN
    logits[3] = -INF
    bias = torch.full((groups, size), -LARGEST)
    for top in (1, 2, groups - 1):
        check_route(logits, 2, bias=bias.reshape(-1), score=score, groups=groups, group_top=top,
                    group_best=2, what="all lowest")
    bias[-1] = -LARGEST * 0.75               # the best, whose sum is too large as well
    bias[1] = 0.0
    for top in (1, 2, groups - 1):
        check_route(logits, 2, bias=bias.reshape(-1), score=score, groups=groups, group_top=top,
                    group_best=2, what="two sums")
        check_route(logits, 2, bias=-bias.reshape(-1), score=score, groups=groups, group_top=top,
                    group_best=2, what="highest")
