"""GPU tests of the operators around an expert layer where their arithmetic is at its
edge, against their definitions in 64 bits."""
import pytest
import torch

from tests import gpu_helpers as H
from tests.test_gpu_experts import SIGMOID, SOFTMAX, check_route
from tests.test_gpu_grouped import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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
