"""GPU tests of the operators around an expert layer where their arithmetic is at its
edge, against their definitions in 64 bits."""
import math

import pytest
import torch

from dense_fp32_gemm_f32_amd import binding
from tests import gpu_helpers as H
from tests.test_gpu_experts import SIGMOID, SOFTMAX, check_grad, check_route
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


# ---- the gradient of routing ----------------------------------------------------------

def centred(share, g):
    """sum_k share_k (g_i - g_k), the formula's g_i - sum share_k g_k (shares add up to
    one, or are all zero), and the sum of magnitudes without i = k."""
    by = g[:, :, None] - g[:, None, :]
    return (share[:, None, :] * by).sum(2), \
        (share[:, None, :] * (g.abs()[:, :, None] + g.abs()[:, None, :])
         * (1 - torch.eye(g.shape[1], dtype=g.dtype))).sum(2)


def check_slopes(logits, choice, dweight, score, renorm, what):
    """route_grad against the formulas in 64 bits, each factor by itself: 1 - s as
    sigmoid(-x), and a share that is nearly one by the others' sum.  Gates: of an exponential
    2U and U |x|, a sum (E / 64 + 6) U, a quotient U: of a factor (D + E / 64 + 16) U, D the
    widest distance; three of them, the products, and the sum over the choices (and over
    the experts where all take part) of the sum of magnitudes."""
    T, E = logits.shape
    top = choice.shape[1]
    got = binding.route_grad(dweight.cuda(), logits.cuda(), choice.int().cuda(), score=score,
                             renorm=renorm).cpu().double()
    x, d = logits.double(), dweight.double()
    cx = x.gather(1, choice)
    slope = torch.sigmoid(-cx)                       # 1 - s
    if renorm:
        log = torch.nn.functional.logsigmoid(cx) if score == SIGMOID else cx
        share = torch.softmax(log, 1)
        value, mag = centred(share, d)
        value, mag = share * value, share * mag
        if score == SIGMOID:
            value, mag = value * slope, mag * slope
        zero = torch.zeros(T, E, dtype=torch.float64)
        want = zero.scatter_add(1, choice, value)
        mag = zero.scatter_add(1, choice, mag)
    elif score == SIGMOID:
        zero = torch.zeros(T, E, dtype=torch.float64)
        want = zero.scatter_add(1, choice, torch.sigmoid(cx) * slope * d)
        mag = want.abs()
    else:
        g = torch.zeros(T, E, dtype=torch.float64).scatter_add(1, choice, d)
        share = torch.softmax(x, 1)
        value, mag = centred(share, g)
        want, mag = share * value, share * mag
    D = float((x.max(1).values - x.min(1).values).max())
    steps = 6 * D + E / 16 + 3 * top + 64
    err = (got - want).abs()
    bound = steps * U * mag + 2.0 ** -126
    assert bool((err <= bound).all()), f"{what}: off by {float((err / bound).max()):.2f} of the gate"


@pytest.mark.parametrize("T,E,top", [(40, 2, 2), (40, 1, 1), (30, 64, 8), (20, 130, 6),
                                     (9, 300, 3), (5, 1024, 20)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_of_large_sigmoid_logits(gpu_lib, T, E, top, renorm):
    """Logits of +8 to +30, where 1 - s has to come from the logit."""
    H.say(f"route_grad sigmoid, large logits T={T} E={E} top={top} renorm={renorm}")
    g = gen(T + E)
    logits = 8 + 22 * torch.rand(T, E, generator=g)
    if not renorm:   # and far below zero
        logits[::3] *= -1
    choice = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)])
    check_slopes(logits, choice, torch.randn(T, top, generator=g), SIGMOID, renorm, "large")


@pytest.mark.parametrize("T,E,top", [(40, 2, 1), (40, 2, 2), (30, 64, 8), (20, 130, 6),
                                     (9, 300, 3), (5, 1024, 20)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_of_one_expert_above_all(gpu_lib, T, E, top, score, renorm):
    """One expert's share is nearly one: 1 less that share has to come from the others'.
    Chosen in most rows, not in some, and two that share the lead."""
    H.say(f"route_grad one above all T={T} E={E} top={top} score={score} renorm={renorm}")
    g = gen(T * E + 1)
    logits = torch.randn(T, E, generator=g)
    if score == SIGMOID:   # where a sigmoid is the exponential
        logits -= 45
    choice = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)])
    lead = choice[:, top // 2].clone()
    lead[::5] = torch.randint(0, E, lead[::5].shape, generator=g)
    logits[torch.arange(T), lead] += 2 + 30 * torch.rand(T, generator=g)
    second = choice[1::4, 0]
    logits[1::4].scatter_(1, second[:, None], logits[1::4].max(1, keepdim=True).values)
    check_slopes(logits, choice, torch.randn(T, top, generator=g), score, renorm, "one above")


@pytest.mark.parametrize("T,E,top", [(40, 2, 2), (30, 64, 8), (9, 300, 3)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_grad_of_one_above_and_nearly_equal_gradients(gpu_lib, T, E, top, score):
    """Where a share is above a half the gradients enter by their differences, which are
    exact: the gate is of sum_k share_k |g_i - g_k|, for g that differ by 2^-20 of
    themselves."""
    H.say(f"route_grad nearly equal T={T} E={E} top={top} score={score}")
    g = gen(T + E + 3)
    logits = torch.randn(T, E, generator=g) - (45 if score == SIGMOID else 0)
    choice = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)])
    logits.scatter_add_(1, choice[:, :1], 9 + 20 * torch.rand(T, 1, generator=g))
    dweight = 1 + torch.randint(-8, 9, (T, top), generator=g) * 2.0 ** -23
    got = binding.route_grad(dweight.cuda(), logits.cuda(), choice.int().cuda(), score=score,
                             renorm=True).cpu().double().gather(1, choice)
    cx, d = logits.double().gather(1, choice), dweight.double()
    share = torch.softmax(torch.nn.functional.logsigmoid(cx) if score == SIGMOID else cx, 1)
    by = share[:, None, :] * (d[:, :, None] - d[:, None, :])
    slope = torch.sigmoid(-cx) if score == SIGMOID else torch.ones_like(cx)
    want, mag = share * slope * by.sum(2), share * slope * by.abs().sum(2)
    # as check_slopes; g_i - g_m and the sum are each at most twice the sum of magnitudes
    steps = 4 * (6 * float((cx.max(1).values - cx.min(1).values).max()) + 3 * top + 64)
    assert bool(((got - want).abs() <= steps * U * mag + 2.0 ** -126).all())


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_grad_of_tokens_with_fewer_choices(gpu_lib, renorm, score):
    """Tokens with some choices, but fewer than top, as routing leaves them: masks, and
    groups that hold fewer experts.  Nothing reaches an expert that was not chosen by way of
    the entries without a choice."""
    H.say(f"route_grad fewer choices score={score} renorm={renorm}")
    g = gen(17)
    logits = torch.randn(40, 12, generator=g)
    logits[torch.rand(40, 12, generator=g) < 0.3] = -INF
    logits[0] = -INF
    dweight = torch.randn(40, 7, generator=g)
    for how in ({}, {"groups": 3, "group_top": 1}, {"groups": 6, "group_top": 2, "group_best": 2}):
        choice, _ = check_route(logits, 7, score=score, renorm=renorm, what=str(how), **how)
        choice = choice.cpu().long()
        assert bool(((choice < 0).any(1) & (choice >= 0).any(1)).any())
        check_grad(logits, choice, dweight, score, renorm, 2.5, what=str(how))


# ---- clipping ------------------------------------------------------------------------

@pytest.mark.parametrize("limit", [1.0, 1e-3, 1e-8, 1e-30, 1e-37])
@pytest.mark.parametrize("size", [3e38, 1e30, 1e-3])
def test_clip_by_factors_below_the_smallest_float(gpu_lib, limit, size):
    """limit / norm below 2^-126, where a float of it has few bits or none, times elements
    that are as large.  Chunks of 16 bytes, ends, and elements by themselves."""
    H.say(f"clip limit={limit} size={size}")
    g = gen(31)
    xs = [(torch.rand(n, generator=g) * 2 - 1) * size for n in (40000, 1, 5, 1027)]
    big = torch.tensor(limit).item()
    exact = math.sqrt(sum(float((x.double() ** 2).sum()) for x in xs))
    outs = [torch.full_like(x, NAN).cuda() for x in xs]
    norm = binding.clip_norm([x.cuda() for x in xs], limit, out=outs).item()
    assert norm == (INF if exact > LARGEST else norm)
    for x, y in zip(xs, outs):
        want = x.double() * min(1.0, big / exact)
        # the factor and the product each round; below 2^-126 by half of 2^-149
        assert bool(((y.cpu().double() - want).abs() <= 3 * U * want.abs() + 2.0 ** -150).all())
