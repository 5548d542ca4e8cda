"""GPU tests of the operators around an expert layer (``gemm_f32_route``,
``gemm_f32_route_grad``, ``gemm_f32_join_rows``, ``gemm_f32_join_rows_grad``,
``gemm_f32_norm``, ``gemm_f32_clip``) against their definitions in 64 bits, and of
the layer they make with the grouped products.

Gates, in steps U = 2^-24 (half an fp32 step relative to the value).  Choices are
equal.  A sigmoid is an exponential (a step, 2U, and U |l| for a rounded argument
of the same kind as below), a sum and a quotient: 8U.  A softmax rounds l - m (U |l -
m| of the exponential), takes it (2U), sums E / 64 + 6 deep, and divides: with D the
widest distance, (2 D + E / 64 + 16) U covers it and the scale.  Its gradient has
three such factors and a sum over the choices: (6 D + E / 16 + 3 top + 64) U of the
sum of magnitudes.  A sum of n products is off by n U of the sum of magnitudes.
"""
import math

import pytest
import torch

from dense_fp32_gemm_f32_amd import binding
from tests import gpu_helpers as H
from tests.test_gpu_grouped import device, gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SOFTMAX, SIGMOID = binding.SCORE_SOFTMAX, binding.SCORE_SIGMOID
INF, NAN = math.inf, math.nan
LARGEST = torch.finfo(torch.float32).max


def live(x):
    return x > -INF   # false for NaN


def scores(row, score):
    """Scores in 64 bits of one token's logits (a list)."""
    row = [min(x, LARGEST) if live(x) else -INF for x in row]
    if score == SIGMOID:
        return [0.0 if x == -INF else 1 / (1 + math.exp(-x)) if x > -700 else math.exp(x)
                for x in row]
    m = max(row, default=-INF)
    e = [0.0 if x == -INF else math.exp(x - m) for x in row]
    total = sum(e)
    return [x / total if total > 0 else 0.0 for x in e]


def choose(row, top, bias, score, groups, group_top, group_best):
    """The definition, for one token."""
    s = scores(row, score)
    E = len(row)
    v = []
    for i in range(E):
        x = (min(row[i], LARGEST) if bias is None else s[i] + min(bias[i], LARGEST)
             if bias[i] == bias[i] else NAN)
        v.append(x if live(row[i]) and live(x) else -INF)
    if group_top < groups:
        size = E // groups
        best = []
        for g in range(groups):
            part = [(s[i] if bias is None and group_best == 2 else v[i])
                    for i in range(g * size, (g + 1) * size) if v[i] > -INF]
            part.sort(reverse=True)
            best.append(sum(part[:group_best]) if part else -INF)
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:group_top]
        v = [x if i // size in kept else -INF for i, x in enumerate(v)]
    order = [i for i in sorted(range(E), key=lambda i: (-v[i], i)) if v[i] > -INF][:top]
    return order + [-1] * (top - len(order))


def weights(logits, choice, score, renorm, scale):
    """Weights in 64 bits as a function of the logits, the choices fixed."""
    x = torch.where(live(logits), logits.clamp_max(LARGEST), torch.full_like(logits, -INF))
    there = choice >= 0
    at = choice.clamp_min(0)
    if renorm:
        # log-scores of the chosen, so that no score underflows
        log = torch.nn.functional.logsigmoid(x) if score == SIGMOID else x
        log = torch.where(there, log.gather(1, at), torch.full_like(log[:, :1], -INF))
        w = torch.softmax(log.masked_fill(~there.any(1, keepdim=True), 0.0), 1)
    elif score == SIGMOID:
        w = torch.sigmoid(x).gather(1, at)
    else:
        w = torch.softmax(x.masked_fill(~live(x).any(1, keepdim=True), 0.0), 1).gather(1, at)
    return scale * torch.where(there, w, torch.zeros_like(w))


def spread(logits):
    ok = live(logits) & (logits < INF)
    x = logits.double()[ok]
    return float(x.max() - x.min()) if x.numel() else 0.0


def check_route(logits, top, *, bias=None, score=SOFTMAX, groups=1, group_top=None, group_best=1,
                renorm=False, scale=1.0, pad=0, shift=0, what=""):
    T, E = logits.shape
    gt = groups if group_top is None else group_top
    choice, weight = binding.route(device(logits, pad, shift), top,
                                   bias=None if bias is None else bias.cuda(), score=score,
                                   groups=groups, group_top=gt, group_best=group_best,
                                   renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    b = None if bias is None else bias.tolist()
    want = torch.tensor([choose(row, top, b, score, groups, gt, group_best)
                         for row in logits.tolist()], dtype=torch.int64).view(T, top)
    got = choice.cpu().long()
    assert torch.equal(got, want), \
        f"{what}: {(got != want).any(1).sum()} of {T} tokens have other choices"
    if E:
        w = weights(logits.double(), want, score, renorm, scale)
    else:
        w = torch.zeros(T, top, dtype=torch.float64)
    bound = ((2 * spread(logits) + E / 64 + 16) * w.abs() + abs(scale) * 2.0 ** -102) * U
    err = (weight.cpu().double() - w).abs()
    assert bool((err <= bound).all()), f"{what}: weights off by {float((err / bound).max()):.2f}"
    return choice, weight


# ---- routing -----------------------------------------------------------------------

@pytest.mark.parametrize("E", [1, 2, 3, 31, 64, 65, 128, 200, 256, 511, 1024])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_sizes(gpu_lib, E, score):
    for T, top, biased, renorm in ((1, 1, False, True), (5, min(E, 8), True, False),
                                   (9, min(E, 3), True, True)):
        g = gen(1000 * E + T)
        logits = torch.randn(T, E, generator=g) * 2
        bias = torch.randn(E, generator=g) * 0.1 if biased else None
        H.say(f"route T={T} E={E} top={top} score={score} bias={biased} renorm={renorm}")
        check_route(logits, top, bias=bias, score=score, renorm=renorm, scale=2.5, pad=T % 4,
                    shift=T % 3, what=f"T={T}")


@pytest.mark.parametrize("E,groups,group_top", [
    (8, 8, 3), (8, 2, 1), (64, 8, 4), (256, 8, 4), (96, 3, 2), (60, 4, 1), (100, 50, 7),
    (1024, 1024, 5), (1024, 2, 1), (7, 7, 6), (16, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_groups(gpu_lib, E, groups, group_top, biased, score):
    g = gen(E + groups)
    logits = torch.randn(11, E, generator=g)
    logits[3, ::2] = -INF
    logits[4, :E // groups] = -INF
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    for best in (1, 2):
        H.say(f"route groups E={E} groups={groups} top={group_top} best={best} bias={biased}")
        check_route(logits, min(E, 6), bias=bias, score=score, groups=groups,
                    group_top=group_top, group_best=best, renorm=best == 2, what=f"best={best}")


def test_route_ties_go_to_the_lowest(gpu_lib):
    H.say("route ties")
    g = gen(5)
    logits = torch.randint(-1, 2, (40, 96), generator=g).float()
    bias = torch.randint(-1, 2, (96,), generator=g).float()
    for score in (SOFTMAX, SIGMOID):
        check_route(logits, 10, score=score, what="logits")
        check_route(logits, 10, score=score, bias=torch.zeros(96), what="zero bias")
        check_route(logits, 10, score=score, groups=8, group_top=3, what="groups")
        check_route(torch.zeros(3, 96), 9, score=score, bias=bias, groups=12, group_top=5,
                    group_best=2, what="bias alone")


def test_route_scores_that_32_bits_cannot_tell_apart(gpu_lib):
    """Neighbouring fp32 logits far from zero have the same fp32 sigmoid, and sums
    with a bias that differ by less than a step."""
    H.say("route near ties")
    base = torch.full((64,), 12.0)
    steps = torch.randperm(64, generator=gen(1)).float()
    logits = (base + steps * 2.0 ** -20).repeat(6, 1)
    check_route(logits, 20, score=SIGMOID, what="no bias")
    check_route(logits, 20, score=SIGMOID, bias=torch.full((64,), 0.25), what="one bias")
    check_route(logits, 20, score=SOFTMAX, bias=torch.full((64,), 3.0), what="softmax")
    check_route(logits, 20, score=SIGMOID, bias=torch.full((64,), 0.25), groups=16, group_top=4,
                group_best=2, what="groups")


@pytest.mark.parametrize("E,groups,group_top", [(64, 1, 1), (100, 1, 1), (256, 8, 3), (250, 10, 4),
                                                (384, 12, 5), (1000, 1, 1), (1000, 8, 2)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_close_scores(gpu_lib, E, groups, group_top, score):
    """Clusters of scores that differ by about a step of 32 bits or not at all, at the
    last choice and the last group too."""
    g = gen(3 * E + groups)
    H.say(f"route close scores E={E} groups={groups} score={score}")
    for levels, steps in ((E // 5, 3), (2, 40), (1, 2)):
        logits = torch.randint(0, levels, (24, E), generator=g) * (2.0 / levels)
        logits = logits.float() + torch.randint(0, steps, (24, E), generator=g) * 2.0 ** -22
        bias = torch.randint(0, 2, (E,), generator=g) * 0.125
        logits[7, 3:] = -INF
        for best in (1, 2):
            check_route(logits, 8, bias=bias, score=score, groups=groups, group_top=group_top,
                        group_best=best, renorm=True, what=f"{levels} levels, best={best}")
        check_route(logits, 64, bias=bias, score=score, what=f"{levels} levels, 64 choices")


def test_route_masks_and_values_that_are_not_finite(gpu_lib):
    H.say("route masks")
    g = gen(7)
    logits = torch.randn(12, 70, generator=g)
    logits[0] = -INF                       # nothing left
    logits[1] = NAN
    logits[2, :68] = -INF                  # fewer than top
    logits[3, 5] = NAN
    logits[4, 6] = INF
    logits[5, [7, 9]] = INF
    logits[6, 1::2] = torch.finfo(torch.float32).min
    logits[7] = torch.finfo(torch.float32).min
    logits[8] = INF
    logits[9] = -200.0
    bias = torch.randn(70, generator=g)
    bias[[11, 12, 13]] = torch.tensor([NAN, -INF, INF])
    for score in (SOFTMAX, SIGMOID):
        for b in (None, bias):
            for renorm in (False, True):
                rows = logits[[0, 1, 2, 3, 6, 7, 9, 10, 11]]
                choice, weight = check_route(rows, 5, bias=b, score=score, renorm=renorm,
                                             what=f"score={score} bias={b is not None}")
                assert choice[0].tolist() == [-1] * 5 and weight[0].tolist() == [0.0] * 5
                assert choice[2].tolist()[2:] == [-1] * 3
    # +infinity counts as the largest finite number
    for renorm in (False, True):
        choice, weight = binding.route(logits[[4, 5, 8]].cuda(), 3, renorm=renorm)
        assert choice[0, 0] == 6 and choice[1, :2].tolist() == [7, 9]
        assert choice[2].tolist() == [0, 1, 2]
        assert weight[0].tolist() == [1.0, 0.0, 0.0]
        assert weight[1].tolist() == [0.5, 0.5, 0.0]


def test_route_renormalised_weights_of_scores_that_underflow(gpu_lib):
    """Chosen experts far below the others of an excluded group, or far below zero."""
    H.say("route underflow")
    logits = torch.tensor([[300.0, 299, 0, 1, 2, 3], [-300.0, -301, -299, -310, -305, -302]])
    bias = torch.tensor([-5.0, -5, 0, 0, 0, 0])
    check_route(logits[:1], 3, bias=bias, score=SOFTMAX, renorm=True, what="softmax")
    check_route(logits[1:], 3, score=SIGMOID, renorm=True, what="sigmoid")


def test_route_without_experts_and_of_all_experts(gpu_lib):
    H.say("route extremes")
    check_route(torch.zeros(4, 0), 3, what="no experts")
    check_route(torch.randn(6, 40, generator=gen(3)), 64, what="more than there are")
    check_route(torch.randn(6, 64, generator=gen(3)), 64, score=SIGMOID, renorm=True, what="all")
    assert binding.route(torch.zeros(0, 8, device="cuda"), 2)[0].shape == (0, 2)
    assert binding.route(torch.zeros(3, 8, device="cuda"), 0)[1].shape == (3, 0)


def test_route_of_many_tokens(gpu_lib):
    """Every token of a long batch is routed as it is alone."""
    H.say("route many tokens")
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(5003, 160, generator=g, device="cuda")
    how = {"score": SIGMOID, "groups": 8, "group_top": 3, "group_best": 2, "renorm": True,
           "bias": torch.randn(160, generator=g, device="cuda") * 0.1}
    choice, weight = binding.route(logits, 6, **how)
    for t in (0, 1, 2, 3, 4, 63, 64, 2500, 5002):
        c, w = binding.route(logits[t:t + 1], 6, **how)
        assert torch.equal(c[0], choice[t]) and torch.equal(w[0], weight[t])


# ---- the gradient of routing ----------------------------------------------------------

def check_grad(logits, choice, dweight, score, renorm, scale, pad=0, what=""):
    T, E = logits.shape
    top = choice.shape[1]
    out = device(torch.zeros(T, E), pad)
    got = binding.route_grad(dweight.cuda(), device(logits, pad), choice.int().cuda(), score=score,
                             renorm=renorm, scale=scale, dlogits=out)
    torch.cuda.synchronize()
    valid = (choice >= 0) & (choice < E)
    c = torch.where(valid, choice, torch.full_like(choice, -1))
    c = torch.where((c >= 0) & live(logits.gather(1, c.clamp_min(0))), c, torch.full_like(c, -1))
    x = logits.double().clone()
    x[~live(x)] = -INF
    x.requires_grad_(True)
    d = torch.where(c >= 0, dweight.double(), torch.zeros(1, dtype=torch.float64))
    w = weights(x, c, score, renorm, scale)
    w.backward(d)
    want = torch.where(live(logits), x.grad, torch.zeros(1, dtype=torch.float64)).nan_to_num()
    with torch.no_grad():
        # magnitudes: every term of the formula taken as positive
        share = weights(x.detach(), c, score, renorm, 1.0)
        size = (share * d.abs()).sum(1, keepdim=True) * abs(scale)
        mag = torch.zeros(T, E, dtype=torch.float64).scatter_add_(
            1, c.clamp_min(0), torch.where(c >= 0, share * (abs(scale) * d.abs() + size),
                                           torch.zeros(1, dtype=torch.float64)))
        if score == SOFTMAX and not renorm:
            full = torch.softmax(x.detach().masked_fill(~live(x).any(1, keepdim=True), 0.0), 1)
            mag = mag + full * size
    steps = 6 * spread(logits) + E / 16 + 3 * top + 64
    err = (got.cpu().double() - want).abs()
    bound = steps * U * mag + 2.0 ** -126
    assert bool((err <= bound).all()), f"{what}: off by {float((err / bound).max()):.2f} of the gate"
    return want


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (3, 8, 2), (5, 64, 8), (7, 65, 6), (4, 200, 5),
                                     (3, 512, 64), (2, 1024, 9), (6, 40, 40)])
def test_route_grad(gpu_lib, score, renorm, T, E, top):
    g = gen(T * E + top)
    logits = torch.randn(T, E, generator=g) * 1.5
    choice = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)])
    dweight = torch.randn(T, top, generator=g)
    H.say(f"route_grad T={T} E={E} top={top} score={score} renorm={renorm}")
    check_grad(logits, choice, dweight, score, renorm, 2.5, pad=T % 3, what="")


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_of_masked_rows(gpu_lib, score, renorm):
    """Rows without a choice, choices of nobody or outside, masked logits, and
    gradients that are not finite where nothing was chosen."""
    H.say(f"route_grad masks score={score} renorm={renorm}")
    g = gen(9)
    logits = torch.randn(8, 70, generator=g)
    logits[0] = -INF
    logits[1, 3] = NAN
    logits[2, 5:] = -INF
    choice = torch.stack([torch.randperm(5, generator=g)[:4] for _ in range(8)])
    choice[0] = -1
    choice[3, 1:] = -1
    choice[4, 2] = 70
    choice[5] = torch.tensor([2 ** 31 - 1, -2 ** 31, 4, 0])
    choice[1, 0] = 3                       # names the NaN
    choice[1, 1:] = torch.tensor([0, 1, 2])
    dweight = torch.randn(8, 4, generator=g)
    dweight[3, 1:] = NAN
    dweight[0] = INF
    want = check_grad(logits, choice, dweight, score, renorm, 1.0, what="masks")
    assert torch.equal(want[0], torch.zeros(70, dtype=torch.float64))


def test_route_grad_adds_an_expert_named_twice(gpu_lib):
    H.say("route_grad twice")
    logits = torch.randn(3, 9, generator=gen(4))
    choice = torch.tensor([[2, 2, 5], [0, 0, 0], [8, 1, 8]])
    dweight = torch.randn(3, 3, generator=gen(5))
    for renorm in (False, True):
        check_grad(logits, choice, dweight, SIGMOID, renorm, 1.0, what="sigmoid")
        check_grad(logits, choice, dweight, SOFTMAX, renorm, 1.0, what="softmax")


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_against_differences(gpu_lib, score, renorm):
    """Central differences of the weights in 64 bits.  With h = 2^-10 their error is
    h^2 / 6 times a third derivative, which for these scores of order one is below
    8 times the sum of |dw|."""
    H.say(f"route_grad differences score={score} renorm={renorm}")
    g = gen(11)
    logits = torch.randn(3, 12, generator=g)
    choice, _ = binding.route(logits.cuda(), 4, score=score, renorm=renorm)
    dweight = torch.randn(3, 4, generator=g)
    got = binding.route_grad(dweight.cuda(), logits.cuda(), choice, score=score,
                             renorm=renorm).cpu().double()
    c, x, h = choice.cpu().long(), logits.double(), 2.0 ** -10
    for i in range(12):
        e = torch.zeros(12, dtype=torch.float64)
        e[i] = h
        up, down = (weights(x + s * e, c, score, renorm, 1.0) for s in (1, -1))
        want = ((up - down) / (2 * h) * dweight.double()).sum(1)
        bound = (h * h / 6 * 8 + 200 * U) * dweight.double().abs().sum(1)
        assert bool(((got[:, i] - want).abs() <= bound).all())


# ---- the join of the experts' rows -------------------------------------------------------

def check_join(T, top, N, dropped, beta=0.0, pad=0, shift=0, groups=16):
    g = gen(T * 31 + top * 7 + N)
    h, w = torch.randn(T * top, N, generator=g), torch.randn(T, top, generator=g)
    choice = None
    there = torch.ones(T, top, dtype=torch.bool)
    hd = h.clone()
    if dropped:
        choice = torch.randint(0, groups, (T, top), generator=g).int()
        out = torch.rand(T, top, generator=g) < 0.3
        choice[out] = torch.tensor([-1, groups, 2 ** 31 - 1, -2 ** 31]).int()[
            torch.randint(0, 4, (int(out.sum()),), generator=g)]
        if T > 2:
            choice[1] = -1
        there = (choice >= 0) & (choice < groups)
        hd[~there.view(-1)] = NAN          # rows that nobody wrote
        h[~there.view(-1)] = 0
    y0 = torch.randn(T, N, generator=g)
    dy = torch.randn(T, N, generator=g)
    H.say(f"join T={T} top={top} N={N} dropped={dropped} beta={beta} pad={pad} shift={shift}")
    Hd, Wd = device(hd, pad, shift), w.cuda()
    cd = None if choice is None else choice.cuda()
    Yd = device(y0 if beta else torch.full_like(y0, NAN), pad, shift)
    got = binding.join_rows(Hd, Wd, cd, Yd, groups=groups, beta=beta)
    assert got.data_ptr() == Yd.data_ptr()
    dH = device(torch.full((T * top, N), NAN), pad, shift)
    dh, dw = binding.join_rows_grad(device(dy, pad, shift), Hd, Wd, cd, dH, groups=groups)
    torch.cuda.synchronize()
    wz = torch.where(there, w, torch.zeros(1)).double()
    terms = wz[:, :, None] * h.double().view(T, top, N)
    want = terms.sum(1) + beta * y0.double()
    mag = terms.abs().sum(1) + abs(beta) * y0.double().abs()
    assert bool(((got.cpu().double() - want).abs() <= (top + 2) * U * mag).all())
    want = (wz[:, :, None] * dy.double()[:, None, :]).view(T * top, N)
    assert bool(((dh.cpu().double() - want).abs() <= U * want.abs()).all())
    prod = h.double().view(T, top, N) * dy.double()[:, None, :]
    err = (dw.cpu().double() - prod.sum(2)).abs()
    assert bool((err <= (N + 2) * U * prod.abs().sum(2)).all())
    if pad:   # the pitch's padding is left as it was
        flat = torch.as_strided(got, (T, N + pad), (N + pad, 1), shift).cpu()
        assert bool(flat[:, N:].isnan().all())
        flat = torch.as_strided(dh, (T * top, N + pad), (N + pad, 1), shift).cpu()
        assert bool(flat[:, N:].isnan().all())


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 31, 32, 63, 255, 256, 257, 1023, 1024, 1030, 4100])
@pytest.mark.parametrize("dropped", [False, True])
def test_join_widths(gpu_lib, N, dropped):
    check_join(5, 3, N, dropped)
    check_join(4, 2, N, dropped, beta=0.5, pad=3, shift=1)


@pytest.mark.parametrize("T,top", [(1, 1), (1, 8), (3, 64), (257, 1), (300, 5), (64, 7), (2, 100)])
@pytest.mark.parametrize("N", [40, 600])
def test_join_rows_of_tokens(gpu_lib, T, top, N):
    check_join(T, top, N, T % 2 == 0, beta=-1.0 if top == 5 else 0.0)


def test_join_of_nothing(gpu_lib):
    H.say("join of nothing")
    y = binding.join_rows(torch.zeros(0, 9, device="cuda"), torch.zeros(4, 0, device="cuda"))
    assert torch.equal(y, torch.zeros(4, 9, device="cuda"))
    old = torch.ones(4, 9, device="cuda")
    binding.join_rows(torch.zeros(0, 9, device="cuda"), torch.zeros(4, 0, device="cuda"), None, old,
                      beta=2.0)
    assert torch.equal(old, torch.full((4, 9), 2.0, device="cuda"))
    _, dw = binding.join_rows_grad(torch.zeros(3, 0, device="cuda"), torch.zeros(6, 0, device="cuda"),
                                   torch.ones(3, 2, device="cuda"))
    assert torch.equal(dw, torch.zeros(3, 2, device="cuda"))


# ---- the norm of many arrays, and clipping ------------------------------------------------

def arrays(sizes, seed, scale=1.0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n + shift, generator=g, device="cuda") * scale)[shift:] for n in sizes]


SIZES = {
    "one": [1], "few": [3, 0, 5, 1023, 1, 4096], "chunks": [16383, 16384, 16385, 40000],
    "many": [(37 * i) % 900 for i in range(230)], "large": [5000003, 17, 1 << 20],
    "nothing": [0, 0]}


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("factor", [0.5, 2.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(gpu_lib, name, shift, factor, in_place):
    H.say(f"clip {name} shift={shift} factor={factor} in_place={in_place}")
    xs = arrays(SIZES[name], 3, shift=shift)
    before = [x.cpu().double() for x in xs]
    exact = math.sqrt(sum(float((x * x).sum()) for x in before))
    limit = torch.tensor(exact * factor, dtype=torch.float32).item()
    alone = binding.norm(xs)
    outs = None if in_place else [torch.full_like(x, NAN) for x in xs]
    norm = binding.clip_norm(xs, limit, out=outs)
    torch.cuda.synchronize()
    assert torch.equal(alone, norm)
    # 64-bit sums, rounded once
    assert abs(norm.item() - exact) <= exact * (U + 2.0 ** -40)
    by = limit / exact if exact > limit else 1.0
    for x, old, y in zip(xs, before, xs if in_place else outs):
        got = y.cpu().double()
        if by == 1.0:
            assert torch.equal(got, old)
        else:   # the factor and the product each round once
            assert bool(((got - old * by).abs() <= 3 * U * (old * by).abs()).all())
        if not in_place:
            assert torch.equal(x.cpu().double(), old)


def test_norm_of_extreme_values(gpu_lib):
    H.say("norm extremes")
    big, small = 3e38, 1e-38
    one = lambda *v: torch.tensor(v, device="cuda")
    assert binding.norm([one(big), one(0.0)]).item() == torch.tensor(big).item()
    want = torch.tensor(small).item()
    assert abs(binding.norm([one(small)]).item() - want) <= want * U
    assert binding.norm([one(big, big)]).item() == INF     # past the largest float
    x = [one(big, big)]
    binding.clip_norm(x, 1.0)                              # ... but finite: it is scaled
    assert bool(((x[0].cpu().double() - 0.5 ** 0.5).abs() < 4 * U).all())
    for bad in (INF, -INF, NAN):
        x = [one(1.0, bad, 2.0), one(5.0)]
        norm = binding.clip_norm(x, 1.0)
        assert not math.isfinite(norm.item())
        assert x[0][0].item() == 1.0 and x[0][2].item() == 2.0 and x[1].item() == 5.0
    x = [one(3.0, 4.0)]
    assert binding.clip_norm(x, 0.0).item() == 5.0 and x[0].tolist() == [0.0, 0.0]
    x = [one(3.0, 4.0)]
    binding.clip_norm(x, INF)
    assert x[0].tolist() == [3.0, 4.0]


def test_clip_repeats_bit_for_bit(gpu_lib):
    H.say("clip repeats")
    xs = arrays([300000, 7, 65536, 12345], 8)
    outs = [[torch.empty_like(x) for x in xs] for _ in range(3)]
    norms = [binding.clip_norm(xs, 10.0, out=o) for o in outs]
    for norm, out in zip(norms[1:], outs[1:]):
        assert torch.equal(norm, norms[0])
        assert all(torch.equal(a, b) for a, b in zip(out, outs[0]))


def test_clip_refuses_arrays_that_overlap(gpu_lib):
    H.say("clip overlap")
    x = torch.ones(100, device="cuda")
    for call in (lambda: binding.clip_norm([x, x], 1.0), lambda: binding.clip_norm([x, x[50:]], 1.0),
                 lambda: binding.clip_norm([x[:50], x[50:]], 1.0, out=[x[50:], x[:50]])):
        with pytest.raises(binding.GemmError) as e:
            call()
        assert e.value.status == 4
    assert torch.equal(x, torch.ones(100, device="cuda"))
    assert abs(binding.norm([x, x]).item() - 200 ** 0.5) < 1e-5


# ---- graphs and streams ---------------------------------------------------------------------

def test_captured_calls_replay(gpu_lib):
    """One graph of routing, its order, the join, the gradients and clipping; new
    inputs and eager work between the replays."""
    H.say("captured layer")
    T, E, top, N = 37, 24, 3, 130
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    h = torch.randn(T * top, N, generator=g, device="cuda")
    dy = torch.randn(T, N, generator=g, device="cuda")
    grads = arrays([5000, 33, 70000], 2)
    outs = [torch.empty_like(x) for x in grads]

    def step():
        choice, weight = binding.route(logits, top, score=SIGMOID, renorm=True, groups=4,
                                       group_top=2)
        order = binding.group_rows(choice.view(-1), E, per_row=top)
        y = binding.join_rows(h, weight, choice, groups=E)
        dh, dw = binding.join_rows_grad(dy, h, weight, choice, groups=E)
        dl = binding.route_grad(dw, logits, choice, score=SIGMOID, renorm=True)
        return [choice, weight, *order, y, dh, dw, dl, binding.clip_norm(grads, 5.0, out=outs),
                *outs]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = step()
        for seed in (5, 6, 7):
            g.manual_seed(seed)
            for t in (logits, h, dy, *grads):
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
            graph.replay()
            stream.synchronize()
            kept = [t.clone() for t in captured]
            for a, b in zip(kept, step()):
                assert torch.equal(a, b)
            stream.synchronize()


def test_calls_on_streams_at_once(gpu_lib):
    """The calls in turn on four streams, each with its inputs: as one after another."""
    H.say("calls on streams at once")
    T, E, top, N, K = 300, 64, 4, 520, 384
    streams = [torch.cuda.Stream() for _ in range(4)]

    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device="cuda")
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        return dict(logits=draw(T, E), bias=draw(E), h=draw(T * top, N), a=draw(T, K),
                    codes=codes, scale=draw(N, K // 32).abs(),
                    grads=[draw(n) for n in (70001, 3, 200000)])

    def calls(x):
        choice, weight = binding.route(x["logits"], top, bias=x["bias"], score=SIGMOID)
        y = binding.join_rows(x["h"], weight, choice, groups=E)
        few = binding.gemm_q4(x["a"][:3], x["codes"], x["scale"], group=32)
        many = binding.gemm_q4(x["a"], x["codes"], x["scale"], group=32)
        outs = [torch.empty_like(t) for t in x["grads"]]
        return [choice, weight, y, few, many, binding.clip_norm(x["grads"], 5.0, out=outs), *outs]

    sets = [inputs(seed) for seed in range(4)]
    want = [calls(x) for x in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for stream, x in zip(streams, sets):
            with torch.cuda.stream(stream):
                got.append(calls(x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_clip_needs_its_workspace_before_capture(gpu_lib):
    H.say("clip captured without a workspace")
    x = [torch.ones(1000, device="cuda")]
    norm = torch.empty(1, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            with pytest.raises(binding.GemmError) as e:
                binding.clip_norm(x, 1.0, norm=norm)
            norm.zero_()
    assert e.value.status == 6


# ---- together -----------------------------------------------------------------------------------

def test_an_expert_layer_forward_and_backward(gpu_lib):
    """logits, routing, order, up and down products, join, and every gradient back to
    the router's logits and the input, then clipping; against 64 bits with the same
    choices."""
    H.say("expert layer")
    T, E, top, D, F = 61, 6, 2, 40, 56
    g = gen(21)
    x, wr = torch.randn(T, D, generator=g), torch.randn(D, E, generator=g) * 0.3
    up = torch.randn(E, D, F, generator=g) * D ** -0.5
    down = torch.randn(E, F, D, generator=g) * F ** -0.5
    dy = torch.randn(T, D, generator=g)
    X, WR, UP, DOWN, DY = (t.cuda() for t in (x, wr, up, down, dy))
    b = binding
    logits = b.gemm(X, WR)
    choice, weight = b.route(logits, top, renorm=True)
    offsets, order, token = b.group_rows(choice.view(-1), E, per_row=top)
    h = b.gemm_grouped(X, UP, offsets, index_a=token, act=b.ACT_RELU)
    out = X.new_empty(T * top, D)
    b.gemm_grouped(h, DOWN, offsets, out, index_c=order)
    y = b.join_rows(out, weight, choice, groups=E)
    dout, dweight = b.join_rows_grad(DY, out, weight, choice, groups=E)
    dlogits = b.route_grad(dweight, logits, choice, renorm=True)
    dh = b.gemm_grouped(dout, DOWN, offsets, trans_b=True, index_a=order) * (h > 0)
    d_down = b.gemm_grouped_wgrad(h, dout, offsets, index_b=order)
    d_up = b.gemm_grouped_wgrad(X, dh, offsets, index_a=token)
    d_wr = b.gemm_ex(X, dlogits, trans_a=True)
    got = {"y": y, "wr": d_wr, "up": d_up, "down": d_down}

    P = {k: v.double().requires_grad_(True) for k, v in
         (("wr", wr), ("up", up), ("down", down))}
    xd, c = x.double(), choice.cpu().long()
    lg = xd @ P["wr"]
    w = torch.softmax(lg.gather(1, c), 1)
    hidden = torch.relu(torch.einsum("td,tkdf->tkf", xd, P["up"][c]))
    rows = torch.einsum("tkf,tkfd->tkd", hidden, P["down"][c])
    want = (w[:, :, None] * rows).sum(1)
    want.backward(dy.double())
    # sums of up to T top products of factors that carry K-term sums themselves: the
    # largest magnitude times the depth of all sums covers each entry
    steps = (D + F + T * top + 64) * U
    for name, t in got.items():
        ref = want.detach() if name == "y" else P[name].grad
        err = (t.cpu().double() - ref).abs().max()
        assert err <= steps * 16 * ref.abs().max(), f"{name}: {float(err)}"
    grads = [d_wr, d_up, d_down]
    norm = b.clip_norm(grads, 1.0)
    exact = math.sqrt(sum(float((P[k].grad ** 2).sum()) for k in P))
    assert abs(norm.item() - exact) <= exact * steps * 16
    assert abs(b.norm(grads).item() - 1.0) < 8 * U
