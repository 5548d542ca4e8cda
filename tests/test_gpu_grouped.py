"""GPU tests of the products whose rows belong to different weights
(``gemm_f32_group_rows``, ``gemm_f32_grouped``, ``gemm_f32_grouped_wgrad``,
``gemm_f32_adapters``) against their definitions in 64 bits.

Gates.  Whole-number inputs (-2 .. 2, and halves where a factor scales them):
every partial sum is exact in fp32, so the result equals the 64-bit one bit
for bit whatever the order.  General inputs: a sum of K products and n further
fp32 operations is off by at most (K + n) 2^-24 of the sum of magnitudes
(each rounding half a step), in any order of summation.
"""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def draw(g, *shape, integer):
    if integer:
        return torch.randint(-2, 3, shape, generator=g).float()
    return torch.randn(*shape, generator=g)


def device(x, pad=0, shift=0, fill=float("nan")):
    """x on the GPU with its last-but-one stride padded and its start shifted,
    NaN in between."""
    *lead, rows, cols = x.shape
    pitch = cols + pad
    n = 1
    for d in lead:
        n *= d
    flat = torch.full((n * rows * pitch + shift + 4,), fill)
    view = torch.as_strided(flat, (n, rows, cols), (rows * pitch, pitch, 1), shift)
    view.copy_(x.reshape(n, rows, cols))
    return torch.as_strided(flat.cuda(), tuple(lead) + (rows, cols),
                            (rows * pitch,) * len(lead) + (pitch, 1), shift)


def spans(counts, spare=0):
    """offsets of groups with these counts, and the number of places."""
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32), off[-1] + spare


def check(got, want, mag, ops, integer, what):
    got = got.cpu().double()
    if integer:
        assert torch.equal(got, want), f"{what}: {(got != want).sum()} of {got.numel()} differ"
    else:
        err = (got - want).abs()
        assert bool((err <= ops * U * mag).all()), \
            f"{what}: off by {float((err / mag.clamp_min(1e-30)).max()) / U:.1f} of {ops} steps"


# ---- rows ordered by group -------------------------------------------------------

@pytest.mark.parametrize("n,groups,per_row", [
    (0, 5, 1), (1, 1, 1), (3, 0, 1), (63, 2, 1), (64, 64, 2), (65, 3, 5), (1000, 7, 4),
    (1024, 1, 1), (4099, 1024, 3), (5000, 257, 1), (70001, 64, 4), (300007, 33, 1)])
def test_group_rows(gpu_lib, n, groups, per_row):
    g = gen(n + groups)
    index = torch.randint(-1, groups + 1, (n,), generator=g).int()
    if n > 10:   # far outside, and the neighbours of the range
        index[::7] = torch.tensor([-2 ** 31, 2 ** 31 - 1, groups, -1]).int().repeat(n)[:len(index[::7])]
    H.say(f"group_rows n={n} groups={groups} per_row={per_row}")
    offsets, order, rows = gpu_lib.group_rows(index.cuda(), groups, per_row=per_row)
    torch.cuda.synchronize()
    i = index.long()
    kept = (i >= 0) & (i < groups)
    places = torch.nonzero(kept)[:, 0]
    want = places[torch.sort(i[places], stable=True).indices]
    counts = torch.bincount(i[places], minlength=groups)[:groups]
    assert offsets.cpu().tolist() == [0] + torch.cumsum(counts, 0).tolist()
    tail = torch.full((n - want.numel(),), -1)
    assert torch.equal(order.cpu().long(), torch.cat([want, tail]))
    assert torch.equal(rows.cpu().long(), torch.cat([want // per_row, tail]))


@pytest.mark.parametrize("value", [-1, 0, 4, 5])
def test_group_rows_of_one_value(gpu_lib, value):
    """All entries in one group, or in none."""
    n, groups = 777, 5
    H.say(f"group_rows all {value}")
    offsets, order, _ = gpu_lib.group_rows(torch.full((n,), value, dtype=torch.int32).cuda(),
                                           groups)
    inside = 0 <= value < groups
    assert offsets.cpu().tolist() == [n if inside and g > value else 0 for g in range(groups + 1)]
    assert order.cpu().tolist() == (list(range(n)) if inside else [-1] * n)


# ---- products grouped by expert ---------------------------------------------------

COUNTS = {
    "one": [1],
    "few": [0, 3, 0, 1, 17, 0],
    "even": [16, 16, 16, 16],
    "skewed": [0, 130, 1, 64, 65, 0, 300, 7],
    "many": [(7 * i) % 5 for i in range(150)],
    "none": [0, 0, 0],
    "long": [513, 700],
    "most": [2 if i in (0, 700, 1023) else 0 for i in range(1024)],
}


def grouped_case(lib, counts, K, N, trans, gather, scatter, epilogue, integer, seed, pads=(0, 0, 0),
                 shifts=(0, 0, 0), spare=3):
    """One product against its definition; returns nothing, asserts everything:
    values, and NaN wherever nothing may be written."""
    g = gen(seed)
    offsets, rows = spans(counts, spare)
    G = len(counts)
    rows_a = rows + 5 if not gather else max(1, rows // 2)
    rows_c = rows + 9
    A = draw(g, rows_a, K, integer=integer)
    W = draw(g, G, *((N, K) if trans else (K, N)), integer=integer)
    ia = torch.randint(0, rows_a, (rows,), generator=g).int() if gather else None
    ic = torch.randperm(rows_c, generator=g)[:rows].int() if scatter else None
    alpha, beta, bias, act = (0.5, -2.0, draw(g, G, N, integer=integer), 1) if epilogue else \
        (1.0, 0.0, None, 0)
    C0 = draw(g, rows_c, N, integer=integer)
    Ad, Wd = device(A, pads[0], shifts[0]), device(W, pads[1], shifts[1])
    Cd = device(C0 if epilogue else torch.full_like(C0, float("nan")), pads[2], shifts[2])
    before = Cd.cpu().double()
    H.say(f"grouped counts={counts[:8]} K={K} N={N} trans={trans} gather={gather} "
          f"scatter={scatter} epilogue={epilogue} int={integer} pads={pads} shifts={shifts}")
    lib.gemm_grouped(Ad, Wd, offsets.cuda(), Cd, trans_b=trans, alpha=alpha, beta=beta,
                     bias=None if bias is None else bias.cuda(), act=act,
                     index_a=None if ia is None else ia.cuda(),
                     index_c=None if ic is None else ic.cuda())
    torch.cuda.synchronize()
    want, mag = before.clone(), torch.ones_like(before)
    for e, (b, f) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        if f == b:
            continue
        at = torch.arange(b, f)
        src = ia[b:f].long() if gather else at
        dst = ic[b:f].long() if scatter else at
        w = W[e].double().t() if trans else W[e].double()
        v = alpha * (A[src].double() @ w)
        m = abs(alpha) * (A[src].double().abs() @ w.abs())
        if epilogue:
            v = v + beta * before[dst] + bias[e].double()
            m = m + (beta * before[dst]).abs() + bias[e].double().abs()
            v = v.clamp_min(0)
        want[dst], mag[dst] = v, m
    named = ~torch.isnan(want)
    got = Cd.cpu()
    assert torch.equal(~torch.isnan(got), named), "a row that no place names was written"
    check(got[named], want[named], mag[named], K + 4, integer, "grouped")


@pytest.mark.parametrize("integer", [True, False])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_grouped_counts(gpu_lib, counts, trans, integer):
    grouped_case(gpu_lib, COUNTS[counts], 64, 96, trans, True, False, False, integer, 11)


@pytest.mark.parametrize("gather,scatter,epilogue", [
    (False, False, True), (True, True, False), (False, True, True), (True, True, True)])
@pytest.mark.parametrize("counts", ["few", "skewed"])
def test_grouped_indexes_and_epilogue(gpu_lib, counts, gather, scatter, epilogue):
    for trans in (False, True):
        for integer in (True, False):
            grouped_case(gpu_lib, COUNTS[counts], 48, 132, trans, gather, scatter, epilogue,
                         integer, 12)


@pytest.mark.parametrize("K", [0, 1, 3, 4, 15, 16, 17, 31, 36, 100, 127, 260, 1031])
def test_grouped_inner_sizes(gpu_lib, K):
    for counts in ("few", "skewed"):
        for trans in (False, True):
            grouped_case(gpu_lib, COUNTS[counts], K, 68, trans, True, True, True, True, 13)
            grouped_case(gpu_lib, COUNTS[counts], K, 68, trans, True, False, False, False, 14)


@pytest.mark.parametrize("N", [1, 2, 5, 16, 33, 64, 129, 260, 515])
def test_grouped_widths(gpu_lib, N):
    for counts in ("few", "skewed"):
        for trans in (False, True):
            grouped_case(gpu_lib, COUNTS[counts], 40, N, trans, True, True, True, True, 15)


@pytest.mark.parametrize("pads,shifts", [((4, 8, 4), (0, 0, 0)), ((1, 3, 5), (0, 0, 0)),
                                         ((0, 0, 0), (1, 2, 3)), ((2, 0, 1), (0, 3, 0)),
                                         ((0, 1, 0), (0, 0, 1))])
def test_grouped_pitches_and_alignment(gpu_lib, pads, shifts):
    for counts in ("few", "skewed"):
        for trans in (False, True):
            grouped_case(gpu_lib, COUNTS[counts], 96, 72, trans, True, True, True, True, 16, pads,
                         shifts)


@pytest.mark.parametrize("K,N", [(512, 384), (1000, 260), (773, 517)])
@pytest.mark.parametrize("trans", [False, True])
def test_grouped_larger(gpu_lib, K, N, trans):
    for counts in ([700, 0, 1300, 90], [5, 9, 0, 2, 16, 16, 15], [1] * 40):
        grouped_case(gpu_lib, counts, K, N, trans, True, False, False, True, 17)
        grouped_case(gpu_lib, counts, K, N, trans, False, True, True, False, 18)


# 24 uneven groups, one of them empty: enough tiles that every tiled kernel takes some
# width (even and odd, two thirds of a round over one, four rounds and more)
MANY_TILES = [0] + [100 + (131 * i) % 400 for i in range(1, 24)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K,N", [(0, 600), (4, 600), (100, 600), (36, 440), (132, 2048),
                                 (1, 601), (17, 601), (127, 601), (3, 2047), (65, 2047)])
def test_grouped_uneven_tiles(gpu_lib, K, N, trans):
    grouped_case(gpu_lib, MANY_TILES, K, N, trans, True, True, True, True, 66)
    grouped_case(gpu_lib, MANY_TILES, K, N, trans, False, False, False, False, 67)


@pytest.mark.parametrize("pads,shifts", [((4, 8, 4), (0, 0, 0)), ((1, 3, 5), (0, 0, 0)),
                                         ((0, 0, 0), (1, 2, 3)), ((0, 0, 3), (0, 0, 1))])
@pytest.mark.parametrize("N", [600, 2048])
def test_grouped_uneven_tiles_pitches(gpu_lib, N, pads, shifts):
    for trans in (False, True):
        grouped_case(gpu_lib, MANY_TILES, 48, N, trans, True, False, True, True, 68, pads, shifts)


@pytest.mark.parametrize("rows,N", [(90, 64), (90, 200), (3000, 1024), (3000, 1025)])
@pytest.mark.parametrize("trans", [False, True])
def test_grouped_rows_outside_meet_no_weight(gpu_lib, rows, N, trans):
    """A row of A whose index is outside gives the update of an empty sum, also
    where the weights it would meet are not finite, in every kernel."""
    g = gen(69)
    K = 64
    A, W = draw(g, rows, K, integer=True), torch.full((2, K, N), float("inf"))
    W[1] = draw(g, K, N, integer=True)
    b = draw(g, 2, N, integer=True)
    half = rows // 2
    offsets, _ = spans([half, rows - half])
    ia = torch.arange(rows).int()
    ia[:half] = -1
    ia[half + 1] = rows
    H.say(f"grouped rows outside rows={rows} N={N} trans={trans}")
    B = W.transpose(1, 2).contiguous() if trans else W
    got = gpu_lib.gemm_grouped(A.cuda(), B.cuda(), offsets.cuda(), trans_b=trans, bias=b.cuda(),
                               index_a=ia.cuda()).cpu()
    want = A @ W[1] + b[1]
    want[:half], want[half + 1] = b[0], b[1]
    assert torch.equal(got, want)


def test_grouped_shared_weight_and_bias(gpu_lib):
    """Strides of 0: one weight and one bias for every group."""
    g = gen(19)
    A, W, b = (draw(g, *s, integer=True) for s in ((40, 32), (1, 32, 48), (1, 48)))
    offsets, _ = spans([10, 0, 25])
    got = gpu_lib.gemm_grouped(A.cuda(), W.cuda().expand(3, 32, 48), offsets.cuda(),
                               bias=b.cuda().expand(3, 48))
    assert torch.equal(got.cpu()[:35], (A @ W[0] + b)[:35])


def test_grouped_indexes_outside_are_not_followed(gpu_lib):
    """A row of A whose index is outside counts as zeros (not NaN, not 0 * x); a
    row of C whose index is outside is not written."""
    g = gen(20)
    rows, K, N = 90, 64, 64
    A, W = draw(g, rows, K, integer=True), draw(g, 2, K, N, integer=True)
    offsets, _ = spans([50, 40])
    ia, ic = torch.arange(rows).int(), torch.arange(rows).int()
    ia[3], ia[60], ia[89] = -1, rows, 2 ** 31 - 1
    ic[4], ic[49], ic[88] = -2 ** 31, rows, -1
    C = torch.full((rows, N), 7.0, device="cuda")
    H.say("grouped indexes outside")
    gpu_lib.gemm_grouped(A.cuda(), W.cuda(), offsets.cuda(), C, index_a=ia.cuda(),
                         index_c=ic.cuda())
    want = torch.cat([A[:50] @ W[0], A[50:] @ W[1]])
    want[[3, 60, 89]] = 0
    want[[4, 49, 88]] = 7
    assert torch.equal(C.cpu(), want)


def test_grouped_offsets_outside_or_falling(gpu_lib):
    """Offsets are taken into [0, rows]; a group that ends before it begins is
    empty; nothing outside C is written."""
    g = gen(21)
    rows, K, N = 70, 32, 40
    A, W = draw(g, rows, K, integer=True), draw(g, 4, K, N, integer=True)
    for off, want_groups in [([-5, 20, 20, 70, 1000], [(0, 20, 0), (20, 70, 2)]),
                             ([0, 30, 10, 10, 10], [(0, 30, 0)]),
                             ([2 ** 31 - 1, -2 ** 31, 5, 6, 7], [(0, 5, 1), (5, 6, 2), (6, 7, 3)])]:
        C, flat = H.sentinel_output(rows, N)
        H.say(f"grouped offsets {off}")
        gpu_lib.gemm_grouped(A.cuda(), W.cuda(), torch.tensor(off).int().cuda(), C)
        got = C.cpu()
        H.check_outside_untouched(flat, rows, N, N)
        want = torch.full((rows, N), float("nan"))
        for b, f, e in want_groups:
            want[b:f] = A[b:f] @ W[e]
        assert torch.equal(torch.nan_to_num(got, nan=9e9), torch.nan_to_num(want, nan=9e9)), off


def test_grouped_non_finite_rows_stay_in_their_row(gpu_lib):
    """NaN and Inf in one row of A reach that row of C only; NaN in another
    group's weights and in rows that no place names reach nothing."""
    g = gen(22)
    counts = [20, 5, 70]
    offsets, rows = spans(counts, 6)
    A, W = draw(g, rows, 100, integer=True), draw(g, 3, 100, 80, integer=True)
    A[7, 3], A[40, 99] = float("nan"), float("inf")
    A[95:] = float("nan")
    W[1] = float("nan")
    for trans in (False, True):
        Wd = (W.transpose(1, 2).contiguous() if trans else W).cuda()
        C = torch.zeros(rows, 80, device="cuda")
        gpu_lib.gemm_grouped(A.cuda(), Wd, offsets.cuda(), C, trans_b=trans)
        got = C.cpu()
        bad = torch.zeros(rows, dtype=torch.bool)
        bad[7], bad[20:25] = True, True
        assert bool(torch.isnan(got[bad]).all())
        assert bool((~torch.isfinite(got[40])).all())
        bad[40] = True
        want = torch.cat([A[:20] @ W[0], torch.zeros(5, 80), A[25:95] @ W[2], torch.zeros(6, 80)])
        assert torch.equal(got[~bad], want[~bad])


# ---- the gradient of the weights --------------------------------------------------

def wgrad_case(lib, counts, M, N, gather_a, gather_b, alpha, beta, integer, seed, pads=(0, 0, 0),
               shifts=(0, 0, 0), spare=3):
    g = gen(seed)
    offsets, rows = spans(counts, spare)
    G = len(counts)
    rows_a = max(1, rows // 2) if gather_a else rows + 2
    rows_b = rows + 4
    A, B = draw(g, rows_a, M, integer=integer), draw(g, rows_b, N, integer=integer)
    if not gather_a:
        A[rows - spare:] = float("nan")    # behind the last place: never used
    ia = torch.randint(0, rows_a, (rows,), generator=g).int() if gather_a else None
    ib = torch.randperm(rows_b, generator=g)[:rows].int() if gather_b else None
    C0 = draw(g, G, M, N, integer=integer)
    Cd = device(C0 if beta else torch.full_like(C0, float("nan")), pads[2], shifts[2])
    H.say(f"wgrad counts={counts[:8]} M={M} N={N} gather={gather_a},{gather_b} alpha={alpha} "
          f"beta={beta} int={integer} pads={pads} shifts={shifts}")
    lib.gemm_grouped_wgrad(device(A, pads[0], shifts[0]), device(B, pads[1], shifts[1]),
                           offsets.cuda(), Cd, alpha=alpha, beta=beta,
                           index_a=None if ia is None else ia.cuda(),
                           index_b=None if ib is None else ib.cuda())
    torch.cuda.synchronize()
    want, mag = torch.zeros(G, M, N).double(), torch.zeros(G, M, N).double()
    for e, (b, f) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        at = torch.arange(b, f)
        a = A[ia[b:f].long() if gather_a else at].double()
        c = B[ib[b:f].long() if gather_b else at].double()
        want[e] = alpha * (a.t() @ c)
        mag[e] = abs(alpha) * (a.abs().t() @ c.abs())
    if beta:
        want, mag = want + beta * C0.double(), mag + abs(beta) * C0.double().abs()
    check(Cd, want, mag, max(counts) + 4, integer, "wgrad")


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("integer", [True, False])
def test_wgrad_counts(gpu_lib, counts, integer):
    M, N = (36, 52) if counts in ("many", "most") else (96, 132)
    wgrad_case(gpu_lib, COUNTS[counts], M, N, True, True, 1.0, 0.0, integer, 31)
    wgrad_case(gpu_lib, COUNTS[counts], M, N, False, True, 0.5, -2.0, integer, 32)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 200), (200, 1), (8, 260), (260, 8), (16, 64),
                                 (64, 16), (33, 65), (129, 31), (300, 513), (512, 384)])
def test_wgrad_sizes(gpu_lib, M, N):
    for counts in ("few", "skewed", "long"):
        wgrad_case(gpu_lib, COUNTS[counts], M, N, False, False, 1.0, 0.0, True, 33)
        wgrad_case(gpu_lib, COUNTS[counts], M, N, True, False, 1.0, 1.0, False, 34)


@pytest.mark.parametrize("pads,shifts", [((4, 8, 4), (0, 0, 0)), ((1, 3, 5), (0, 0, 0)),
                                         ((0, 0, 0), (1, 2, 3)), ((2, 0, 1), (0, 3, 0))])
def test_wgrad_pitches_and_alignment(gpu_lib, pads, shifts):
    for counts in ("few", "skewed", "long"):
        for M, N in ((64, 128), (16, 96)):
            wgrad_case(gpu_lib, COUNTS[counts], M, N, True, True, 1.0, 1.0, True, 35, pads, shifts)


def test_wgrad_long_group(gpu_lib):
    """Few outputs and many rows: 20000 places in one group, both thin shapes."""
    for M, N in ((8, 512), (512, 8), (4, 4), (1, 300)):
        wgrad_case(gpu_lib, [20000, 3], M, N, True, False, 1.0, 0.0, True, 36)
        wgrad_case(gpu_lib, [3000, 0, 17000], M, N, False, True, 1.0, 0.0, False, 37)


@pytest.mark.parametrize("M,N", [(100, 140), (68, 512), (129, 67), (300, 257)])
def test_wgrad_slices(gpu_lib, M, N):
    """Few outputs and long groups: slices that end at, inside and before the
    group's last K-tile, groups shorter than their slices, and none at all."""
    for counts in ([5000, 0, 3], [2049], [0, 0, 4097, 31], [512] * 3, [640, 1, 639]):
        wgrad_case(gpu_lib, counts, M, N, True, True, 1.0, 0.0, True, 60)
        wgrad_case(gpu_lib, counts, M, N, False, True, 0.5, -2.0, True, 61)
        wgrad_case(gpu_lib, counts, M, N, True, False, -1.0, 1.0, False, 62, (1, 3, 5), (1, 0, 2))


def test_wgrad_indexes_outside_count_as_zeros(gpu_lib):
    g = gen(38)
    rows, M, N = 60, 64, 64
    A, B = draw(g, rows, M, integer=True), draw(g, rows, N, integer=True)
    B[5] = float("nan")   # multiplied by a row that counts as zeros elsewhere: named by nothing
    ia, ib = torch.arange(rows).int(), torch.arange(rows).int()
    ia[10], ia[59], ib[5], ib[30] = -1, rows, -7, 2 ** 31 - 1
    offsets, _ = spans([rows])
    H.say("wgrad indexes outside")
    got = gpu_lib.gemm_grouped_wgrad(A.cuda(), B.cuda(), offsets.cuda(), index_a=ia.cuda(),
                                     index_b=ib.cuda())
    keep = [i for i in range(rows) if i not in (5, 10, 30, 59)]
    assert torch.equal(got.cpu()[0], A[keep].t() @ B[keep])


def test_wgrad_of_ones_is_the_bias_gradient(gpu_lib):
    g = gen(39)
    offsets, rows = spans([0, 40, 3])
    dC = draw(g, rows, 77, integer=True)
    got = gpu_lib.gemm_grouped_wgrad(torch.ones(rows, 1, device="cuda"), dC.cuda(),
                                     offsets.cuda())
    want = torch.stack([torch.zeros(77), dC[:40].sum(0), dC[40:].sum(0)])
    assert torch.equal(got.cpu()[:, 0], want)


# ---- low-rank adapters ------------------------------------------------------------

def adapters_reference(X, W, down, up, scale, bias, offsets, order, trans):
    """(Y, H, and the sums of magnitudes of both) in 64 bits."""
    X, W, down, up, scale = (t.double() for t in (X, W, down, up, scale))
    if trans:
        W, down, up = W.t(), down.transpose(1, 2), up.transpose(1, 2)
    Y, MY = X @ W, X.abs() @ W.abs()
    if bias is not None:
        Y, MY = Y + bias.double(), MY + bias.double().abs()
    Hh = torch.full((order.numel(), down.shape[2]), float("nan")).double()
    MH = torch.ones_like(Hh)
    for e, (b, f) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        r = order[b:f].long()
        Hh[b:f] = scale[e] * (X[r] @ down[e])
        MH[b:f] = scale[e].abs() * (X[r].abs() @ down[e].abs())
        Y[r] += Hh[b:f] @ up[e]
        MY[r] += MH[b:f] @ up[e].abs()
    return Y, Hh, MY, MH


def adapters_data(M, N, K, R, adapters, trans, integer, seed, none=True):
    g = gen(seed)
    index = torch.randint(-1 if none else 0, adapters, (M,), generator=g).int()
    X = draw(g, M, K, integer=integer)
    W = draw(g, *((N, K) if trans else (K, N)), integer=integer)
    down = draw(g, adapters, *((R, K) if trans else (K, R)), integer=integer)
    up = draw(g, adapters, *((N, R) if trans else (R, N)), integer=integer)
    scale = torch.tensor([0.5, 2.0, -1.0, 1.0] * adapters)[:adapters]
    return index, X, W, down, up, scale, draw(g, N, integer=integer), draw(g, M, N, integer=integer)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K,R,adapters", [
    (1, 64, 48, 8, 1), (1, 33, 17, 3, 2), (5, 128, 256, 16, 3), (16, 200, 100, 4, 20),
    (32, 512, 384, 16, 8), (70, 65, 129, 64, 5), (300, 260, 192, 32, 4), (513, 96, 64, 1, 2),
    (200, 64, 1000, 24, 3), (40, 31, 40, 100, 3), (1000, 384, 256, 8, 3)])
def test_adapters(gpu_lib, M, N, K, R, adapters, trans):
    for integer in (True, False):
        index, X, W, down, up, scale, bias, _ = adapters_data(M, N, K, R, adapters, trans, integer,
                                                              41)
        H.say(f"adapters M={M} N={N} K={K} R={R} adapters={adapters} trans={trans} int={integer}")
        offsets, order, _ = gpu_lib.group_rows(index.cuda(), adapters)
        Hd = torch.full((M, R), float("nan"), device="cuda")
        Y, Hd = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down.cuda(), up.cuda(), offsets, order,
                                      H=Hd, trans=trans, scale=scale.cuda(), bias=bias.cuda())
        wy, wh, my, mh = adapters_reference(X, W, down, up, scale, bias, offsets.cpu(),
                                            order.cpu(), trans)
        used = int(offsets[-1])
        assert bool(torch.isnan(Hd[used:]).all()), "H behind the last place was written"
        check(Hd[:used], wh[:used], mh[:used], K + 2, integer, "H")
        check(Y, wy, my, K + R + 6, integer, "Y")


def test_adapters_without_scale_bias_or_adapters(gpu_lib):
    index, X, W, down, up, _, _, _ = adapters_data(50, 96, 64, 8, 3, False, True, 42)
    ones = torch.ones(3)
    offsets, order, _ = gpu_lib.group_rows(index.cuda(), 3)
    Y, _ = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down.cuda(), up.cuda(), offsets, order)
    want = adapters_reference(X, W, down, up, ones, None, offsets.cpu(), order.cpu(), False)[0]
    assert torch.equal(Y.cpu().double(), want)
    # no row has an adapter; no adapters; rank 0
    none = torch.full((50,), -1, dtype=torch.int32)
    offsets, order, _ = gpu_lib.group_rows(none.cuda(), 3)
    Y, _ = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down.cuda(), up.cuda(), offsets, order)
    assert torch.equal(Y.cpu(), X @ W)
    offsets, order, _ = gpu_lib.group_rows(none.cuda(), 0)
    Y, _ = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down[:0].cuda(), up[:0].cuda(), offsets,
                                 order)
    assert torch.equal(Y.cpu(), X @ W)
    offsets, order, _ = gpu_lib.group_rows(index.cuda(), 3)
    Y, _ = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down[:, :, :0].contiguous().cuda(),
                                 up[:, :0].contiguous().cuda(), offsets, order)
    assert torch.equal(Y.cpu(), X @ W)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K,R,adapters", [(1, 40, 24, 4, 2), (70, 65, 129, 8, 5),
                                              (300, 260, 192, 16, 4), (900, 96, 128, 32, 3)])
def test_adapters_gradients_against_the_formulas(gpu_lib, M, N, K, R, adapters, trans):
    """Whole numbers: exact.  G = s dY op(U)^T, dX = dY op(W)^T + G op(D)^T,
    dD = X^T G, dU = H^T dY over each adapter's rows."""
    index, X, W, down, up, scale, _, dY = adapters_data(M, N, K, R, adapters, trans, True, 43)
    if M * K * R > 10 ** 6:   # keep every sum below 2^24
        X, dY = X.clamp(-1, 1), dY.clamp(-1, 1)
        down, up, W = down.clamp(-1, 1), up.clamp(-1, 1), W.clamp(-1, 1)
    H.say(f"adapter gradients M={M} N={N} K={K} R={R} trans={trans}")
    offsets, order, _ = gpu_lib.group_rows(index.cuda(), adapters)
    args = [t.cuda() for t in (X, W, down, up)]
    _, Hd = gpu_lib.gemm_adapters(*args, offsets, order, trans=trans, scale=scale.cuda())
    dX, d_down, d_up = gpu_lib.gemm_adapters_grad(dY.cuda(), *args, offsets, order, Hd,
                                                  trans=trans, scale=scale.cuda())
    Xd, Wd, Dd, Ud, dYd = (t.double() for t in (X, W, down, up, dY))
    if trans:
        Wd, Dd, Ud = Wd.t(), Dd.transpose(1, 2), Ud.transpose(1, 2)
    wx, wd, wu = dYd @ Wd.t(), torch.zeros_like(Dd), torch.zeros_like(Ud)
    for e in range(adapters):
        r = torch.nonzero(index == e)[:, 0]
        s = float(scale[e])
        G = s * dYd[r] @ Ud[e].t()
        wx[r] += G @ Dd[e].t()
        wd[e] = Xd[r].t() @ G
        wu[e] = (s * Xd[r] @ Dd[e]).t() @ dYd[r]
    assert float(max(wd.abs().max(), wu.abs().max(), wx.abs().max())) < 2 ** 23
    if trans:
        wd, wu = wd.transpose(1, 2), wu.transpose(1, 2)
    for got, want, name in ((dX, wx, "dX"), (d_down, wd, "d_down"), (d_up, wu, "d_up")):
        check(got, want, None, 0, True, name)


def test_adapters_gradients_against_differences(gpu_lib):
    """The loss sum(dY * Y) is linear in X and in each factor alone, so a
    difference of whole-number losses is the gradient exactly."""
    index, X, W, down, up, scale, bias, dY = adapters_data(30, 20, 24, 4, 3, False, True, 44)
    offsets, order, _ = gpu_lib.group_rows(index.cuda(), 3)

    def forward(X, down, up):
        return gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down.cuda(), up.cuda(), offsets, order,
                                     scale=scale.cuda(), bias=bias.cuda())

    def loss(X, down, up):
        return float((forward(X, down, up)[0].cpu().double() * dY.double()).sum())

    Hd = forward(X, down, up)[1]
    grads = gpu_lib.gemm_adapters_grad(dY.cuda(), X.cuda(), W.cuda(), down.cuda(), up.cuda(),
                                       offsets, order, Hd, scale=scale.cuda())
    params = [X, down, up]
    g = gen(45)
    for which, grad in enumerate(grads):
        for _ in range(6):
            at = tuple(int(torch.randint(0, d, (1,), generator=g)) for d in params[which].shape)
            up_, dn_ = [t.clone() for t in params], [t.clone() for t in params]
            up_[which][at] += 1
            dn_[which][at] -= 1
            assert (loss(*up_) - loss(*dn_)) / 2 == float(grad[at]), (which, at)


# ---- the operators together ---------------------------------------------------------

def test_expert_layer_forward_and_backward(gpu_lib):
    """A sparse layer as a user runs it: choices ordered by expert, the up
    product with bias and ReLU on gathered tokens, the down product scattered to
    the choices' slots, the choices combined by their weights with
    gemm_batched, and every gradient, against the formulas in 64 bits."""
    T, top, G, D, F = 75, 3, 9, 40, 56
    g = gen(50)
    X = torch.randn(T, D, generator=g)
    W1, b1 = torch.randn(G, D, F, generator=g) * D ** -0.5, torch.randn(G, F, generator=g)
    W2 = torch.randn(G, F, D, generator=g) * F ** -0.5
    choice = torch.stack([torch.randperm(G, generator=g)[:top] for _ in range(T)])
    choice[torch.rand(T, top, generator=g) < 0.15] = -1
    weight = torch.rand(T, top, generator=g)
    dY = torch.randn(T, D, generator=g)
    Xd, W1d, b1d, W2d, wd, dYd = (t.cuda() for t in (X, W1, b1, W2, weight, dY))
    offsets, slot, token = gpu_lib.group_rows(choice.reshape(-1).int().cuda(), G, per_row=top)
    P = T * top
    h = gpu_lib.gemm_grouped(Xd, W1d, offsets, torch.zeros(P, F, device="cuda"), bias=b1d,
                             act=gpu_lib.ACT_RELU, index_a=token)
    y = gpu_lib.gemm_grouped(h, W2d, offsets, torch.zeros(P, D, device="cuda"), index_c=slot)
    Y = gpu_lib.gemm_batched(wd.view(T, 1, top), y.view(T, top, D)).view(T, D)
    # backward: to the slots, through the down product, ReLU and the up product
    dy = gpu_lib.gemm_batched(wd.view(T, top, 1), dYd.view(T, 1, D)).view(P, D)
    dw = gpu_lib.gemm_batched(y.view(T, top, D), dYd.view(T, D, 1)).view(T, top)
    dh = gpu_lib.gemm_grouped(dy, W2d, offsets, torch.zeros(P, F, device="cuda"), trans_b=True,
                              index_a=slot)
    dh = dh * (h > 0)
    dW2 = gpu_lib.gemm_grouped_wgrad(h, dy, offsets, index_b=slot)
    dW1 = gpu_lib.gemm_grouped_wgrad(Xd, dh, offsets, index_a=token)
    db1 = gpu_lib.gemm_grouped_wgrad(torch.ones(P, 1, device="cuda"), dh, offsets)[:, 0]
    dx = gpu_lib.gemm_grouped(dh, W1d, offsets, torch.zeros(P, D, device="cuda"), trans_b=True,
                              index_c=slot)
    ones = torch.ones(1, 1, top, device="cuda").expand(T, 1, top)
    dX = gpu_lib.gemm_batched(ones, dx.view(T, top, D)).view(T, D)
    # the same in 64 bits by autograd
    leaves = [t.double().requires_grad_() for t in (X, W1, b1, W2, weight)]
    x, w1, bb, w2, ww = leaves
    out = []
    for t in range(T):
        v = torch.zeros(D).double()
        for j in range(top):
            e = int(choice[t, j])
            if e >= 0:
                v = v + ww[t, j] * (torch.relu(x[t] @ w1[e] + bb[e]) @ w2[e])
        out.append(v)
    want = torch.stack(out)
    (want * dY.double()).sum().backward()
    # each path has fewer than 4 products in a row of at most T * top terms of
    # magnitude a few; (200 + terms) 2^-24 of the largest value covers them
    for got, ref, name in ((Y, want, "Y"), (dX, x.grad, "dX"), (dW1, w1.grad, "dW1"),
                           (db1, bb.grad, "db1"), (dW2, w2.grad, "dW2"), (dw, ww.grad, "dw")):
        ref = ref.detach()
        err = float((got.cpu().double() - ref).abs().max())
        assert err <= 425 * U * float(ref.abs().max()), (name, err)


# ---- streams, graphs, repeats --------------------------------------------------------

def together(lib, s):
    """Every operator once, on the state's tensors."""
    offsets, slot, token = lib.group_rows(s["index"], 6, per_row=2)
    h = lib.gemm_grouped(s["x"], s["w"], offsets, index_a=token, act=1, C=s["h"])
    lib.gemm_grouped_wgrad(s["x"], h, offsets, s["dw"], index_a=token)
    o2, order, _ = lib.group_rows(s["adapter"], 3)
    y, hh = lib.gemm_adapters(s["x"], s["wp"], s["down"], s["up"], o2, order, s["y"])
    dx, dd, du = lib.gemm_adapters_grad(s["y0"], s["x"], s["wp"], s["down"], s["up"], o2, order, hh)
    return [h, s["dw"], y, dx, dd, du]


def state(seed, T=60):
    g = gen(seed)
    f = lambda *sh: torch.randn(*sh, generator=g).cuda()
    s = {"x": f(T, 96), "w": f(6, 96, 160), "wp": f(96, 160), "down": f(3, 96, 8),
         "up": f(3, 8, 160), "y0": f(T, 160),
         "index": torch.randint(0, 6, (2 * T,), generator=g).int().cuda(),
         "adapter": torch.randint(0, 3, (T,), generator=g).int().cuda()}
    s["h"] = torch.zeros(2 * T, 160, device="cuda")
    s["dw"] = torch.zeros(6, 96, 160, device="cuda")
    s["y"] = torch.zeros(T, 160, device="cuda")
    return s


@pytest.mark.parametrize("T", [3, 60, 700])
def test_captured_graphs_replay_as_eager(gpu_lib, T):
    """Two graphs of all operators captured on one stream, replayed in turn with
    new inputs and eager work between the replays."""
    stream = torch.cuda.Stream()
    states = [state(60, T), state(61, T)]
    graphs, outs = [], []
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for s in states:
            together(gpu_lib, s)
    torch.cuda.synchronize()
    H.say(f"capture T={T}")
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(together(gpu_lib, s))
        graphs.append(graph)
    torch.cuda.synchronize()
    for rep in range(3):
        for i, s in enumerate(states):
            fresh = state(70 + 2 * rep + i, T)
            for k in s:
                s[k].copy_(fresh[k])
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs[i]]
            want = together(gpu_lib, fresh)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b), f"replay {rep} of graph {i} differs"


@pytest.mark.parametrize("T", [40, 700])
def test_two_streams_at_once(gpu_lib, T):
    """Calls on two streams overlap without sharing anything."""
    a, b = state(80, T), state(81, T)
    want = [[t.clone() for t in together(gpu_lib, s)] for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                got.append(together(gpu_lib, s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for p, q in zip(x, y):
                assert torch.equal(p, q)


# ---- sizes that take the larger tiles -----------------------------------------------

@pytest.mark.parametrize("K,N,pads", [(64, 1280, (0, 0, 0)), (35, 1301, (0, 0, 0)),
                                      (36, 1284, (0, 0, 1)), (33, 1280, (3, 0, 0))])
@pytest.mark.parametrize("trans", [False, True])
def test_grouped_many_tiles(gpu_lib, K, N, pads, trans):
    """Whole rounds of 128 x 128 tiles, the part-full round after them, and
    groups that end in a short tile; 16-byte and single-float copies."""
    counts = [3000, 0, 2500, 64, 1500, 129]
    grouped_case(gpu_lib, counts, K, N, trans, True, True, True, True, 51, pads)
    grouped_case(gpu_lib, counts, K, N, trans, False, False, False, False, 52, pads)


@pytest.mark.parametrize("M,N", [(512, 1024), (513, 1029)])
def test_wgrad_many_tiles(gpu_lib, M, N):
    counts = [300, 0, 17, 500, 64, 1, 90, 33, 0, 128, 40, 7, 256]
    wgrad_case(gpu_lib, counts, M, N, True, True, 1.0, 0.0, True, 53)
    wgrad_case(gpu_lib, counts, M, N, False, False, 0.5, -2.0, False, 54)


def test_wgrad_more_groups_than_a_wave(gpu_lib):
    """Groups beyond 64 are not ordered by size."""
    counts = [(11 * i) % 40 for i in range(100)]
    wgrad_case(gpu_lib, counts, 200, 260, True, False, 1.0, 0.0, True, 55)


def test_grouped_no_row_of_a_at_all(gpu_lib):
    """A without rows: every index is outside, every sum empty."""
    offsets, rows = spans([100, 50])
    index = torch.zeros(rows, dtype=torch.int32).cuda()
    b = torch.arange(300.).reshape(2, 150).cuda()
    for n in (150, 40):   # the tiles, and the kernel for few columns
        C = gpu_lib.gemm_grouped(torch.empty(0, 64, device="cuda"),
                                 torch.ones(2, 64, n, device="cuda"), offsets.cuda(),
                                 bias=b[:, :n], index_a=index)
        want = torch.cat([b[0, :n].expand(100, n), b[1, :n].expand(50, n)])
        assert torch.equal(C, want)


@pytest.mark.parametrize("M,N,K,R", [(30, 96, 64, 8), (200, 260, 256, 16), (700, 1280, 512, 32),
                                     (4000, 1300, 512, 32), (300, 96, 129, 5)])
@pytest.mark.parametrize("trans", [False, True])
def test_adapters_non_finite_factors_stay_with_their_rows(gpu_lib, M, N, K, R, trans):
    """An infinite or NaN factor of one adapter reaches the rows of that adapter
    only, though rows of others share their tiles."""
    index, X, W, down, up, scale, bias, _ = adapters_data(M, N, K, R, 3, trans, True, 46)
    good = adapters_data(M, N, K, R, 3, trans, True, 46)[3:5]
    up[1] = float("nan")
    up[2].view(-1)[5] = float("inf")
    down[2].view(-1)[3] = float("nan")
    H.say(f"adapters non-finite M={M} N={N} K={K} R={R} trans={trans}")
    offsets, order, _ = gpu_lib.group_rows(index.cuda(), 3)
    Y, _ = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down.cuda(), up.cuda(), offsets, order,
                                 trans=trans, scale=scale.cuda(), bias=bias.cuda())
    want = adapters_reference(X, W, *good, scale, bias, offsets.cpu(), order.cpu(), trans)[0]
    rows = index < 1
    assert torch.equal(Y.cpu()[rows].double(), want[rows])
    assert bool(torch.isnan(Y.cpu()[index == 1]).all())


@pytest.mark.parametrize("M,K,N,R", [(20, 64, 96, 8), (300, 128, 160, 16)])
@pytest.mark.parametrize("trans", [False, True])
def test_adapters_places_without_rows(gpu_lib, M, K, N, R, trans):
    """More places than rows, places of adapters whose row is outside X (their H
    is that of a row of zeros, no row of Y takes it), places before the first
    adapter and behind the last."""
    index, X, W, down, up, _, _, _ = adapters_data(M, N, K, R, 3, trans, True, 47)
    places = min(64, 2 * M) if M <= 64 else 2 * M
    order = torch.full((places,), -1, dtype=torch.int32)
    used = torch.randperm(M, generator=gen(48))[:M - 5].int()
    order[4:4 + len(used)] = used
    order[7], order[9], order[11] = M, -3, 2 ** 31 - 1
    order[1] = used[0]          # in no adapter: before the first place
    offsets = torch.tensor([4, 10, 10, 4 + len(used)]).int()
    H.say(f"adapters places without rows M={M} trans={trans}")
    Hd = torch.full((places, R), float("nan"), device="cuda")
    Y, Hd = gpu_lib.gemm_adapters(X.cuda(), W.cuda(), down.cuda(), up.cuda(), offsets.cuda(),
                                  order.cuda(), H=Hd, trans=trans)
    Wf, D, Uf = (W.t(), down.transpose(1, 2), up.transpose(1, 2)) if trans else (W, down, up)
    wy, wh = X @ Wf, torch.full((places, R), float("nan"))
    for g, (b, e) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        for i in range(b, e):
            r = int(order[i])
            wh[i] = X[r] @ D[g] if 0 <= r < M else 0
            if 0 <= r < M:
                wy[r] += wh[i] @ Uf[g]
    assert torch.equal(Y.cpu(), wy)
    assert torch.equal(torch.nan_to_num(Hd.cpu(), nan=9e9), torch.nan_to_num(wh, nan=9e9))


# the refused call enqueues nothing, so the captured graph is empty by design
@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_capture_without_workspace_is_refused(gpu_lib):
    """Adapters of few rows and thin gradients of long groups take the stream's
    workspace: without one a capturing stream cannot get it."""
    index, X, W, down, up, _, _, _ = [t.cuda() for t in
                                      adapters_data(8, 512, 2048, 8, 2, False, True, 49)]
    offsets, order, _ = gpu_lib.group_rows(index, 2)
    long, _ = spans([20000])
    A, B = torch.zeros(20000, 8, device="cuda"), torch.zeros(20000, 64, device="cuda")
    C = torch.empty(1, 8, 64, device="cuda")
    Y, Hh = torch.empty(8, 512, device="cuda"), torch.empty(8, 8, device="cuda")
    long = long.cuda()
    torch.cuda.synchronize()
    for call in (lambda: gpu_lib.gemm_adapters(X, W, down, up, offsets, order, Y, Hh),
                 lambda: gpu_lib.gemm_grouped_wgrad(A, B, long, C)):
        assert gpu_lib.gemm_f32_release_workspaces() == 0
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            with pytest.raises(gpu_lib.GemmError) as err:
                call()
        assert err.value.status == 6
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits(gpu_lib):
    """Weights, rows of A and rows of C further apart than 2^31 floats."""
    g = gen(56)
    far = 2 ** 31 + 64
    flat, out = (torch.empty(far + (1 << 20), device="cuda") for _ in range(2))
    for rows, K, N, trans in ((40, 64, 48, False), (40, 64, 48, True), (300, 64, 256, False),
                              (300, 64, 256, True), (300, 61, 131, False)):
        A, W = draw(g, 2, K, integer=True), draw(g, 2, *((N, K) if trans else (K, N)), integer=True)
        Wd = torch.as_strided(flat, W.shape, (far, W.shape[2], 1))
        Ad = torch.as_strided(flat, (2, K), (far, 1), 1 << 18)
        Wd.copy_(W)
        Ad.copy_(A)
        offsets, _ = spans([rows // 2, rows - rows // 2])
        index = torch.randint(0, 2, (rows,), generator=g).int()
        H.say(f"far operands rows={rows} K={K} N={N} trans={trans}")
        got = gpu_lib.gemm_grouped(Ad, Wd, offsets.cuda(), trans_b=trans, index_a=index.cuda())
        Wf = W.transpose(1, 2) if trans else W
        want = torch.cat([A[index[:rows // 2].long()] @ Wf[0], A[index[rows // 2:].long()] @ Wf[1]])
        assert torch.equal(got.cpu(), want)
        # the same rows as the operand of a gradient, and a far C
        B = draw(g, rows, N, integer=True)
        Cd = torch.as_strided(out, (2, K, N), (far, N, 1))
        gpu_lib.gemm_grouped_wgrad(Ad, B.cuda(), offsets.cuda(), Cd, index_a=index.cuda())
        for e, (b, f) in enumerate(((0, rows // 2), (rows // 2, rows))):
            assert torch.equal(Cd[e].cpu(), A[index[b:f].long()].t() @ B[b:f])
        Cr = torch.as_strided(out, (2, N), (far, 1))
        one, _ = spans([1, 1])
        gpu_lib.gemm_grouped(Ad, Wd, one.cuda(), Cr, trans_b=trans)
        assert torch.equal(Cr.cpu(), torch.stack([A[0] @ Wf[0], A[1] @ Wf[1]]))


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
@pytest.mark.parametrize("M,N", [(100, 140), (16, 2048)])
def test_sliced_wgrad_under_capture(gpu_lib, M, N):
    """Sums of slices need the stream's workspace: refused without one, and
    replayed with new inputs after a call has made it."""
    offsets = spans([3000, 0, 1500])[0].cuda()
    A, B = torch.zeros(4500, M, device="cuda"), torch.zeros(4500, N, device="cuda")
    C = torch.empty(3, M, N, device="cuda")
    torch.cuda.synchronize()
    assert gpu_lib.gemm_f32_release_workspaces() == 0
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with pytest.raises(gpu_lib.GemmError) as err:
            gpu_lib.gemm_grouped_wgrad(A, B, offsets, C)
    assert err.value.status == 6
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        gpu_lib.gemm_grouped_wgrad(A, B, offsets, C)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gpu_lib.gemm_grouped_wgrad(A, B, offsets, C)
    for seed in (63, 64, 65):
        r = gen(seed)
        a, b = draw(r, 4500, M, integer=True), draw(r, 4500, N, integer=True)
        A.copy_(a)
        B.copy_(b)
        C.fill_(float("nan"))
        torch.cuda.synchronize()
        H.say(f"sliced wgrad replay M={M} N={N} seed={seed}")
        g.replay()
        torch.cuda.synchronize()
        want = torch.stack([a[:3000].t() @ b[:3000], torch.zeros(M, N), a[3000:].t() @ b[3000:]])
        assert torch.equal(C.cpu(), want)
