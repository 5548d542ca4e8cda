"""GPU tests of the edges of the grouped products that every kernel has to keep
by itself: indexes outside, offsets outside or falling, operands beyond 32-bit
offsets, values that are not finite.  Each runs at sizes of each kernel
(test_grouped_routes_host.py asserts which kernel they take).

Inputs are whole numbers from -2 to 2, so that every partial sum is exact in
fp32 and results equal the 64-bit ones bit for bit.
"""
import pytest
import torch

from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def draw(g, *shape):
    return torch.randint(-2, 3, shape, generator=g).float()


def int32(*values):
    return torch.tensor(values, dtype=torch.int32)


# ---- the products --------------------------------------------------------------------

# kernel, layout of B: places of each group, K, N
PRODUCT = {
    ("rows", False): ([33, 0, 40, 20], 100, 200),
    ("rows", True): ([33, 0, 40, 20], 99, 201),
    ("mixed", False): ([700, 0, 1501, 799], 36, 1408),
    ("mixed", True): ([700, 0, 1501, 799], 36, 1402),
    ("64, 4 floats", False): ([100, 0, 500, 400], 36, 1024),
    ("64, 4 floats", True): ([100, 0, 500, 400], 36, 1021),
    ("64, 1 float", False): ([700, 0, 1501, 799], 35, 1601),
    ("128, 1 float", False): ([1700, 0, 2500, 800], 35, 1601),
    ("128, 1 float", True): ([4000, 0, 3001, 1999], 35, 1801),
}
KERNELS = pytest.mark.parametrize("kernel,trans", list(PRODUCT))


def product_case(kernel, trans, seed):
    counts, K, N = PRODUCT[kernel, trans]
    g = gen(seed)
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows = offsets[-1]
    H.say(f"product {kernel} trans={trans} rows={rows} K={K} N={N}")
    return g, offsets, rows, draw(g, rows, K), draw(g, len(counts), K, N), draw(g, len(counts), N)


def stored(W, trans):
    return (W.transpose(1, 2).contiguous() if trans else W).cuda()


@KERNELS
@pytest.mark.parametrize("update", [False, True])
def test_product_indexes_outside(gpu_lib, kernel, trans, update):
    """A row of A outside leaves the update of an empty sum, also opposite
    weights that are not finite; a row of C outside is not written."""
    g, offsets, rows, A, W, b = product_case(kernel, trans, 11)
    ia, ic = torch.arange(rows).int(), torch.randperm(rows, generator=g).int()
    gone = torch.randperm(rows, generator=g)
    no_a, no_c = gone[:rows // 3], gone[rows // 3:rows // 2]
    no_a = torch.cat([no_a, torch.arange(offsets[0], offsets[1])]).unique()   # all of group 0
    ia[no_a] = int32(-1, rows, 2 ** 31 - 1, -2 ** 31).repeat(len(no_a))[:len(no_a)]
    lost = ic[no_c].long()
    ic[no_c] = int32(-2 ** 31, -1, rows, 2 ** 31 - 1).repeat(len(no_c))[:len(no_c)]
    C0 = draw(g, rows, N := W.shape[2])
    Wd = W.clone()
    Wd[0] = INF
    Wd[0, :, ::2] = NAN
    C = C0.cuda()
    how = dict(alpha=0.5, beta=-2.0, bias=b.cuda(), act=1) if update else dict(bias=b.cuda())
    gpu_lib.gemm_grouped(A.cuda(), stored(Wd, trans), int32(*offsets).cuda(), C, trans_b=trans,
                         index_a=ia.cuda(), index_c=ic.cuda(), **how)
    A[no_a] = 0
    want = C0.clone()
    for e, (p, q) in enumerate(zip(offsets, offsets[1:])):
        named = [i for i in range(p, q) if 0 <= int(ic[i]) < rows]
        to = ic[named].long()
        v = A[named] @ (W[e] if e else torch.zeros_like(W[0]))
        v = 0.5 * v - 2 * C0[to] + b[e] if update else v + b[e]
        want[to] = v.clamp_min(0) if update else v
    assert torch.equal(want[lost], C0[lost])
    assert torch.equal(C.cpu(), want)


@KERNELS
def test_product_offsets_outside_or_falling(gpu_lib, kernel, trans):
    """Offsets are taken into [0, rows]; a group that ends before it begins is
    empty; what no place names stays as it was."""
    g, _, rows, A, W, _ = product_case(kernel, trans, 12)
    Ad, Wd, third = A.cuda(), stored(W, trans), rows // 3
    for off, groups in [
            ([-5, third, third, rows, 2 ** 31 - 1], [(0, third, 0), (third, rows, 2)]),
            ([0, rows - 3, 10, 10, 10], [(0, rows - 3, 0)]),
            ([2 ** 31 - 1, -2 ** 31, third, third + 1, rows],
             [(0, third, 1), (third, third + 1, 2), (third + 1, rows, 3)]),
            ([rows, rows, rows, rows, rows], [])]:
        C, flat = H.sentinel_output(rows, W.shape[2])
        gpu_lib.gemm_grouped(Ad, Wd, int32(*off).cuda(), C, trans_b=trans)
        got = C.cpu()
        H.check_outside_untouched(flat, rows, W.shape[2], W.shape[2])
        want = torch.full_like(got, NAN)
        for p, q, e in groups:
            want[p:q] = A[p:q] @ W[e]
        assert torch.equal(got.nan_to_num(nan=9e9), want.nan_to_num(nan=9e9)), off


@KERNELS
def test_product_without_rows_of_a(gpu_lib, kernel, trans):
    """A without rows: every index is outside, every sum empty."""
    _, offsets, rows, A, W, b = product_case(kernel, trans, 13)
    got = gpu_lib.gemm_grouped(torch.empty(0, A.shape[1], device="cuda"), stored(W, trans),
                               int32(*offsets).cuda(), trans_b=trans, bias=b.cuda(),
                               index_a=torch.zeros(rows, dtype=torch.int32).cuda())
    for e, (p, q) in enumerate(zip(offsets, offsets[1:])):
        assert torch.equal(got[p:q].cpu(), b[e].expand(q - p, -1)), e


@KERNELS
def test_product_not_finite_stays_in_its_row(gpu_lib, kernel, trans):
    """NaN and Inf in a row of A reach that row of C only, NaN in a group's
    weights the rows of that group only."""
    _, offsets, rows, A, W, _ = product_case(kernel, trans, 14)
    W[0] = NAN
    first, last = offsets[2], offsets[3] - 1
    A[first, 3], A[last, -1] = NAN, INF
    got = gpu_lib.gemm_grouped(A.cuda(), stored(W, trans), int32(*offsets).cuda(),
                               trans_b=trans).cpu()
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[:offsets[1]] = bad[first] = True
    assert bool(got[bad].isnan().all())
    assert bool((~got[last].isfinite()).all())
    bad[last] = True
    for e in (2, 3):
        at = torch.arange(offsets[e], offsets[e + 1])
        at = at[~bad[at]]
        assert torch.equal(got[at], A[at] @ W[e]), e


FAR = 2 ** 31 + 64


@pytest.fixture(scope="module")
def far_memory():
    """Three buffers whose ends are more than 2^31 floats from their starts."""
    yield [torch.empty(FAR + (1 << 25), device="cuda") for _ in range(3)]
    torch.cuda.empty_cache()


def spread(flat, x, single):
    """x laid out over flat so that its last row (of one matrix) or its last
    matrix starts beyond 2^31 floats; single: at a pitch that 16 bytes do not fit."""
    n = x.shape[0] - 1
    pitch = (FAR + n - 1) // n
    pitch += (1 if single else 0) - pitch % 4 + 4
    assert n * pitch + x[0].numel() <= flat.numel() and n * pitch > 2 ** 31
    inner = () if x.dim() == 2 else (x.shape[2],)
    view = torch.as_strided(flat, x.shape, (pitch, *inner, 1))
    view.copy_(x)
    return view


@KERNELS
def test_product_operands_beyond_32_bits(gpu_lib, far_memory, kernel, trans):
    g, offsets, rows, A, W, b = product_case(kernel, trans, 15)
    single = "1 float" in kernel
    ia, ic = (torch.randperm(rows, generator=g).int() for _ in range(2))
    C = spread(far_memory[2], torch.zeros(rows, W.shape[2]), single)
    gpu_lib.gemm_grouped(spread(far_memory[0], A, single),
                         spread(far_memory[1], stored(W, trans), single), int32(*offsets).cuda(),
                         C, trans_b=trans, beta=1.0, bias=b.cuda(), index_a=ia.cuda(),
                         index_c=ic.cuda())
    got = C.cpu()
    for e, (p, q) in enumerate(zip(offsets, offsets[1:])):
        assert torch.equal(got[ic[p:q].long()], A[ia[p:q].long()] @ W[e] + b[e]), e


# ---- the gradient of the weights ---------------------------------------------------

# kernel: places of each group, M, N (the sizes with 4-float copies are multiples of 4)
GRADIENT = {
    "thin": ([40, 0, 30], 16, 96),
    "thin, slices": ([3000, 0, 70], 96, 16),
    "64, 4 floats": ([70, 0, 61], 100, 140),
    "64, 1 float": ([70, 0, 61], 101, 139),
    "64, 4 floats, slices": ([1500, 0, 600], 100, 140),
    "64, 1 float, slices": ([1500, 0, 600], 101, 139),
    "128, 4 floats": ([33 * (e % 3) for e in range(32)], 512, 512),
    "128, 1 float": ([33 * (e % 3) for e in range(32)], 509, 511),
}


def gradient_case(kernel, seed):
    counts, M, N = GRADIENT[kernel]
    g = gen(seed)
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows = offsets[-1]
    H.say(f"gradient {kernel} rows={rows} M={M} N={N}")
    return g, offsets, rows, draw(g, rows, M), draw(g, rows, N)


@pytest.mark.parametrize("kernel", list(GRADIENT))
@pytest.mark.parametrize("bad", [NAN, INF])
def test_gradient_places_outside_add_nothing(gpu_lib, kernel, bad):
    """A place whose row of A is outside adds nothing, also opposite a row of B
    that is not finite, and the other way round."""
    g, offsets, rows, A, B = gradient_case(kernel, 1)
    ia, ib = torch.arange(rows).int(), torch.arange(rows).int()
    drop = torch.randperm(rows, generator=g)[:rows // 3]
    for n, i in enumerate(drop.tolist()):
        (ia if n % 2 else ib)[i] = (-1, rows, 2 ** 31 - 1, -2 ** 31)[n // 2 % 4]
        (B if n % 2 else A)[i] = bad
    got = gpu_lib.gemm_grouped_wgrad(A.cuda(), B.cuda(), int32(*offsets).cuda(),
                                     index_a=ia.cuda(), index_b=ib.cuda()).cpu()
    A[drop], B[drop] = 0, 0
    for e, (b, f) in enumerate(zip(offsets, offsets[1:])):
        assert torch.equal(got[e], A[b:f].t() @ B[b:f]), e


@pytest.mark.parametrize("kernel", list(GRADIENT))
def test_gradient_offsets_outside_or_falling(gpu_lib, kernel):
    """Offsets are taken into [0, rows]; a group that ends before it begins is
    empty and gets the update of an empty sum."""
    g, offsets, rows, A, B = gradient_case(kernel, 2)
    G, third = len(offsets) - 1, rows // 3
    C0 = draw(g, G, A.shape[1], B.shape[1])
    for head in ([-5, third, 10, 2 ** 31 - 1], [rows, -2 ** 31, third, rows],
                 [2 ** 31 - 1, 7, 7, third]):
        off = head + [2 * third] * (G + 1 - len(head))
        C = C0.cuda()
        gpu_lib.gemm_grouped_wgrad(A.cuda(), B.cuda(), int32(*off).cuda(), C, beta=1.0)
        got = C.cpu()
        for e, (b, f) in enumerate(zip(off, off[1:])):
            b, f = max(0, min(b, rows)), max(0, min(f, rows))
            want = C0[e] + A[b:f].t() @ B[b:f] if f > b else C0[e]
            assert torch.equal(got[e], want), (head, e)


@pytest.mark.parametrize("kernel", list(GRADIENT))
@pytest.mark.parametrize("empty", ["A", "B"])
def test_gradient_without_rows(gpu_lib, kernel, empty):
    """A or B without rows: every place is outside, every sum empty."""
    _, offsets, rows, A, B = gradient_case(kernel, 3)
    none, there = torch.zeros(rows, dtype=torch.int32), torch.arange(rows).int()
    ia, ib = (none, there) if empty == "A" else (there, none)
    got = gpu_lib.gemm_grouped_wgrad((A[:0] if empty == "A" else A).cuda(),
                                     (B[:0] if empty == "B" else B).cuda(),
                                     int32(*offsets).cuda(), index_a=ia.cuda(), index_b=ib.cuda())
    assert bool((got == 0).all())


@pytest.mark.parametrize("kernel", list(GRADIENT))
def test_gradient_not_finite_stays_in_its_group(gpu_lib, kernel):
    _, offsets, rows, A, B = gradient_case(kernel, 4)
    last = len(offsets) - 2
    A[offsets[last] - 1, 5] = NAN       # the last place of a group before the last one
    hit = max(e for e in range(last) if offsets[e + 1] == offsets[last] and
              offsets[e] < offsets[e + 1])
    got = gpu_lib.gemm_grouped_wgrad(A.cuda(), B.cuda(), int32(*offsets).cuda()).cpu()
    for e, (b, f) in enumerate(zip(offsets, offsets[1:])):
        want = A[b:f].nan_to_num(nan=0.0).t() @ B[b:f]
        if e == hit:
            assert bool(got[e, 5].isnan().all())
            want[5] = got[e][5] = 0
        assert torch.equal(got[e], want), e


@pytest.mark.parametrize("kernel", list(GRADIENT))
def test_gradient_operands_beyond_32_bits(gpu_lib, far_memory, kernel):
    g, offsets, rows, A, B = gradient_case(kernel, 5)
    single = "1 float" in kernel
    ia, ib = (torch.randperm(rows, generator=g).int() for _ in range(2))
    C = spread(far_memory[2], draw(g, len(offsets) - 1, A.shape[1], B.shape[1]), single)
    C0 = C.cpu()
    gpu_lib.gemm_grouped_wgrad(spread(far_memory[0], A, single), spread(far_memory[1], B, single),
                               int32(*offsets).cuda(), C, beta=1.0, index_a=ia.cuda(),
                               index_b=ib.cuda())
    got = C.cpu()
    for e, (b, f) in enumerate(zip(offsets, offsets[1:])):
        want = C0[e] + A[ia[b:f].long()].t() @ B[ib[b:f].long()]
        assert torch.equal(got[e], want), e
