"""GPU tests of the products with 4-bit weights (``gemm_f32_q4``,
``gemm_f32_q4_grouped``) against their definition in 64 bits.

Gates.  Whole-number inputs and scales that are powers of two: every partial sum is
exact in fp32, so the result equals the 64-bit one bit for bit.  General inputs: the
products are exact; a sum of K terms, of the groups' sums times their scales (a
product each) and of the parts of K that run apart (at most 64), and the update of
four operations are off by at most (K + 2 groups + 72) 2^-24 of the sum of
magnitudes, in any order.
"""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding, q4
from tests import gpu_helpers as H
from tests.test_gpu_grouped import device, gen, spans

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INT, E2M1 = binding.Q4_INT, binding.Q4_E2M1
KINDS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e8m0": torch.uint8}


def weights(g, N, K, group, form, kind, lead=(), integer=False):
    """codes, scale, zero on the CPU and the 64-bit weights they stand for."""
    along = (K + group - 1) // group
    codes = torch.randint(0, 16, (*lead, N, K), generator=g)
    fmt = E2M1 if form == "e2m1" else INT
    if kind == "e8m0":
        scale = torch.randint(125, 130, (*lead, N, along), generator=g).to(torch.uint8)
    elif integer:
        scale = 2.0 ** torch.randint(-1, 2, (*lead, N, along), generator=g).to(torch.float32)
        scale = scale.to(KINDS[kind])
    else:
        scale = (torch.rand(*lead, N, along, generator=g) + 0.25).to(KINDS[kind])
    zero = None
    if form == "zeros":
        zero = torch.randint(0, 16, (*lead, N, along), generator=g).to(torch.uint8)
    packed = q4.pack(codes)
    if K % 2:   # the half that is no weight's may hold anything
        packed[..., -1] |= 0xd0
    W = q4.dequantize(packed, scale, K, zero=zero, group=group, format=fmt, dtype=torch.float64)
    return packed, scale, zero, W


def on_device(t, pad=0, shift=0):
    """A tensor of bytes or scales with padded rows and a shifted start."""
    if t is None:
        return None
    *lead, rows, cols = t.shape
    n = 1
    for d in lead:
        n *= d
    pitch = cols + pad
    flat = torch.full((n * rows * pitch + shift + 8,), 0x6b, dtype=torch.uint8)
    if t.dtype != torch.uint8:
        flat = torch.full((n * rows * pitch + shift + 8,), float("nan")).to(t.dtype)
    torch.as_strided(flat, (n, rows, cols), (rows * pitch, pitch, 1), shift).copy_(
        t.reshape(n, rows, cols))
    return torch.as_strided(flat.cuda(), tuple(lead) + (rows, cols),
                            (rows * pitch,) * len(lead) + (pitch, 1), shift)


def check(got, want, mag, K, group, integer, what):
    got = got.cpu().double()
    if integer:
        assert torch.equal(got, want), f"{what}: {(got != want).sum()} of {got.numel()} differ"
    else:
        ops = K + 2 * ((K + group - 1) // group) + 72
        err = (got - want).abs()
        assert bool((err <= ops * U * mag).all()), \
            f"{what}: off by {float((err / mag.clamp_min(1e-30)).max()) / U:.1f} of {ops} steps"


def dense(M, N, K, form="symmetric", kind="f32", group=128, integer=False, alpha=1.0, beta=0.0,
          bias=False, act=0, pad=0, shift=0):
    H.say(f"q4 {M}x{N}x{K} {form} {kind} group={group} int={integer} alpha={alpha} beta={beta} "
          f"bias={bias} act={act} pad={pad} shift={shift}")
    g = gen(M * 7 + N * 3 + K)
    draw = ((lambda *s: torch.randint(-2, 3, s, generator=g).float()) if integer else
            (lambda *s: torch.randn(*s, generator=g)))
    a, c0, bv = draw(M, K), draw(M, N), draw(N)
    packed, scale, zero, W = weights(g, N, K, group, form, kind, integer=integer)
    C = device(c0 if beta else torch.full_like(c0, float("nan")), pad, shift)
    got = binding.gemm_q4(device(a, pad, shift), on_device(packed, pad, shift),
                          on_device(scale, pad, shift), C, zero=on_device(zero, pad, shift),
                          group=group, format=E2M1 if form == "e2m1" else INT, alpha=alpha,
                          beta=beta, bias=bv.cuda() if bias else None, act=act)
    torch.cuda.synchronize()
    ad = a.double()
    want = alpha * (ad @ W.t()) + beta * c0.double() + (bv.double() if bias else 0)
    mag = abs(alpha) * (ad.abs() @ W.abs().t()) + abs(beta) * c0.double().abs() + \
        (bv.double().abs() if bias else 0)
    if act:
        want = want.clamp_min(0)
    check(got, want, mag, K, group, integer, f"{M}x{N}x{K}")
    if pad:
        flat = torch.as_strided(got, (M, N + pad), (N + pad, 1), shift).cpu()
        assert bool(flat[:, N:].isnan().all())
    return got


@pytest.mark.parametrize("M", [1, 2, 3, 5, 6, 7, 10, 11, 15, 16, 17, 20, 21, 33, 64, 65, 100, 130,
                               200, 257])
@pytest.mark.parametrize("form", ["symmetric", "zeros", "e2m1"])
def test_rows(gpu_lib, M, form):
    dense(M, 70, 300, form, integer=True)
    dense(M, 70, 300, form, group=32)


@pytest.mark.parametrize("K", [1, 2, 3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 255, 256, 300,
                               1023, 1024, 1025, 2047, 2050, 4100])
@pytest.mark.parametrize("form", ["symmetric", "e2m1"])
def test_depths(gpu_lib, K, form):
    for M in (1, 7, 40, 150):
        dense(M, 33, K, form, integer=True, group=64)
        dense(M, 33, K, form, group=32)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 256,
                               257, 1000])
def test_widths(gpu_lib, N):
    for M in (1, 8, 33, 140):
        dense(M, N, 130, "zeros", integer=True, group=32)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("form", ["symmetric", "zeros", "e2m1"])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 1 << 40])
def test_scales_and_groups(gpu_lib, kind, form, group):
    for M in (3, 9, 130):
        dense(M, 50, 520, form, kind, group=group, integer=True)
    dense(70, 50, 520, form, kind, group=group)


@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 1), (4, 4), (16, 3), (0, 1)])
@pytest.mark.parametrize("form", ["zeros", "e2m1"])
def test_pitches_and_alignment(gpu_lib, pad, shift, form):
    for M in (1, 12, 70, 140):
        for kind in ("f32", "f16", "e8m0"):
            dense(M, 36, 200, form, kind, group=64, integer=True, pad=pad, shift=shift)


@pytest.mark.parametrize("alpha,beta,bias,act", [(0.5, 0.0, False, 0), (1.0, 1.0, False, 0),
                                                (-2.0, 0.5, True, 1), (0.0, 0.0, True, 1),
                                                (1.0, 0.0, True, 0)])
def test_updates(gpu_lib, alpha, beta, bias, act):
    for M in (1, 14, 90):
        dense(M, 41, 96, "symmetric", integer=True, alpha=alpha, beta=beta, bias=bias, act=act)
        dense(M, 41, 96, "zeros", alpha=alpha, beta=beta, bias=bias, act=act)


def test_empty_sum(gpu_lib):
    H.say("q4 K=0")
    codes, scale = torch.zeros(5, 0, dtype=torch.uint8).cuda(), torch.zeros(5, 0).cuda()
    bias = torch.arange(5.0).cuda() - 2
    for M in (1, 20, 200):
        got = binding.gemm_q4(torch.zeros(M, 0).cuda(), codes, scale, bias=bias, act=1)
        assert torch.equal(got, bias.clamp_min(0).expand(M, 5))


def test_zero_points_of_a_whole_byte(gpu_lib):
    """A zero point up to 255 is taken as it is."""
    for M in (2, 50, 150):
        H.say(f"q4 zero points of a byte M={M}")
        g = gen(M)
        a = torch.randint(-2, 3, (M, 200), generator=g).float()
        packed, scale, zero, _ = weights(g, 40, 200, 32, "zeros", "f32", integer=True)
        zero = torch.randint(0, 256, zero.shape, generator=g).to(torch.uint8)
        W = q4.dequantize(packed, scale, 200, zero=zero, group=32, dtype=torch.float64)
        got = binding.gemm_q4(a.cuda(), packed.cuda(), scale.cuda(), zero=zero.cuda(), group=32)
        assert torch.equal(got.cpu().double(), a.double() @ W.t())


@pytest.mark.parametrize("M", [1, 4, 9, 20, 64, 130, 300])
@pytest.mark.parametrize("form", ["symmetric", "e2m1"])
def test_values_that_are_not_finite(gpu_lib, M, form):
    """Infinities and NaN of A give what the formula gives, in their own row only; a
    scale that is not finite reaches its own column only."""
    H.say(f"q4 not finite M={M} {form}")
    g = gen(M)
    N, K = 40, 200
    a = torch.randint(-2, 3, (M, K), generator=g).float()
    packed, scale, zero, W = weights(g, N, K, 32, form, "f32", integer=True)
    a[0, 3] = float("inf")
    if M > 1:
        a[1, 150] = float("nan")
    if M > 3:
        a[2, 40] = -float("inf")
        a[3, 41] = float("inf")
        a[3, 42] = float("-inf")
    tiny = torch.tensor([0x7f800001], dtype=torch.int32).view(torch.float32)   # NaN by its low bits
    if M > 8:
        a[8, 0] = tiny[0]
    scale[7, 2] = float("inf")
    scale[8, 1] = float("nan")
    W = q4.dequantize(packed, scale, K, zero=zero, group=32,
                      format=E2M1 if form == "e2m1" else INT, dtype=torch.float64)
    got = binding.gemm_q4(a.cuda(), packed.cuda(), scale.cuda(), group=32,
                          format=E2M1 if form == "e2m1" else INT).cpu().double()
    want = a.double() @ W.t()
    finite = torch.isfinite(want)
    assert torch.equal(finite, torch.isfinite(got))
    assert torch.equal(got[finite], want[finite])
    # rows of one infinity: its sign, or NaN where the weight is 0 (columns of finite scales)
    columns = [n for n in range(N) if n not in (7, 8)]
    for r in (0, 2) if M > 3 else (0,):
        assert torch.equal(got[r, columns].isnan(), want[r, columns].isnan())
        both = ~want[r, columns].isnan()
        assert torch.equal(got[r, columns][both], want[r, columns][both])


def test_large_and_small_values(gpu_lib):
    """Values near the largest float and near the smallest normal one keep all their
    bits; sums of single products are exact."""
    H.say("q4 extreme values")
    x = torch.tensor([1.0 + 2.0 ** -23, 3.4e38 / 16, -1.1754944e-38 * 2.0 ** 17, 1e-30, -123456.789])
    a = torch.diag(x)
    codes = torch.full((6, 5), 9)                       # weight 1
    for M in (5, 140):
        A = torch.zeros(M, 5)
        A[:5] = a
        got = binding.gemm_q4(A.cuda(), q4.pack(codes).cuda(), torch.ones(6, 1).cuda(), group=32)
        assert torch.equal(got[:5].cpu(), x[:, None].expand(5, 6))


# rows x columns that reach each kernel (test_q4_routes_host.py asks the rules)
KERNELS = {"few": (10, 1000), "32x32": (60, 4000), "32x64": (126, 4090), "64x64": (250, 4090),
           "64x128": (500, 4090), "128x128": (1000, 4090), "256x128": (2000, 4090),
           "256x192": (4000, 2990), "256x256": (4000, 4090)}


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("form", ["symmetric", "zeros", "e2m1"])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_every_kernel(gpu_lib, kernel, form, kind):
    """Sums exact, K with whole steps for all, some and none of the waves that share it,
    and a rest."""
    M, N = KERNELS[kernel]
    for K in ((640, 515) if kernel == "few" else (1, 32, 203)):
        dense(M, N, K, form, kind, group=32, integer=True)
    dense(M, N, 640 if kernel == "few" else 160, form, kind, group=64, pad=3, shift=1, beta=0.5,
          bias=True, act=1)


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_smallest_and_largest_powers(gpu_lib, kernel):
    """e8m0 scales from the subnormal 2^-127 to the last that keeps every weight finite."""
    M, N = KERNELS[kernel]
    K = 640 if kernel == "few" else 64
    g = gen(M)
    a = torch.randint(-2, 3, (M, K), generator=g).float()
    packed = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    for fmt, most in ((INT, 251), (E2M1, 252)):
        ones = torch.full((N, K // 32), 127, dtype=torch.uint8)
        W = q4.dequantize(packed, ones, K, group=32, format=fmt).double()
        want = a.double() @ W.t()
        for e, size in ((0, 2.0 ** 100), (1, 2.0 ** 100), (127, 1.0), (most, 2.0 ** -40)):
            H.say(f"q4 powers {kernel} format={fmt} e={e}")
            got = binding.gemm_q4((a * size).cuda(), packed.cuda(),
                                  torch.full_like(ones, e).cuda(), group=32, format=fmt)
            assert torch.equal(got.cpu().double(), want * size * 2.0 ** (e - 127))


# rows, columns, K of the kernel for few rows: its row tiles of each size, one and more of
# them, all and some of its waves along K, K in one pass and in several
FEW = [(M, N, K) for M in (1, 4, 5, 8, 9, 12) for N, K in ((1000, 2100), (8192, 1031),
                                                           (33, 16400), (28672, 1031))]
FEW += [(M, N, K) for M in (13, 16) for N, K in ((1000, 2100), (4096, 1000), (28672, 1031))]
FEW += [(17, 28672, 515), (17, 1000, 2100), (30, 1000, 640), (40, 300, 2100), (150, 16, 4096)]


@pytest.mark.parametrize("M,N,K", FEW)
def test_few_rows(gpu_lib, M, N, K):
    dense(M, N, K, "zeros", "f16", group=128)
    dense(M, N, K, "e2m1", "e8m0", group=32, beta=0.5, bias=True, pad=5, shift=3)


GROUPS = {"one": [1], "few": [0, 3, 0, 1, 17, 0], "even": [16, 16, 16, 16],
          "skewed": [0, 130, 1, 64, 65, 0, 300, 7], "many": [(7 * i) % 5 for i in range(150)],
          "long": [400, 500, 333]}


def grouped(counts, K, N, form, kind="f32", group=64, integer=True, spare=0, gather=True,
            scatter=True, bias=True, act=1, beta=0.0, pad=0, shift=0):
    H.say(f"q4 grouped {counts[:9]} {K}x{N} {form} {kind} group={group} gather={gather} "
          f"scatter={scatter} pad={pad} shift={shift}")
    offsets, rows = spans(counts, spare)
    g = gen(K + N + rows)
    draw = ((lambda *s: torch.randint(-2, 3, s, generator=g).float()) if integer else
            (lambda *s: torch.randn(*s, generator=g)))
    G = len(counts)
    rows_a, rows_c = (rows + 3 if gather else rows), (rows + 5 if scatter else rows)
    a, c0, bv = draw(rows_a, K), draw(rows_c, N), draw(G, N)
    packed, scale, zero, W = weights(g, N, K, group, form, kind, lead=(G,), integer=integer)
    ia = torch.randint(0, rows_a, (rows,), generator=g) if gather else torch.arange(rows)
    ic = torch.randperm(rows_c, generator=g)[:rows] if scatter else torch.arange(rows)
    if gather and rows > 8:     # rows outside A: an empty sum
        ia[2], ia[5] = -1, rows_a
    if scatter and rows > 8:    # rows outside C: not written
        ic[3], ic[7] = -1, rows_c
    C = device(c0, pad, shift)
    got = binding.gemm_q4_grouped(
        device(a, pad, shift), on_device(packed, pad, shift), on_device(scale, pad, shift),
        offsets.cuda(), C, zero=on_device(zero, pad, shift), group=group,
        format=E2M1 if form == "e2m1" else INT, beta=beta, bias=bv.cuda() if bias else None,
        act=act, index_a=ia.int().cuda() if gather else None,
        index_c=ic.int().cuda() if scatter else None)
    torch.cuda.synchronize()
    want, mag = c0.double().clone(), torch.zeros(rows_c, N, dtype=torch.float64)
    o = offsets.tolist()
    for e in range(G):
        places = torch.arange(o[e], o[e + 1])
        places = places[(ic[places] >= 0) & (ic[places] < rows_c)]
        if not len(places):
            continue
        read, to = ia[places], ic[places]
        x = a[read.clamp(0, rows_a - 1)].double()
        x[(read < 0) | (read >= rows_a)] = 0
        old = c0[to].double()
        v = x @ W[e].t() + beta * old + (bv[e].double() if bias else 0)
        mag[to] = x.abs() @ W[e].abs().t() + abs(beta) * old.abs() + \
            (bv[e].double().abs() if bias else 0)
        want[to] = v.clamp_min(0) if act else v
    check(got, want, mag, K, group, integer, str(counts[:9]))
    if pad:
        flat = torch.as_strided(got, (rows_c, N + pad), (N + pad, 1), shift).cpu()
        assert bool(flat[:, N:].isnan().all())


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("form", ["symmetric", "zeros", "e2m1"])
@pytest.mark.parametrize("K,N", [(64, 48), (131, 37)])
def test_grouped(gpu_lib, name, form, K, N):
    grouped(GROUPS[name], K, N, form, spare=4)
    grouped(GROUPS[name], K, N, form, group=32, integer=False, gather=False, scatter=False,
            bias=False, act=0)


# uneven groups whose sizes reach each tile: (counts, N)
WIDE = {"few": ([3, 0, 9, 20, 1, 8], 700), "32x32": ([40, 7, 0, 33], 1000),
        "32x64": ([70, 33, 0, 20], 2000), "64x64": ([130, 64, 0, 40], 2900),
        "64x128": ([300, 65, 7, 64], 4000), "128x128": ([500, 129, 3, 128], 4000),
        "256x128": ([1100, 257, 3, 400], 4000),
        "256x192": ([1500, 300, 0, 1100, 900, 1400, 7, 2900], 1000),
        "256x256": ([1500, 257, 3, 2000], 4000)}


@pytest.mark.parametrize("kernel", list(WIDE))
@pytest.mark.parametrize("form,kind", [("symmetric", "bf16"), ("e2m1", "e8m0")])
def test_grouped_in_every_kernel(gpu_lib, kernel, form, kind):
    counts, N = WIDE[kernel]
    grouped(counts, 515 if kernel == "few" else 67, N, form, kind, group=32, spare=3)


@pytest.mark.parametrize("pad,shift", [(3, 1), (8, 4)])
def test_grouped_pitches(gpu_lib, pad, shift):
    for name in ("skewed", "few"):
        grouped(GROUPS[name], 200, 70, "zeros", "f16", pad=pad, shift=shift, beta=0.5)
        grouped(GROUPS[name], 256, 64, "e2m1", "e8m0", group=32, pad=pad, shift=shift)


def test_grouped_offsets_that_leave_the_places(gpu_lib):
    """Offsets are taken into [0, rows]; a group that ends before it begins is empty;
    rows behind the last place stay as they were."""
    H.say("q4 grouped odd offsets")
    g = gen(1)
    K, N, rows = 96, 40, 30
    a = torch.randint(-2, 3, (rows, K), generator=g).float()
    packed, scale, _, W = weights(g, N, K, 32, "symmetric", "f32", lead=(3,), integer=True)
    for off, span in (([-5, 10, 20, 99], [(0, 10), (10, 20), (20, 30)]),
                      ([0, 0, 0, 7], [(0, 0), (0, 0), (0, 7)]),
                      ([4, 12, 12, 20], [(4, 12), (12, 12), (12, 20)])):
        c = torch.full((rows, N), 7.0, device="cuda")
        binding.gemm_q4_grouped(a.cuda(), packed.cuda(), scale.cuda(),
                                torch.tensor(off, dtype=torch.int32).cuda(), c, group=32)
        want = torch.full((rows, N), 7.0, dtype=torch.float64)
        for e, (b, t) in enumerate(span):
            want[b:t] = a[b:t].double() @ W[e].t()
        assert torch.equal(c.cpu().double(), want)


def test_rows_outside_meet_weights_that_are_not_finite(gpu_lib):
    """A row of A outside its matrix leaves an empty sum whatever the weights hold."""
    for rows in (6, 200):
        H.say(f"q4 rows outside, scales not finite, rows={rows}")
        g = gen(2)
        packed, scale, _, _ = weights(g, 40, 96, 32, "symmetric", "f32", integer=True)
        scale[:] = float("nan")
        index = torch.full((rows,), -1, dtype=torch.int32)
        got = binding.gemm_q4_grouped(torch.ones(4, 96).cuda(), packed.cuda()[None],
                                      scale.cuda()[None],
                                      torch.tensor([0, rows], dtype=torch.int32).cuda(),
                                      group=32, index_a=index.cuda())
        assert torch.equal(got.cpu(), torch.zeros(rows, 40))


def test_codes_beyond_32_bit_offsets(gpu_lib):
    """Experts whose codes lie more than 4 GiB apart, scales and outputs too."""
    H.say("q4 beyond 32 bits")
    g = gen(3)
    K, N, far = 64, 32, (1 << 32) + 64
    packed, scale, _, W = weights(g, N, K, 32, "symmetric", "f32", lead=(2,), integer=True)
    room = torch.empty(far + N * K, dtype=torch.uint8, device="cuda")
    codes = torch.as_strided(room, (2, N, K // 2), (far, K // 2, 1))
    codes.copy_(packed)
    a = torch.randint(-2, 3, (8, K), generator=g).float()
    for rows in (8, 150):
        x = a.repeat((rows + 7) // 8, 1)[:rows]
        half = rows // 2
        pitch = (1 << 31) // rows + 100
        c = torch.as_strided(torch.empty((rows - 1) * pitch + N, device="cuda"), (rows, N),
                             (pitch, 1))
        off = torch.tensor([0, half, rows], dtype=torch.int32)
        binding.gemm_q4_grouped(x.cuda(), codes, scale.cuda(), off.cuda(), c, group=32)
        want = torch.cat([x[:half].double() @ W[0].t(), x[half:].double() @ W[1].t()])
        assert torch.equal(c.cpu().double(), want)
        del c


def test_repeats_bit_for_bit(gpu_lib):
    H.say("q4 repeats")
    g = gen(4)
    for M in (1, 13, 300):
        a = torch.randn(M, 1000, generator=g).cuda()
        packed, scale, zero, _ = weights(g, 300, 1000, 32, "zeros", "bf16")
        args = (a, packed.cuda(), scale.cuda())
        first = binding.gemm_q4(*args, zero=zero.cuda(), group=32)
        for _ in range(3):
            assert torch.equal(binding.gemm_q4(*args, zero=zero.cuda(), group=32), first)


def test_captured_products_replay(gpu_lib):
    H.say("q4 captured")
    g = gen(6)
    K, N, E = 320, 200, 5
    packed, scale, zero, _ = weights(g, N, K, 64, "zeros", "f16", lead=(E,))
    packed, scale, zero = packed.cuda(), scale.cuda(), zero.cuda()
    xs = [torch.randn(M, K, generator=g).cuda() for M in (1, 30, 400)]
    offsets = torch.tensor([0, 100, 100, 300, 301, 400], dtype=torch.int32).cuda()

    def step():
        out = [binding.gemm_q4(x, packed[1], scale[1], zero=zero[1], group=64) for x in xs]
        return [*out, binding.gemm_q4_grouped(xs[2], packed, scale, offsets, zero=zero, group=64)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = step()
        for seed in (1, 2, 3):
            for x in xs:
                x.copy_(torch.randn(x.shape, generator=gen(seed)))
            graph.replay()
            stream.synchronize()
            kept = [t.clone() for t in captured]
            for a, b in zip(kept, step()):
                assert torch.equal(a, b)
            stream.synchronize()


def test_a_served_expert_layer(gpu_lib):
    """A decode batch through 4-bit experts: routing, order, up product with ReLU,
    down product scattered to the choices' slots, join; against 64 bits."""
    H.say("q4 expert layer")
    T, E, top, D, F = 9, 8, 2, 96, 160
    g = gen(8)
    x, logits = torch.randn(T, D, generator=g), torch.randn(T, E, generator=g)
    logits[4] = -float("inf")                           # a padded token
    up = q4.quantize(torch.randn(E, F, D, generator=g) * D ** -0.5, group=32, format=E2M1,
                     scale_dtype=torch.uint8)
    down = q4.quantize(torch.randn(E, D, F, generator=g) * F ** -0.5, group=64, symmetric=False,
                       scale_dtype=torch.float16)
    choice, weight = binding.route(logits.cuda(), top, renorm=True)
    offsets, order, token = binding.group_rows(choice.view(-1), E, per_row=top)
    X = x.cuda()
    h = binding.gemm_q4_grouped(X, up[0].cuda(), up[1].cuda(), offsets, group=32, format=E2M1,
                                index_a=token, act=binding.ACT_RELU)
    out = X.new_full((T * top, D), float("nan"))
    binding.gemm_q4_grouped(h, down[0].cuda(), down[1].cuda(), offsets, out, zero=down[2].cuda(),
                            group=64, index_c=order)
    y = binding.join_rows(out, weight, choice, groups=E).cpu().double()
    Wu = q4.dequantize(up[0], up[1], D, group=32, format=E2M1, dtype=torch.float64)
    Wd = q4.dequantize(down[0], down[1], F, zero=down[2], group=64, dtype=torch.float64)
    c, w = choice.cpu().long(), weight.cpu().double()
    for t in range(T):
        want, mag = torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
        for j in range(top):
            if c[t, j] < 0:
                continue
            hid = (Wu[c[t, j]] @ x[t].double()).clamp_min(0)
            want += w[t, j] * (Wd[c[t, j]] @ hid)
            mag += w[t, j] * (Wd[c[t, j]].abs() @ (Wu[c[t, j]].abs() @ x[t].double().abs()))
        assert bool(((y[t] - want).abs() <= (D + F + 300) * U * mag).all())
    assert torch.equal(y[4], torch.zeros(D, dtype=torch.float64))
