"""GPU tests of the products with 4-bit weights at their edges: values that are not
finite and unused codes where K ends inside a step, and groups of very uneven sizes."""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding, q4
from tests import gpu_helpers as H
from tests.test_gpu_grouped import gen
from tests.test_gpu_q4 import E2M1, INT, KERNELS, KINDS, grouped

pytestmark = pytest.mark.gpu

INF = float("inf")


def equal(got, want):
    """The same values, infinities by their sign, and NaN where NaN is."""
    return torch.equal(got.isnan(), want.isnan()) and \
        torch.equal(got[~got.isnan()], want[~want.isnan()])


def edge_depths(kernel):
    """K that end inside a chunk of 128, and inside a step of 32 times the waves that
    share K."""
    return (515, 641, 1030) if kernel == "few" else (40, 97, 203, 333)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64])
def test_infinite_scales_of_the_last_group(gpu_lib, kernel, kind, group):
    """Weights of one sign times values above zero: the formula gives the infinity."""
    M, N = KERNELS[kernel]
    for K in edge_depths(kernel):
        H.say(f"q4 infinite last scales {kernel} {kind} group={group} K={K}")
        g = gen(K + M)
        a = torch.randint(1, 4, (M, K), generator=g).float()
        codes = torch.randint(9, 16, (N, K), generator=g)
        codes[2::5] = 15 - codes[2::5]     # 6 and below: weights below zero
        scale = (2.0 ** torch.randint(-1, 2, (N, (K + group - 1) // group), generator=g)
                 ).to(KINDS[kind])
        scale[1::7, -1] = INF
        scale[2::7, -1] = -INF
        scale[3::7, max(scale.shape[1] - 2, 0)] = INF
        scale[4::7, -1] = float("nan")
        got = binding.gemm_q4(a.cuda(), q4.pack(codes).cuda(), scale.cuda(),
                              group=group).cpu().double()
        W = q4.dequantize(q4.pack(codes), scale, K, group=group, dtype=torch.float64)
        assert not W[1::7].isnan().any()
        # (columns of finite weights as a product, the others by their sign: every weight of
        # the group has it)
        want = a.double() @ torch.where(W.isfinite(), W, torch.zeros_like(W)).t()
        odd = W.sum(1)
        want[:, ~odd.isfinite()] = odd[~odd.isfinite()]
        assert equal(got, want)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("form", ["symmetric", "zeros", "e2m1"])
def test_the_unused_half_beside_large_powers(gpu_lib, kernel, form):
    """An odd K leaves half a byte, which may hold a code whose weight would pass the
    largest float where the real ones do not."""
    M, N = KERNELS[kernel]
    for K in (515, 641) if kernel == "few" else (1, 33, 97, 203):
        for e in (253, 254):
            H.say(f"q4 unused half {kernel} {form} K={K} e={e}")
            g = gen(K + M)
            a = torch.randint(1, 3, (M, K), generator=g).float() * 2.0 ** -30
            along = (K + 31) // 32
            scale = torch.full((N, along), e, dtype=torch.uint8)
            zero = None
            if form == "e2m1":
                codes = torch.randint(0, 3, (N, K), generator=g)        # 0, .5, 1
            else:
                codes = torch.randint(7, 10, (N, K), generator=g)       # -1, 0, 1
            if form == "zeros":
                zero = torch.randint(3, 6, (N, along), generator=g).to(torch.uint8)
                zero[::9] = 200
                codes = codes - 8 + zero.long().clamp_max(14)[:, torch.arange(K) // 32]
                scale[::9] = 100
            packed = q4.pack(codes)
            packed[..., -1] |= 0xf0 if form == "symmetric" else 0x70
            fmt = E2M1 if form == "e2m1" else INT
            W = q4.dequantize(packed, scale, K, zero=zero, group=32, format=fmt,
                              dtype=torch.float64)
            got = binding.gemm_q4(a.cuda(), packed.cuda(), scale.cuda(), format=fmt, group=32,
                                  zero=None if zero is None else zero.cuda())
            # whole numbers times one power: exact in every order
            assert torch.equal(got.cpu().double(), a.double() @ W.t())


# counts and columns: all places in one group, in the last, nearly all, one each in a few of many
UNEVEN = {"one": [192] + [0] * 31, "last": [0] * 31 + [192], "most": [150, 0, 1, 0, 20, 1, 0, 20],
          "alone": [150], "few of many": [1, 0, 0, 0, 2] + [0] * 200 + [5],
          "ends of many": [300] + [0] * 998 + [4] + [1] * 24, "nobody": [0, 0, 0],
          "even": [3] * 100, "full": [12, 13, 20, 21, 24, 25, 40, 41]}


@pytest.mark.parametrize("name", list(UNEVEN))
@pytest.mark.parametrize("K,N", [(640, 300), (131, 16), (2100, 64)])
def test_uneven_groups_of_few_rows(gpu_lib, name, K, N):
    if len(UNEVEN[name]) > 300 and N > 16:
        pytest.skip("as many weights of this size take gigabytes on the host")
    grouped(UNEVEN[name], K, N, "zeros", "f16", group=32, spare=4)
    grouped(UNEVEN[name], K, N, "e2m1", "e8m0", group=64, integer=False, gather=False,
            scatter=False, bias=False, act=0, beta=0.5)


@pytest.mark.parametrize("counts", [[192] + [0] * 31, [0] * 31 + [192],
                                    [96, 40, 20, 10, 10, 8, 4, 4] + [0] * 24])
def test_uneven_groups_fill_the_device(gpu_lib, counts):
    """All rows in one of 32 groups are 10 row tiles, which go beside each other: about as
    long as 6 rows in each (one after another they took 9 times as long).  A factor of 4 is
    far from either."""
    H.say(f"q4 uneven groups in time {counts[:4]}")
    K, N, G = 1024, 2048, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (G, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(120, 125, (G, N, K // 32), generator=g, device="cuda").to(torch.uint8)
    a, c = torch.randn(192, K, generator=g, device="cuda"), torch.empty(192, N, device="cuda")

    def time(rows):
        off = torch.tensor([0, *torch.tensor(rows).cumsum(0).tolist()], dtype=torch.int32).cuda()
        took = []
        for _ in range(20):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            for _ in range(20):
                binding.gemm_q4_grouped(a, codes, scale, off, c, group=32, format=E2M1)
            end.record()
            end.synchronize()
            took.append(begin.elapsed_time(end))
        return sorted(took)[10]
    assert time(counts) < 4 * time([6] * G)


@pytest.mark.parametrize("G", [3, 64, 65, 1024])
@pytest.mark.parametrize("K", [160, 1100])
def test_offsets_that_leave_the_places_with_few_rows(gpu_lib, G, K):
    """Offsets are taken into [0, rows], a group that ends before it begins is empty, and
    rows of no group stay as they were: with the groups in lanes and in threads."""
    H.say(f"q4 few rows, odd offsets G={G} K={K}")
    g = gen(G)
    N, rows = 24, 40
    a = torch.randint(-2, 3, (rows, K), generator=g).float()
    packed = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8)
    scale = torch.ones(G, N, (K + 31) // 32)
    middle = G // 2
    # (groups between the three are empty)
    cases = [([first] + [10] * middle + [33] * (G - 1 - middle) + [last],
              {0: (max(first, 0), 10), middle: (10, 33), G - 1: (33, min(last, rows))})
             for first, last in ((-5, 99), (4, 36))]
    cases.append(([50 - i for i in range(G + 1)], {}))   # each ends before it begins
    for off, span in cases:
        c = torch.full((rows, N), 7.0, device="cuda")
        binding.gemm_q4_grouped(a.cuda(), packed.cuda(), scale.cuda(),
                                torch.tensor(off, dtype=torch.int32).cuda(), c, group=32)
        want = torch.full((rows, N), 7.0, dtype=torch.float64)
        for e, (b, t) in span.items():
            W = q4.dequantize(packed[e], scale[e], K, group=32, dtype=torch.float64)
            want[b:t] = a[b:t].double() @ W.t()
        assert torch.equal(c.cpu().double(), want)


@pytest.mark.parametrize("G", [32, 200])
def test_captured_few_rows_follow_new_offsets(gpu_lib, G):
    """A replay finds the row tiles from the offsets that are there then."""
    H.say(f"q4 few rows captured, new offsets G={G}")
    g = gen(G + 5)
    K, N, rows = 512, 640, 130
    a = torch.randint(-2, 3, (rows, K), generator=g).float().cuda()
    packed = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scale = (2.0 ** torch.randint(-1, 2, (G, N, K // 64), generator=g)).cuda()
    offsets, c = torch.zeros(G + 1, dtype=torch.int32, device="cuda"), torch.zeros(rows, N).cuda()

    def step():
        return binding.gemm_q4_grouped(a, packed, scale, offsets, c, group=64)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for counts in ([rows] + [0] * (G - 1), [0] * (G - 1) + [rows - 7],
                       [rows // G + (i < rows % G) for i in range(G)], [0] * G,
                       [60] + [0] * (G - 3) + [1, 50]):
            offsets.copy_(torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()]))
            c.fill_(3.0)
            graph.replay()
            stream.synchronize()
            got = c.clone()
            c.fill_(3.0)
            step()
            stream.synchronize()
            assert torch.equal(got, c)
            end = sum(counts)
            assert bool((got[end:] == 3.0).all())
            at = 0
            for e, n in enumerate(counts):
                if n:
                    W = q4.dequantize(packed[e].cpu(), scale[e].cpu(), K, group=64,
                                      dtype=torch.float64)
                    assert torch.equal(got[at:at + n].cpu().double(),
                                       a[at:at + n].cpu().double() @ W.t())
                at += n
