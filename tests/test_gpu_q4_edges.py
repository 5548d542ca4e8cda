"""GPU tests of the products with 4-bit weights at their edges: values that are not
finite, and unused codes, where K ends inside a step."""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding, q4
from tests import gpu_helpers as H
from tests.test_gpu_grouped import gen
from tests.test_gpu_q4 import E2M1, INT, KERNELS, KINDS

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
