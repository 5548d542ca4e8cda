"""GPU tests of the products with 4-bit weights at their edges: values that are not
finite where K ends inside a step."""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding, q4
from tests import gpu_helpers as H
from tests.test_gpu_grouped import gen
from tests.test_gpu_q4 import KERNELS, KINDS

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
