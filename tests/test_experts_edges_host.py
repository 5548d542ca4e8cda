"""The operators around an expert layer on the host: a call that the binding refuses, and
which kernel the 4-bit products of uneven and many groups take.
CPU only."""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding
from tests.test_q4_routes_host import route  # noqa: F401


def test_clipping_needs_a_limit():
    """Without one it would give the norm and leave ``out`` unwritten."""
    x = torch.ones(3)
    for out in (None, [torch.ones(3)]):
        with pytest.raises(TypeError, match="max_norm"):
            binding.clip_norm([x], None, out=out)


@pytest.mark.parametrize("rows,N,K,groups,want", [
    (128, 7168, 2048, 32, "few"), (256, 7168, 2048, 32, "few"), (320, 7168, 2048, 32, "few"),
    (1536, 7168, 2048, 32, "64x128"), (64, 2048, 7168, 8, "few"), (8, 2048, 7168, 256, "few"),
    (1024, 2048, 1024, 128, "few"), (150, 16, 4096, 1, "few")])
def test_choices_of_the_4_bit_products(route, rows, N, K, groups, want):
    """A few rows in each of many groups stay with the kernel for few rows (7168 x 2048, 8
    rows in each of 32 groups: 86 us against 236 by tiles), and groups of fewer rows than a
    tile has count one each."""
    assert route(rows, N, K, groups) == want
