"""GPU tests of the edges of the grouped products that every kernel has to keep
by itself: indexes outside, offsets outside or falling, operands beyond 32-bit
offsets, values that are not finite.  Each runs at sizes of each kernel.

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
