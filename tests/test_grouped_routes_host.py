"""Which kernel a grouped call takes (CPU only): the rules are host code without a
HIP call, asked by grouped_routes.cpp.  The sizes at which the GPU tests run each
kernel's edges must go on reaching it."""
import shutil
import subprocess
from pathlib import Path

import pytest

from tests import test_gpu_grouped_tiles as tiles

ROOT = Path(__file__).resolve().parent.parent


@pytest.fixture(scope="module")
def routes(tmp_path_factory):
    if shutil.which("g++") is None or not Path("/opt/rocm/include/hip").is_dir():
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path_factory.mktemp("routes") / "grouped_routes"
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include",
                    ROOT / "tests" / "grouped_routes.cpp", "-o", exe], check=True)

    def ask(*call):
        return subprocess.run([exe], input=" ".join(map(str, call)), capture_output=True,
                              text=True, check=True).stdout.strip()
    return ask


@pytest.mark.parametrize("kernel,trans", list(tiles.PRODUCT))
def test_product_cases_reach_their_kernel(routes, kernel, trans):
    counts, K, N = tiles.PRODUCT[kernel, trans]
    call = ["product", int(trans), sum(counts), N, K, len(counts)]
    assert routes(*call, K, K if trans else N, K * N) == kernel
    # far apart, at pitches that keep (or, for single floats, spoil) 16 bytes
    odd = 1 if "1 float" in kernel else 0
    assert routes(*call, 4000 + odd, K if trans else N, 4 * 10 ** 8 + odd) == kernel


@pytest.mark.parametrize("kernel", list(tiles.GRADIENT))
def test_gradient_cases_reach_their_kernel(routes, kernel):
    counts, M, N = tiles.GRADIENT[kernel]
    call = ["gradient", sum(counts), M, N, len(counts)]
    name = "thin" if kernel.startswith("thin") else kernel
    odd = 1 if "1 float" in kernel else 0
    assert routes(*call, M, N) == name
    assert routes(*call, 4000 + odd, 4000 + odd) == name


def test_every_kernel_has_a_case():
    assert {k for k, _ in tiles.PRODUCT} == {"rows", "mixed", "64, 4 floats", "64, 1 float",
                                            "128, 1 float"}
    assert {k for k in tiles.GRADIENT if "thin" not in k} == {
        "64, 4 floats", "64, 1 float", "64, 4 floats, slices", "64, 1 float, slices",
        "128, 4 floats", "128, 1 float"}


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,N,want", [
    (1408, 2048, "fused"),     # 176 tiles of 128 x 128: gemm_f32_fused takes smaller ones
    (2048, 1536, "grouped"), (3000, 1024, "grouped"), (1600, 1856, "grouped"),
    # four rounds of 64 x 64 tiles: one round of 128 x 128 is faster
    (1664, 2048, "fused"), (1792, 2048, "fused"), (4096, 896, "fused"), (1920, 2048, "fused"),
    (2040, 2040, "fused"), (2304, 2048, "fused")])
def test_projection_of_adapters_by_rounds(routes, trans, M, N, want):
    for K in (512, 1024, 2048):
        assert routes("projection", trans, M, N, K, K, K if trans else N) == want
    # sizes or pitches that 16 bytes do not fit
    assert routes("projection", trans, M, N, 1023, 1023, 1023 if trans else N) == "fused"
    assert routes("projection", trans, M, N, 1024, 1025, 1024 if trans else N) == "fused"


@pytest.mark.parametrize("trans,M,N,want", [
    (1, 100, 2048, "grouped"), (1, 128, 2048, "grouped"), (1, 129, 2048, "fused"),
    (1, 65, 4096, "fused"), (0, 100, 2048, "fused")])
def test_projection_of_adapters_few_rows(routes, trans, M, N, want):
    for K in (512, 2048, 2049):
        assert routes("projection", trans, M, N, K, K, K if trans else N) == want
