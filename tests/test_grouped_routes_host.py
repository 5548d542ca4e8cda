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
