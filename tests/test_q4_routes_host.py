"""Which kernel a product with 4-bit weights takes (CPU only): the rules are host code
without a HIP call, asked by q4_routes.cpp.  The sizes at which the GPU tests run each
kernel must go on reaching it."""
import shutil
import subprocess
from pathlib import Path

import pytest

from tests import test_gpu_q4 as q4

ROOT = Path(__file__).resolve().parent.parent


@pytest.fixture(scope="module")
def route(tmp_path_factory):
    if shutil.which("g++") is None or not Path("/opt/rocm/include/hip").is_dir():
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path_factory.mktemp("routes") / "q4_routes"
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include",
                    ROOT / "tests" / "q4_routes.cpp", "-o", exe], check=True)

    def ask(*call):
        return subprocess.run([exe], input=" ".join(map(str, call)), capture_output=True,
                              text=True, check=True).stdout.strip()
    return ask


@pytest.mark.parametrize("kernel", list(q4.KERNELS))
def test_cases_reach_their_kernel(route, kernel):
    M, N = q4.KERNELS[kernel]
    for K in ((640, 515) if kernel == "few" else (1, 32, 160, 203)):
        assert route(M, N, K, 1) == kernel


@pytest.mark.parametrize("M,N,K", q4.FEW)
def test_few_rows_reach_their_kernel(route, M, N, K):
    assert route(M, N, K, 1) == "few"


@pytest.mark.parametrize("kernel", list(q4.WIDE))
def test_grouped_cases_reach_their_kernel(route, kernel):
    counts, N = q4.WIDE[kernel]
    assert route(sum(counts) + 3, N, 515 if kernel == "few" else 67, len(counts)) == kernel


@pytest.mark.parametrize("rows,N,K,groups,want", [
    (1, 8192, 8192, 1, "few"), (1, 8192, 127, 1, "32x32"), (8, 28672, 8192, 1, "few"),
    (24, 4096, 4096, 1, "32x32"), (32, 1024, 4096, 1, "few"), (4096, 4096, 4096, 1, "256x256"),
    (192, 2048, 1024, 32, "few"), (8192, 1024, 2048, 8, "256x192"),
    (2048, 4096, 4096, 1, "256x128"),
    (1000, 4096, 64, 1, "128x128"), (2147418112, 2147418112, 1, 1, "256x256"),
    (2147418112, 1000, 4096, 1024, "256x256")])
def test_choices(route, rows, N, K, groups, want):
    assert route(rows, N, K, groups) == want
