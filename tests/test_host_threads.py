"""Host threads that call on one stream at once (CPU only): the C-ABI sources
with stand-ins for the HIP calls and the launches (host_threads.cpp).  A call
that passes partial sums through its stream's workspace from one launch to the
next must not be split by another thread's call."""
import re
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
CSRC = ROOT / "dense_fp32_gemm_f32_amd" / "csrc"


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    if shutil.which("g++") is None or not Path("/opt/rocm/include/hip").is_dir():
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path_factory.mktemp("threads") / "host_threads"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-D__HIP_PLATFORM_AMD__=1",
                    "-I/opt/rocm/include", f"-I{ROOT / 'include'}",
                    ROOT / "tests" / "host_threads.cpp", CSRC / "gemm_f32_api.cpp",
                    CSRC / "gemm_f32_grouped_api.cpp", "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    return r.stdout.splitlines()


@pytest.mark.parametrize("name", ["adapters", "wgrad", "few_rows", "noalloc"])
def test_calls_on_one_stream_are_not_split(lines, name):
    found = [re.fullmatch(rf"{name} calls (\d+) refused (\d+) wrong (\d+)", l) for l in lines]
    found = [tuple(map(int, m.groups())) for m in found if m]
    assert found == [(200, 0, 0)] * 2


def test_two_handles_of_one_stream_share_the_fixed_array_in_turn(lines):
    assert "both_handles calls 200 refused 0 wrong 0" in lines


def test_each_threads_own_stream_has_its_own_workspace(lines):
    """hipStreamPerThread is one handle for another stream in every thread."""
    assert "per_thread got 1 shared 0" in lines
