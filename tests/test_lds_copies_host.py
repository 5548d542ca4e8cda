"""The copies from global memory into LDS that are written as inline assembly
(CPU only: reads the sources and the built library).  The compiler inserts the
wait states that the hardware asks for, but sees no load inside a string."""
import re
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "dense_fp32_gemm_f32_amd" / "csrc"


def assembly(text):
    """The instructions of each inline-assembly string of a source."""
    for block in re.findall(r"\basm\b(?:\s+volatile)?\s*\((.*?)\)\s*;", text, re.S):
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', re.split(r"^\s*:", block, flags=re.M)[0]))
        yield [i.strip() for i in re.split(r"\\n|\\t|;", code) if i.strip()]


def hazards(text):
    """Loads into LDS whose M0 is written by the instruction just before."""
    return [(a, b) for code in assembly(text) for a, b in zip(code, code[1:])
            if re.match(r"s_\w+ m0,", a) and re.search(r"\blds\b|_lds_", b)]


def test_a_load_into_lds_waits_for_m0():
    """A scalar write of M0 needs one wait state before a load that writes LDS."""
    copies = 0
    for path in sorted([*CSRC.glob("*.h"), *CSRC.glob("*.hip")]):
        text = path.read_text()
        copies += sum(any("_lds_" in i for i in code) for code in assembly(text))
        assert not hazards(text), path.name
    assert copies >= 4


@pytest.mark.parametrize("between,found", [("", 1), ('"s_nop 0\\n\\t"', 0)])
def test_the_check_sees_a_missing_wait(between, found):
    text = ('asm volatile("s_mov_b32 m0, %2\\n\\t" ' + between
            + ' "global_load_lds_dword %1, off"\n : : "v"(g), "s"(a));')
    assert len(hazards(text)) == found


OBJDUMP = Path("/opt/rocm/llvm/bin/llvm-objdump")


def unwaited(listing):
    """Loads into LDS of a disassembly that come too soon behind the scalar they
    use: one wait state behind a scalar write of M0, five behind a vector
    instruction's write of M0 or of a scalar of their address."""
    found, past = [], []
    for line in listing.splitlines():
        code = line.split("//")[0].strip()
        if not code or code.endswith(":"):
            past = []
            continue
        if "load_lds" in code:
            pair = re.search(r"\bs\[(\d+):(\d+)\]", code)
            states = 0
            for before in reversed(past):
                if states < 1 and re.match(r"s_\w+ m0,", before):
                    found.append((before, code))
                written = re.match(r"v_read(?:first)?lane_b32 (?:s(\d+)|m0),", before)
                if states < 5 and written and (
                        written[1] is None
                        or (pair and int(pair[1]) <= int(written[1]) <= int(pair[2]))):
                    found.append((before, code))
                nop = re.match(r"s_nop (\d+)", before)
                states += int(nop[1]) + 1 if nop else 1
        past = [*past[-7:], code]
    return found


@pytest.mark.parametrize("text,found", [
    ("s_mov_b32 m0, s4\nglobal_load_lds_dword v0, s[0:1]", 1),
    ("s_mov_b32 m0, s4\ns_nop 0\nglobal_load_lds_dword v0, s[0:1]", 0),
    ("v_readfirstlane_b32 s1, v0\ns_nop 3\nglobal_load_lds_dword v0, s[0:1]", 1),
    ("v_readfirstlane_b32 s1, v0\ns_nop 4\nglobal_load_lds_dword v0, s[0:1]", 0),
    ("v_readlane_b32 s2, v0, 3\nglobal_load_lds_dword v0, s[0:1]", 0),
    ("v_readfirstlane_b32 m0, v0\ns_nop 0\nglobal_load_lds_dword v0, s[0:1]", 1),
])
def test_the_disassembly_check_counts_wait_states(text, found):
    assert len(unwaited(text)) == found


@pytest.mark.parametrize("name", ["libgemm_f32.so", "libgemm_f32_sweep.so"])
def test_built_copies_wait_for_their_scalars(name, tmp_path):
    """The same over the code built here: the compiler places what stands around
    the strings."""
    lib = CSRC.parent / name
    if not lib.exists() or not OBJDUMP.exists():
        pytest.skip(f"{name} is not built, or no disassembler")
    (tmp_path / "lib.so").symlink_to(lib)
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True,
                   capture_output=True)
    objects = list(tmp_path.glob("lib.so.*gfx950*"))
    assert objects
    loads = 0
    for obj in objects:
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", obj], check=True,
                              capture_output=True, text=True).stdout
        loads += text.count("load_lds")
        assert not unwaited(text), obj.name
    assert loads > 100
