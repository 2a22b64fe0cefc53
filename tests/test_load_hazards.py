"""Wait states in the built gfx950 code around loads from memory straight into LDS.

Such a load takes its LDS address from M0, and on gfx9 a scalar write of M0 needs one
wait state (any instruction, or an s_nop) before it is read there; a resource that a
vector instruction wrote into scalar registers needs five.  The compiler keeps both for
instructions that it emits itself, but not inside an asm string or across its ends."""
import os
import re
import shutil
import subprocess

import pytest

import arithmetic_reduction_matrix_amd as armx

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
SCALARS = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b")


def scalars(text):
    """Numbers of the scalar registers named in `text`."""
    found = set()
    for lo, hi, one in SCALARS.findall(text):
        found |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return found


@pytest.fixture(scope="module")
def instructions(tmp_path_factory):
    """The instructions of every gfx950 code object of the library, in order."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    folder = tmp_path_factory.mktemp("code")
    shutil.copy(armx.LIB_PATH, folder / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=folder, check=True,
                   capture_output=True)
    objects = sorted(f for f in os.listdir(folder) if f.endswith("gfx950"))
    assert objects
    found = []
    for f in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f], cwd=folder, check=True,
                              capture_output=True, text=True).stdout
        lines = (line.split("//")[0].strip() for line in text.splitlines())
        found.append([line for line in lines if re.match(r"[a-z]+_", line)])
    return found


def lds_loads(code):
    return [i for i, text in enumerate(code)
            if text.startswith(("buffer_load", "global_load")) and text.endswith(" lds")]


def test_m0_is_written_a_wait_state_before_a_load_into_lds(instructions):
    seen = 0
    for code in instructions:
        for i in lds_loads(code):
            seen += 1
            assert not re.match(r"s_\w+ m0,", code[i - 1]), (code[i - 1], code[i])
    assert seen


def test_nothing_else_uses_m0_beside_loads_into_lds(instructions):
    for code in instructions:
        if lds_loads(code):
            assert {text.split(",")[0] for text in code if re.search(r"\bm0\b", text)} == {
                "s_mov_b32 m0"}


def test_resources_are_written_five_wait_states_before_a_load_into_lds(instructions):
    for code in instructions:
        for i in lds_loads(code):
            used, states = scalars(code[i]), 0
            for text in reversed(code[max(i - 5, 0):i]):
                if text.startswith("s_nop"):
                    states += int(text.split()[1])
                if states >= 5:
                    break
                if text.startswith(("v_readfirstlane", "v_readlane", "v_cmp")):
                    assert not scalars(text.split(",")[0]) & used, (text, code[i])
                states += 1
