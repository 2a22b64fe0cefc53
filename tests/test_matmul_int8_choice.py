"""The tile that a product takes, from the library's own log, on the CPU: the shapes that
test every tile on the GPU take the tile that they are named for on a device of 256 compute
units.  The calls run in a child process that sees no device, so each ends in the launch's
error after its choice is written."""
import os
import re
import subprocess
import sys

import pytest

import arithmetic_reduction_matrix_amd as armx
from test_gpu_matmul_int8_tiles import OFF_LINE_SHAPES, SHAPES, STARTS

CHILD = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
devices = ctypes.c_int(0)
lib.hipGetDeviceCount(ctypes.byref(devices))
if devices.value:
    raise SystemExit("a device is visible")
vp, sz = ctypes.c_void_p, ctypes.c_size_t
lib.matmul_int8.argtypes = [vp, sz, vp, vp, sz, vp, vp, sz, sz, sz, vp, sz, ctypes.c_int, vp, vp]
P = 1 << 40        # never dereferenced
for line in sys.stdin:
    m, n, k, lda, ldb, at_a, at_b = map(int, line.split())
    st = lib.matmul_int8(P + at_a, lda, P, P + at_b, ldb, P, None, m, n, k, P, n, 1, None, None)
    if st != -6:
        raise SystemExit(f"status {st} for {line}")
"""


def pitch(k, past):
    pieces = -(-k // 16)
    return 16 * (pieces + (past - pieces) % 8)


def calls():
    """(name of the tile, off the lines or not, the call's numbers), as the GPU tests make
    them."""
    for off, shapes in ((False, SHAPES), (True, OFF_LINE_SHAPES)):
        for name, several in shapes.items():
            for m, n, ks in several:
                for k in ks:
                    pa, pb, sa, sb = STARTS[(m + n + k) % len(STARTS)] if off else (0, 0, 0, 0)
                    yield name, off, (m, n, k, pitch(k, pa), pitch(k, pb), 16 * sa, 16 * sb)


@pytest.fixture(scope="module")
def chosen():
    env = {**os.environ, "ARMX_LOG": "1", "HIP_VISIBLE_DEVICES": "-1"}
    r = subprocess.run([sys.executable, "-c", CHILD, armx.LIB_PATH], text=True, env=env,
                       input="\n".join(" ".join(map(str, c)) for _, _, c in calls()),
                       capture_output=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    return [line for line in r.stderr.splitlines() if line.startswith("armx: matmul_int8 ")]


def test_named_tiles_are_the_ones_taken(chosen):
    wanted = list(calls())
    assert len(chosen) == len(wanted)
    for (name, off, (m, n, k, *_)), line in zip(wanted, chosen):
        assert f" m={m} n={n} k={k} " in line
        assert f" tile={name} " in line and line.endswith(f" off_lines={int(off)}"), (name, line)


def test_every_tile_is_taken(chosen):
    found = {tuple(re.search(r"tile=(\S+) .*off_lines=(\d)", line).groups()) for line in chosen}
    assert found == {(name, str(int(off))) for name, off, _ in calls()}
    assert len(SHAPES) == len(OFF_LINE_SHAPES) == 11
