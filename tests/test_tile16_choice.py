"""The tiles that the products of the cross entropy take, from the library's own log, on the
CPU: the shapes that test every tile on the GPU take those that they are named for on a
device of 256 compute units; and pieces of the vocabulary that 32-bit offsets reach, at the
ends of the sizes that are taken.  The calls run in a child process that sees no device, so each
ends in the launch's error after its choice is written."""
import os
import re
import subprocess
import sys

import pytest

import arithmetic_reduction_matrix_amd as armx
from test_gpu_cross_entropy_tiles import BATCHES, SHAPES

CHILD = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
devices = ctypes.c_int(0)
lib.hipGetDeviceCount(ctypes.byref(devices))
if devices.value:
    raise SystemExit("a device is visible")
vp, sz, ci, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
lib.cross_entropy_rows.argtypes = [vp, sz, vp, sz, vp, ci, sz, sz, sz, i64, vp, vp, vp, sz, vp, vp]
lib.cross_entropy_rows_backward.argtypes = [vp, vp, sz, vp, sz, vp, vp, ci, sz, sz, sz, i64, vp,
                                            sz, vp, sz, ci, vp, sz, vp, vp]
P = 1 << 40        # never dereferenced
Q = P + 4096
for line in sys.stdin:
    rows, vocab, cols = map(int, line.split())
    ld = (cols + 7) // 8 * 8
    st = (lib.cross_entropy_rows(P, ld, P, ld, P, 0, rows, vocab, cols, -100, P, Q, P, P, None,
                                 None),
          lib.cross_entropy_rows_backward(P, P, ld, P, ld, P, P, 0, rows, vocab, cols, -100, P, ld,
                                          Q, ld, 0, P, P, None, None))
    if st != (-6, -6):
        raise SystemExit(f"status {st} for {line}")
"""
TILES = {"256x256", "192x256", "256x128", "128x128", "64x128", "16x128", "16x64"}


def choices(calls):
    """What the library's log says of its calls on these sizes."""
    env = {**os.environ, "ARMX_LOG": "1", "HIP_VISIBLE_DEVICES": "-1"}
    r = subprocess.run([sys.executable, "-c", CHILD, armx.LIB_PATH], text=True, env=env,
                       input="\n".join(" ".join(map(str, c)) for c in calls),
                       capture_output=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    found = {}
    for line in r.stderr.splitlines():
        m = re.match(r"armx: (cross_entropy_rows\S*) rows=(\d+) vocab=(\d+) cols=(\d+) ", line)
        if m:
            found[(m.group(1), *map(int, m.groups()[1:]))] = dict(re.findall(r"(\w+)=(\S+)", line))
    assert len(found) == 2 * len(set(calls))
    return found


@pytest.fixture(scope="module")
def chosen():
    return choices(list(SHAPES) + [(n, 20000, 200) for n, _ in BATCHES])


def test_named_tiles_are_the_ones_taken(chosen):
    for shape, names in SHAPES.items():
        logits, dx, dweight = names.split()
        got = chosen[("cross_entropy_rows_backward", *shape)]
        assert (got["logits"], f'{got["dx"]}/{got["parts"]}', got["dweight"]) == (
            logits, dx, dweight), shape
        assert int(got["piece"]) >= shape[1], shape
        assert chosen[("cross_entropy_rows", *shape)]["tile"] == logits, shape


def test_every_tile_is_taken(chosen):
    names = [n.split() for n in SHAPES.values()]
    assert {n[0] for n in names} == TILES
    assert {n[1].split("/")[0] for n in names} == TILES
    assert {n[2] for n in names} == TILES
    assert {name for _, name in BATCHES} == TILES


def test_batches_of_every_tile(chosen):
    for n, name in BATCHES:
        assert chosen["cross_entropy_rows", n, 20000, 200]["tile"] == name, n


def test_tiles_reach_their_rows():
    # the bytes from the first to the end of the last of a tile's rows, at most 256, in the
    # matrices that the gradients make: dz (rows x piece), its transpose and x's
    rows = [1, 2, 3, 100, 127, 128, 129, 255, 256, 257, 4095, 65536, (1 << 17) - 1, 1 << 17,
            (1 << 17) + 1, (1 << 19) + 77, (1 << 21) - 1, 1 << 21]
    vocabs = [1, 100, 1023, 1025, 50001, 131072, 1 << 24, (1 << 28) - 1, 1 << 28]
    colss = [1, 8, 100, 4096, 65536, (1 << 21) - 1, 1 << 21]

    def tiles(a, b):
        return -(-a // 256) * -(-b // 256)
    calls = [(r, v, c) for r in rows for v in vocabs for c in colss
             if max(tiles(r, v), tiles(r, c)) <= 2097151 and (max(r, v) - 1) * (c + 8) < 1 << 40]
    assert len(calls) > 400
    for (call, r, v, c), got in choices(calls).items():
        if call == "cross_entropy_rows":
            continue
        piece, terms = int(got["piece"]), int(got["terms"])
        assert piece % 256 == 0 and piece >= min(v, 256)
        k = r * terms
        ldz, ldt = piece + 64, k + 255 + 128
        assert (min(r, 256) - 1) * ldz * 2 + piece * 2 <= 0xFFFFFFF0
        assert 255 * ldt * 2 + (k + 63) * 2 <= 0xFFFFFFF0
        # dz and its transpose: 2^27 values and a line a row, or 1024 words and the rounding
        assert r * piece <= max(1 << 27, 1024 * r) + 256 * r
