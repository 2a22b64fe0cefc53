"""The library without the module of the layer calls: a binding that does not compile, or
does not load, leaves libarmx.so and the sums as they are."""
import importlib.util
import os
import subprocess
import sys

import pytest

import arithmetic_reduction_matrix_amd as armx

PKG = os.path.dirname(armx.LIB_PATH)
NAME = os.path.basename(PKG)


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """_build.py with its outputs in a folder of their own and commands that only write
    their output; those whose text has one of `failing` in it fail."""
    spec = importlib.util.spec_from_file_location("_build_under_test",
                                                  os.path.join(PKG, "_build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.failing, mod.ran = [], []
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "objects"))
    for name in ("LIB", "PROBE_LIB", "BINDING"):
        monkeypatch.setattr(mod, name, str(tmp_path / os.path.basename(getattr(mod, name))))
    monkeypatch.setattr(mod, "_hipcc", lambda: "hipcc")

    def run(cmd, verbose):
        mod.ran.append(cmd)
        if any(f in part for f in mod.failing for part in cmd):
            raise RuntimeError("command failed: " + " ".join(cmd))
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(mod, "_run", run)
    return mod


def built(mod):
    return [os.path.exists(p) for p in (mod.LIB, mod.PROBE_LIB, mod.BINDING)]


def test_everything_is_built(builder):
    assert builder.build() == builder.LIB and built(builder) == [True, True, True]
    outputs = [cmd[-1] for cmd in builder.ran if "-shared" in cmd]
    assert outputs[0] == builder.LIB + ".tmp" and outputs[-1] == builder.BINDING + ".tmp"
    sources = builder.HIP_SOURCES + builder.HOST_SOURCES + builder.PROBE_SOURCES
    compiled = [os.path.basename(cmd[cmd.index("-c") + 1]) for cmd in builder.ran if "-c" in cmd]
    assert sorted(compiled) == sorted(sources + builder.BINDING_SOURCES)


@pytest.mark.parametrize("failing", ["binding.cpp", "-ltorch_python"])
def test_a_binding_that_does_not_build_leaves_the_libraries(builder, failing):
    builder.failing.append(failing)
    with pytest.raises(RuntimeError, match=failing):
        builder.build()
    assert built(builder) == [True, True, False]


def test_a_kernel_that_does_not_build_raises(builder):
    builder.failing.append("norm_kernels.hip")
    with pytest.raises(RuntimeError, match="norm_kernels"):
        builder.build()
    assert built(builder) == [False, False, False]


def test_the_libraries_need_no_pytorch(builder, monkeypatch, capsys):
    monkeypatch.setattr(builder.importlib.util, "find_spec", lambda name: None)
    assert builder.build() == builder.LIB
    assert built(builder) == [True, True, False]
    assert "PyTorch is not installed" in capsys.readouterr().err


CHILD = f"""
import torch
import {NAME} as armx
x = torch.zeros(4, 16, dtype=torch.float16)
assert armx.workspace_bytes(armx.OP_SUM, 1 << 28) > 0
for call in (lambda: armx.reduce_sum(x), lambda: armx.reduce_rows(x)):
    try:
        call()
    except ValueError as e:          # as ever: not on a GPU
        assert "GPU" in str(e)
    else:
        raise SystemExit("no error")
s = torch.ones(4)
q = torch.zeros(4, 16, dtype=torch.int8)
for name, args in (("rms_norm_rows", (x, x[0])), ("rms_norm_rows_int8", (x, x[0])),
                   ("rms_norm_rows_backward", (x, x, x[0], s)), ("quantize_rows_int8", (x,)),
                   ("matmul_int8", (q, s, q, s))):
    try:
        getattr(armx, name)(*args)
    except ImportError as e:
        assert name in str(e) and "_binding.so does not load" in str(e) and e.__cause__, e
    else:
        raise SystemExit(name)
print("ok")
"""


@pytest.mark.parametrize("binding", ["missing", "broken"])
def test_the_sums_work_where_the_binding_does_not_load(tmp_path, binding):
    pkg = tmp_path / NAME
    pkg.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py") or f == "libarmx.so":
            os.symlink(os.path.join(PKG, f), pkg / f)
    if binding == "broken":
        (pkg / "_binding.so").write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
