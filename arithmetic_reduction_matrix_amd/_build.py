"""Builds libarmx.so (the HIP kernels and the C entry points) for gfx950,
_binding.so (the layer entry points for PyTorch tensors), and libarmx_probe.so (a
plain read stream, for measurement only).

Run ``python arithmetic_reduction_matrix_amd/_build.py`` or call ``build()`` (it imports
only the standard library, so it runs whether or not a library is built; the
binding is compiled against the headers of the installed PyTorch, and the libraries
need none).
Every source is compiled each time; objects go to ``_build/`` next to this
file and the library is written to ``libarmx.so`` in this package.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libarmx.so")
# measurement only: the plain read stream the reductions are compared with
PROBE_LIB = os.path.join(PKG, "libarmx_probe.so")
PROBE_SOURCES = ["read_probe.hip"]
# the layer entry points for PyTorch tensors (a CPython module)
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCES = ["binding.cpp"]

ARCH = "gfx950"
HIP_SOURCES = ["sum_kernels.hip", "fixed_kernels.hip", "rows_kernels.hip", "exact_kernels.hip",
               "rows_fixed_kernels.hip", "levels_kernels.hip", "short_rows_kernels.hip",
               "norm_kernels.hip", "matmul_int8_kernels.hip", "layer_norm_kernels.hip",
               "cross_entropy_kernels.hip", "cross_entropy_backward_kernels.hip"]
HOST_SOURCES = ["api.cpp", "api_layer.cpp", "plan.cpp"]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
          f"-I{INCLUDE}", f"-I{CSRC}"]
# packed fp32 instructions are kept out of the device code
DEVICE = [f"--offload-arch={ARCH}", "-fno-gpu-rdc", "-ffp-contract=off",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature and says so; that
    # warning is expected and not shown
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in p.stderr.splitlines() if noise not in l)
    if p.returncode != 0:
        raise RuntimeError(f"command failed ({p.returncode}): {' '.join(cmd)}\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def _torch_dir() -> str | None:
    """Where PyTorch is installed (found without importing it); None if it is not."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compiles every source and links libarmx.so; returns its path.

    libarmx.so needs no PyTorch and is linked before the binding's outcome counts: a
    binding that does not compile raises with the library in place, and without PyTorch
    there is none."""
    hipcc = _hipcc()
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(8, os.cpu_count() or 1)

    def compile_all(sources: list[str], flags: list[str]) -> tuple[list[str], list]:
        objs = [os.path.join(BUILD, src + ".o") for src in sources]
        return objs, [pool.submit(_run, [hipcc, *COMMON, *flags, "-c", os.path.join(CSRC, src),
                                         "-o", obj], verbose)
                      for src, obj in zip(sources, objs)]

    def link(out: str, objs: list[str], more: list[str]) -> None:
        tmp = out + ".tmp"
        _run([hipcc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, *more, "-o", tmp],
             verbose)
        os.replace(tmp, out)

    torch_dir = _torch_dir()
    hip = [*DEVICE, "-x", "hip"]
    with ThreadPoolExecutor(max_workers=jobs) as pool:
        if torch_dir is not None:   # first: it takes longest
            include = [os.path.join(torch_dir, "include"),
                       os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                       sysconfig.get_paths()["include"]]
            binding = compile_all(BINDING_SOURCES,
                                  [*(f"-isystem{d}" for d in include), "-DUSE_ROCM"])
        kernels = compile_all(HIP_SOURCES, hip)
        host = compile_all(HOST_SOURCES, [])
        probe = compile_all(PROBE_SOURCES, hip)
        for _, running in (kernels, host, probe):
            for r in running:
                r.result()
        link(LIB, kernels[0] + host[0], [])
        link(PROBE_LIB, probe[0], [])
        if torch_dir is None:
            print("PyTorch is not installed: _binding.so is not built", file=sys.stderr)
            return LIB
        for r in binding[1]:
            r.result()
        torch_lib = os.path.join(torch_dir, "lib")
        link(BINDING, binding[0],
             [f"-L{os.path.dirname(LIB)}", "-l:libarmx.so", f"-L{torch_lib}", "-ltorch_python",
              "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"])
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
