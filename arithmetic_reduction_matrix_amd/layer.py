"""Norms of rows, rows as 8-bit codes, and the product of codes: the binding of
the layer entry points of ``include/armx.h``.

What a transformer layer does around a matrix product, with the guarantees of
this library's sums: a row's result depends on that row only (batch
invariance), codes are those of the exact quotient, and products of codes are
summed exactly.  Matrices are 2-D with contiguous rows (``stride(1) == 1``);
rows of 16-bit values start at multiples of 16 bytes (a row pitch that is a
multiple of 8) and rows of codes too (a multiple of 16).  Matrices of both made here
have such a pitch, so that one call's result is the next one's input, and results of
odd width are not contiguous (float32 products are).  Calls run
on the current stream of the inputs' device and record no autograd graph:
``rms_norm_rows_backward`` gives the norm's gradients.  A tensor given for a result
counts as written in place, so that a backward pass which saved its old values raises.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch   # before the module that is linked against it

from . import Config, _check, _event_handle, lib


class _NotLoaded:
    """Stands for the module of the calls where it does not load: the sums do not need
    it, so only these calls raise."""

    def __init__(self, cause: ImportError):
        self._cause = cause

    def __getattr__(self, name: str):
        raise ImportError(
            f"{name}: arithmetic_reduction_matrix_amd/_binding.so does not load "
            f"({self._cause}): build it with `python arithmetic_reduction_matrix_amd/_build.py` "
            "(or __graft_entry__.build())") from self._cause


try:
    from . import _binding
except ImportError as _cause:
    _binding = _NotLoaded(_cause)

__all__ = ["rms_norm_rows", "rms_norm_rows_int8", "rms_norm_rows_backward",
           "quantize_rows_int8", "matmul_int8", "RmsNorm", "RmsNormInt8", "RmsNormGrads",
           "RowCodes"]


class RmsNorm(NamedTuple):
    """``out``; ``sum`` = x + residual (None without one); ``inv_rms`` (None unless kept)."""
    out: torch.Tensor
    sum: torch.Tensor | None
    inv_rms: torch.Tensor | None


class RmsNormInt8(NamedTuple):
    """int8 ``codes``, a float32 scale per row, ``sum`` = x + residual (None without one)."""
    codes: torch.Tensor
    scales: torch.Tensor
    sum: torch.Tensor | None


class RowCodes(NamedTuple):
    """int8 ``codes`` and a float32 scale per row."""
    codes: torch.Tensor
    scales: torch.Tensor


class RmsNormGrads(NamedTuple):
    """Gradients of a norm's input (and residual) and of its weight."""
    dx: torch.Tensor
    dweight: torch.Tensor


_vp, _sz, _ci, _cf = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
_cfgp = ctypes.POINTER(Config)
lib.rms_norm_rows.argtypes = [_vp, _sz, _vp, _sz, _vp, _ci, _sz, _sz, _cf, _vp, _sz, _vp, _sz,
                              _vp, _cfgp, _vp]
lib.rms_norm_rows_int8.argtypes = [_vp, _sz, _vp, _sz, _vp, _ci, _sz, _sz, _cf, _vp, _sz, _vp,
                                   _vp, _sz, _cfgp, _vp]
lib.quantize_rows_int8.argtypes = [_vp, _sz, _ci, _sz, _sz, _vp, _sz, _vp, _cfgp, _vp]
lib.rms_norm_rows_backward.argtypes = [_vp, _sz, _vp, _sz, _vp, _vp, _vp, _sz, _ci, _sz, _sz,
                                       _vp, _sz, _vp, _vp, _sz, _cfgp, _vp]
lib.matmul_int8.argtypes = [_vp, _sz, _vp, _vp, _sz, _vp, _vp, _sz, _sz, _sz, _vp, _sz, _ci,
                            _cfgp, _vp]
for _f in (lib.rms_norm_rows, lib.rms_norm_rows_int8, lib.quantize_rows_int8,
           lib.rms_norm_rows_backward, lib.matmul_int8):
    _f.restype = ctypes.c_int

_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_new = tuple.__new__


def _done(result, name: str, kind):
    """The named tuple of a call's results; a status raises."""
    if type(result) is int:
        _check(result, name)
    return _new(kind, result)


def rms_norm_rows(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None,
                  eps: float = 1e-6, keep_inv_rms: bool = False,
                  out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                  start_event=None, stop_event=None) -> RmsNorm:
    """Root-mean-square norm of every row of ``x + residual`` (float16 or
    bfloat16, the sum rounded once and returned), times ``weight``.

    ``keep_inv_rms`` returns 1 / rms of every row (float32), which
    ``rms_norm_rows_backward`` takes.  ``out`` and ``sum_out`` may each be ``x`` or
    ``residual`` themselves, not both the same one."""
    return _done(_binding.rms_norm_rows(x, weight, residual, eps, keep_inv_rms, out, None, sum_out,
                                        _event_handle(start_event), _event_handle(stop_event)),
                 "rms_norm_rows", RmsNorm)


def rms_norm_rows_int8(x: torch.Tensor, weight: torch.Tensor, *,
                       residual: torch.Tensor | None = None, eps: float = 1e-6,
                       out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                       sum_out: torch.Tensor | None = None, start_event=None,
                       stop_event=None) -> RmsNormInt8:
    """``rms_norm_rows`` with its result as int8 codes and one scale per row
    (``codes * scales[:, None]`` stands for the norm), as ``matmul_int8`` takes
    them.  ``out`` receives the codes."""
    return _done(_binding.rms_norm_rows_int8(x, weight, residual, eps, None, out, scales, sum_out,
                                             _event_handle(start_event),
                                             _event_handle(stop_event)),
                 "rms_norm_rows_int8", RmsNormInt8)


def quantize_rows_int8(x: torch.Tensor, *, out: torch.Tensor | None = None,
                       scales: torch.Tensor | None = None, start_event=None,
                       stop_event=None) -> RowCodes:
    """Rows of a float16 or bfloat16 matrix as int8 codes with one scale each:
    ``codes`` is 127 x / max|x| of the row, rounded half to even, and ``scales``
    max|x| / 127.  A linear layer's weight (one output channel per row) becomes
    ``matmul_int8``'s second operand."""
    return _done(_binding.quantize_rows_int8(x, out, scales, _event_handle(start_event),
                                             _event_handle(stop_event)),
                 "quantize_rows_int8", RowCodes)


def rms_norm_rows_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                           inv_rms: torch.Tensor, *, dsum: torch.Tensor | None = None,
                           out: torch.Tensor | None = None,
                           dweight: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, start_event=None,
                           stop_event=None) -> RmsNormGrads:
    """Gradients of ``rms_norm_rows``: ``dy`` is the gradient of its result,
    ``h`` what was normalised (its ``sum``, or ``x`` without a residual),
    ``inv_rms`` as it returned them, ``dsum`` the gradient that reaches ``sum``
    from elsewhere.  Returns dx (the gradient of x and of residual alike) and
    dweight (float32).  ``out`` receives dx and may be ``dy`` or ``dsum``.
    Without ``workspace`` one is taken from the allocator for this call."""
    return _done(_binding.rms_norm_rows_backward(dy, h, weight, inv_rms, dsum, out, dweight,
                                                 workspace, _event_handle(start_event),
                                                 _event_handle(stop_event)),
                 "rms_norm_rows_backward", RmsNormGrads)


def matmul_int8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                b_scales: torch.Tensor, *, bias: torch.Tensor | None = None,
                out: torch.Tensor | None = None, dtype: torch.dtype = torch.float16,
                start_event=None, stop_event=None) -> torch.Tensor:
    """``(a @ b.T) * a_scales[:, None] * b_scales + bias`` of int8 codes ``a``
    (m, k) and ``b`` (n, k), one float32 scale per row of either, as a (m, n)
    tensor of ``dtype`` (float16, bfloat16 or float32; ``out``'s if given;
    ``bias`` has it too).  The sum over k (at most 131071) is exact, so a
    result depends on its row and column only."""
    r = _binding.matmul_int8(a, a_scales, b, b_scales, bias, out, _TYPES.get(dtype, 3),
                             _event_handle(start_event), _event_handle(stop_event))
    if type(r) is int:
        _check(r, "matmul_int8")
    return r[0]
