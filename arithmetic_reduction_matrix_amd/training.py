"""What a training step needs beside the row norms and the product: layer norm with
its gradients, dropout, and the loss of rows against a vocabulary: the binding of
those entry points of ``include/armx.h``.

The conventions of ``layer.py`` hold: matrices are 2-D with contiguous rows that start
at multiples of 16 bytes, calls run on the current stream of the inputs' device and
record no autograd graph (each has its gradients' call), and a tensor given for a
result counts as written in place.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import Config, _event_handle, lib
from .layer import _TYPES, _binding, _done

__all__ = ["dropout_rows", "layer_norm_rows", "layer_norm_rows_backward", "cross_entropy_rows",
           "cross_entropy_rows_backward", "Dropout", "LayerNorm", "LayerNormGrads",
           "CrossEntropy", "CrossEntropyGrads"]


class Dropout(NamedTuple):
    """A dropout of ``p`` (0 to 1, in steps of 2^-16), whose mask is a function of
    ``seed``, of ``offset + step`` and of the place in the matrix, and is never stored:
    the same Dropout in a backward call means the same mask.

    Places in a model that shall be dropped out unlike each other need offsets of their
    own.  ``step`` is an int64 tensor of one value on the inputs' device (or None), read
    when the kernel runs, so that a captured graph can advance it from one replay to the
    next (behind the backward pass, which reads it too).  ``first_row`` is the place of
    row 0 in a matrix that is taken in parts."""
    p: float
    seed: int
    offset: int = 0
    step: torch.Tensor | None = None
    first_row: int = 0


class LayerNorm(NamedTuple):
    """``out``; ``sum`` = what was normalised (None where that is x); ``mean`` and
    ``inv_std`` of every row (None unless kept)."""
    out: torch.Tensor
    sum: torch.Tensor | None
    mean: torch.Tensor | None
    inv_std: torch.Tensor | None


class LayerNormGrads(NamedTuple):
    """Gradients of a norm's input, weight and bias, and of its residual (None without a
    dropout: then ``dx`` is that too)."""
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: torch.Tensor
    dresidual: torch.Tensor | None


class CrossEntropy(NamedTuple):
    """float32 ``loss`` of every row and ``lse``, the log of its sum of exponentials."""
    loss: torch.Tensor
    lse: torch.Tensor


class CrossEntropyGrads(NamedTuple):
    """Gradients of a loss's hidden states and of its weight (None if not wanted)."""
    dx: torch.Tensor | None
    dweight: torch.Tensor | None


class _DropoutArgs(ctypes.Structure):
    """Mirror of ``armx_dropout``."""

    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step", ctypes.c_void_p), ("first_row", ctypes.c_uint64)]


_vp, _sz, _ci, _cf = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
_cfgp, _dropp = ctypes.POINTER(Config), ctypes.POINTER(_DropoutArgs)
lib.dropout_rows.argtypes = [_vp, _sz, _vp, _sz, _ci, _sz, _sz, _dropp, _vp, _sz, _cfgp, _vp]
lib.layer_norm_rows.argtypes = [_vp, _sz, _vp, _sz, _vp, _vp, _ci, _sz, _sz, _cf, _dropp, _vp, _sz,
                                _vp, _sz, _vp, _vp, _cfgp, _vp]
lib.layer_norm_rows_backward.argtypes = [_vp, _sz, _vp, _sz, _vp, _vp, _vp, _vp, _sz, _ci, _sz,
                                         _sz, _dropp, _vp, _sz, _vp, _sz, _vp, _vp, _vp, _sz,
                                         _cfgp, _vp]
_i64 = ctypes.c_int64
lib.cross_entropy_rows.argtypes = [_vp, _sz, _vp, _sz, _vp, _ci, _sz, _sz, _sz, _i64, _vp, _vp,
                                   _vp, _sz, _cfgp, _vp]
lib.cross_entropy_rows_backward.argtypes = [_vp, _vp, _sz, _vp, _sz, _vp, _vp, _ci, _sz, _sz, _sz,
                                            _i64, _vp, _sz, _vp, _sz, _ci, _vp, _sz, _cfgp, _vp]
lib.armx_cross_entropy_workspace_bytes.argtypes = [_sz, _sz, _sz]
lib.armx_cross_entropy_backward_workspace_bytes.argtypes = [_sz, _sz, _sz, _ci, _ci]
for _f in (lib.dropout_rows, lib.layer_norm_rows, lib.layer_norm_rows_backward,
           lib.cross_entropy_rows, lib.cross_entropy_rows_backward):
    _f.restype = ctypes.c_int
for _f in (lib.armx_cross_entropy_workspace_bytes,
           lib.armx_cross_entropy_backward_workspace_bytes):
    _f.restype = _sz


def dropout_rows(x: torch.Tensor, dropout: Dropout, *, residual: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, start_event=None,
                 stop_event=None) -> torch.Tensor:
    """``x`` (float16 or bfloat16) with each value dropped with the probability
    ``dropout.p`` and the others multiplied by 1 / (1 - p), plus ``residual``, rounded
    once.  The gradient of x is the same call on the result's gradient without a
    residual.  ``out`` may be ``x`` or ``residual``."""
    return _done(_binding.dropout_rows(x, dropout, residual, out, _event_handle(start_event),
                                       _event_handle(stop_event)), "dropout_rows", tuple)[0]


def layer_norm_rows(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *,
                    residual: torch.Tensor | None = None, dropout: Dropout | None = None,
                    eps: float = 1e-5, keep_stats: bool = False,
                    out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                    start_event=None, stop_event=None) -> LayerNorm:
    """Mean and variance norm of every row of ``dropout(x) + residual`` (float16 or
    bfloat16, rounded once and returned as ``sum``), times ``weight`` plus ``bias``.

    ``keep_stats`` returns the mean and 1 / standard deviation of every row (float32),
    which ``layer_norm_rows_backward`` takes.  ``out`` and ``sum_out`` may each be ``x``
    or ``residual`` themselves, not both the same one."""
    return _done(_binding.layer_norm_rows(x, weight, bias, residual, dropout, eps, keep_stats, out,
                                          sum_out, _event_handle(start_event),
                                          _event_handle(stop_event)),
                 "layer_norm_rows", LayerNorm)


def layer_norm_rows_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                             mean: torch.Tensor, inv_std: torch.Tensor, *,
                             dsum: torch.Tensor | None = None, dropout: Dropout | None = None,
                             out: torch.Tensor | None = None,
                             dresidual: torch.Tensor | None = None,
                             dweight: torch.Tensor | None = None,
                             dbias: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, start_event=None,
                             stop_event=None) -> LayerNormGrads:
    """Gradients of ``layer_norm_rows``: ``dy`` is the gradient of its result, ``h`` what
    was normalised (its ``sum``, or ``x``), ``mean`` and ``inv_std`` as it returned them,
    ``dsum`` the gradient that reaches ``sum`` from elsewhere, ``dropout`` as it was
    given.  Returns dx, dweight and dbias (float32) and, with a dropout, dresidual; dx is
    the gradient of x and of residual alike without one.  ``out`` receives dx; it and
    ``dresidual`` may each be ``dy`` or ``dsum``, not both the same one.  Without
    ``workspace`` one is taken from the allocator for this call."""
    return _done(_binding.layer_norm_rows_backward(dy, h, weight, mean, inv_std, dsum, dropout,
                                                   out, dresidual, dweight, dbias, workspace,
                                                   _event_handle(start_event),
                                                   _event_handle(stop_event)),
                 "layer_norm_rows_backward", LayerNormGrads)


def cross_entropy_rows(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                       ignore_index: int = -100, loss: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       start_event=None, stop_event=None) -> CrossEntropy:
    """Softmax cross entropy of every row of ``x`` (rows, cols; float16 or bfloat16)
    against the vocabulary of ``weight`` (vocab, cols): the loss of the logits
    ``x @ weight.T``, which are never stored, at ``targets`` (int64), and the log of their
    sums of exponentials, which ``cross_entropy_rows_backward`` takes (both float32).

    Rows whose target is ``ignore_index`` have loss 0 (the mean is ``loss.sum()`` over the
    count of the others); another target outside the vocabulary gives NaN.  A row's loss
    depends on that row and the weight only."""
    return _done(_binding.cross_entropy_rows(x, weight, targets, ignore_index, loss, lse,
                                             workspace, _event_handle(start_event),
                                             _event_handle(stop_event)),
                 "cross_entropy_rows", CrossEntropy)


def cross_entropy_rows_backward(dloss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                                targets: torch.Tensor, lse: torch.Tensor, *,
                                ignore_index: int = -100, need_dx: bool = True,
                                need_dweight: bool = True, out: torch.Tensor | None = None,
                                dweight: torch.Tensor | None = None,
                                dweight_dtype: torch.dtype | None = None,
                                workspace: torch.Tensor | None = None, start_event=None,
                                stop_event=None) -> CrossEntropyGrads:
    """Gradients of ``cross_entropy_rows``: ``dloss`` (float32) is the gradient of every
    row's loss, ``lse`` as it returned them.  Returns dx (of x's type; ``out`` receives
    it) and dweight (x's type, or float32 by ``dweight_dtype`` or by ``dweight``), each
    None if not wanted.  The logits are made again, a piece of the vocabulary at a time, and
    their gradients enter both products as values of x's type: of more than 128 rows, a row
    of dweight that one token alone makes has the accuracy of that type, as float32 too;
    without ``workspace`` one is taken from the allocator for this call (about 0.7 GB of
    pieces and transposes at 4096 rows of 4096 values)."""
    code = None if dweight_dtype is None else _TYPES.get(dweight_dtype, 3)
    return _done(_binding.cross_entropy_rows_backward(dloss, x, weight, targets, lse,
                                                      ignore_index, need_dx, need_dweight, out,
                                                      dweight, code, workspace,
                                                      _event_handle(start_event),
                                                      _event_handle(stop_event)),
                 "cross_entropy_rows_backward", CrossEntropyGrads)
