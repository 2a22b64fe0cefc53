"""Norms of rows, rows as 8-bit codes, and the product of codes: the binding of
the layer entry points of ``include/armx.h``.

What a transformer layer does around a matrix product, with the guarantees of
this library's sums: a row's result depends on that row only (batch
invariance), codes are those of the exact quotient, and products of codes are
summed exactly.  Matrices are 2-D with contiguous rows (``stride(1) == 1``);
rows of 16-bit values start at multiples of 16 bytes (a row pitch that is a
multiple of 8) and rows of codes too (a multiple of 16).  Matrices made here
have such a pitch, so results of odd width are views of wider ones.  Calls run
on the current stream of the inputs' device and record no autograd graph:
``rms_norm_rows_backward`` gives the norm's gradients.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import OP_RMS_BACKWARD, Config, _check, _config, _on_device, lib

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
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _first(x, name: str, what: str, dtypes) -> None:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: {what} must be a torch.Tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name}: {what} must be {' or '.join(str(d) for d in dtypes)}, "
                        f"got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name}: {what} must be on a GPU (HIP) device")
    if x.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D {what}, got {x.dim()}-D")


def _matrix(t, name: str, what: str, shape, dtype, device) -> tuple[int | None, int]:
    """Pointer and row pitch of a matrix that must have this shape and type."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape \
            or t.device != device:
        raise ValueError(f"{name}: {what} must be a {tuple(shape)} {dtype} tensor on {device}")
    rows, cols = shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows of {what} must be contiguous (stride(1) == 1)")
    return t.data_ptr() or None, t.stride(0) if rows > 1 else cols


def _vector(t, name: str, what: str, n: int, dtype, device) -> int | None:
    """Pointer of n contiguous values."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != n \
            or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be {n} contiguous {dtype} values on {device}")
    return t.data_ptr() or None


def _rows_like(rows: int, cols: int, multiple: int, dtype, device) -> torch.Tensor:
    """An uninitialised matrix whose rows start at multiples of `multiple` values."""
    pitch = -(-cols // multiple) * multiple
    m = torch.empty((rows, pitch), dtype=dtype, device=device)
    return m if pitch == cols else m[:, :cols]


def _events(start_event, stop_event):
    if start_event is None and stop_event is None:
        return None
    return ctypes.byref(_config(start_event=start_event, stop_event=stop_event))


def _norm_inputs(x, weight, residual, sum_out, name):
    _first(x, name, "x", (torch.float16, torch.bfloat16))
    shape, dtype, dev = x.shape, x.dtype, x.device
    xp, ldx = _matrix(x, name, "x", shape, dtype, dev)
    wp = _vector(weight, name, "weight", shape[1], dtype, dev)
    if residual is None:
        if sum_out is not None:
            raise ValueError(f"{name}: sum_out goes with a residual")
        return xp, ldx, wp, None, 0, None, None, 0
    rp, ldr = _matrix(residual, name, "residual", shape, dtype, dev)
    if sum_out is None:
        sum_out = _rows_like(*shape, 8, dtype, dev)
    sp, lds = _matrix(sum_out, name, "sum_out", shape, dtype, dev)
    return xp, ldx, wp, rp, ldr, sum_out, sp, lds


def rms_norm_rows(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None,
                  eps: float = 1e-6, keep_inv_rms: bool = False,
                  out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                  start_event=None, stop_event=None) -> RmsNorm:
    """Root-mean-square norm of every row of ``x + residual`` (float16 or
    bfloat16, the sum rounded once and returned), times ``weight``.

    ``keep_inv_rms`` returns 1 / rms of every row (float32), which
    ``rms_norm_rows_backward`` takes.  ``out`` and ``sum_out`` may be ``x`` or
    ``residual`` themselves."""
    name = "rms_norm_rows"
    xp, ldx, wp, rp, ldr, sum_out, sp, lds = _norm_inputs(x, weight, residual, sum_out, name)
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = _rows_like(rows, cols, 8, x.dtype, dev)
    op, ldo = _matrix(out, name, "out", x.shape, x.dtype, dev)
    inv = torch.empty(rows, dtype=torch.float32, device=dev) if keep_inv_rms else None
    with _on_device(dev):
        st = lib.rms_norm_rows(xp, ldx, rp, ldr, wp, _TYPES[x.dtype], rows, cols, eps, op, ldo,
                               sp, lds, inv.data_ptr() or None if keep_inv_rms else None,
                               _events(start_event, stop_event), _stream_of(dev.index))
    _check(st, name)
    return RmsNorm(out, sum_out, inv)


def rms_norm_rows_int8(x: torch.Tensor, weight: torch.Tensor, *,
                       residual: torch.Tensor | None = None, eps: float = 1e-6,
                       out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                       sum_out: torch.Tensor | None = None, start_event=None,
                       stop_event=None) -> RmsNormInt8:
    """``rms_norm_rows`` with its result as int8 codes and one scale per row
    (``codes * scales[:, None]`` stands for the norm), as ``matmul_int8`` takes
    them.  ``out`` receives the codes."""
    name = "rms_norm_rows_int8"
    xp, ldx, wp, rp, ldr, sum_out, sp, lds = _norm_inputs(x, weight, residual, sum_out, name)
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = _rows_like(rows, cols, 16, torch.int8, dev)
    op, ldo = _matrix(out, name, "out", x.shape, torch.int8, dev)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=dev)
    cp = _vector(scales, name, "scales", rows, torch.float32, dev)
    with _on_device(dev):
        st = lib.rms_norm_rows_int8(xp, ldx, rp, ldr, wp, _TYPES[x.dtype], rows, cols, eps, op,
                                    ldo, cp, sp, lds, _events(start_event, stop_event),
                                    _stream_of(dev.index))
    _check(st, name)
    return RmsNormInt8(out, scales, sum_out)


def quantize_rows_int8(x: torch.Tensor, *, out: torch.Tensor | None = None,
                       scales: torch.Tensor | None = None, start_event=None,
                       stop_event=None) -> RowCodes:
    """Rows of a float16 or bfloat16 matrix as int8 codes with one scale each:
    ``codes`` is 127 x / max|x| of the row, rounded half to even, and ``scales``
    max|x| / 127.  A linear layer's weight (one output channel per row) becomes
    ``matmul_int8``'s second operand."""
    name = "quantize_rows_int8"
    _first(x, name, "x", (torch.float16, torch.bfloat16))
    rows, cols = x.shape
    dev = x.device
    xp, ldx = _matrix(x, name, "x", x.shape, x.dtype, dev)
    if out is None:
        out = _rows_like(rows, cols, 16, torch.int8, dev)
    op, ldo = _matrix(out, name, "out", x.shape, torch.int8, dev)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=dev)
    cp = _vector(scales, name, "scales", rows, torch.float32, dev)
    with _on_device(dev):
        st = lib.quantize_rows_int8(xp, ldx, _TYPES[x.dtype], rows, cols, op, ldo, cp,
                                    _events(start_event, stop_event), _stream_of(dev.index))
    _check(st, name)
    return RowCodes(out, scales)


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
    name = "rms_norm_rows_backward"
    _first(dy, name, "dy", (torch.float16, torch.bfloat16))
    shape, dtype, dev = dy.shape, dy.dtype, dy.device
    rows, cols = shape
    yp, ldy = _matrix(dy, name, "dy", shape, dtype, dev)
    hp, ldh = _matrix(h, name, "h", shape, dtype, dev)
    wp = _vector(weight, name, "weight", cols, dtype, dev)
    ip = _vector(inv_rms, name, "inv_rms", rows, torch.float32, dev)
    dp, ldd = (None, 0) if dsum is None else _matrix(dsum, name, "dsum", shape, dtype, dev)
    if out is None:
        out = _rows_like(rows, cols, 8, dtype, dev)
    op, ldo = _matrix(out, name, "out", shape, dtype, dev)
    if dweight is None:
        dweight = torch.empty(cols, dtype=torch.float32, device=dev)
    gp = _vector(dweight, name, "dweight", cols, torch.float32, dev)
    with _on_device(dev):
        if workspace is None:
            need = lib.armx_workspace_bytes(OP_RMS_BACKWARD, rows, cols, None)
            # from the allocator, which knows streams and graph captures: it
            # needs no zeros, so nothing is gained by keeping one
            workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"{name}: workspace must be a contiguous tensor on {dev}")
        ws, ws_bytes = (None, 0) if workspace is None else (
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
        st = lib.rms_norm_rows_backward(yp, ldy, hp, ldh, wp, ip, dp, ldd, _TYPES[dtype], rows,
                                        cols, op, ldo, gp, ws, ws_bytes,
                                        _events(start_event, stop_event), _stream_of(dev.index))
    _check(st, name)
    return RmsNormGrads(out, dweight)


def _code_rows(t, name: str, what: str, rows: int, k: int, dev) -> tuple[int | None, int]:
    """Pointer and pitch of a matrix of codes whose rows can be read in pieces
    of 16 to their end."""
    p, ld = _matrix(t, name, what, (rows, k), torch.int8, dev)
    if k % 16 and rows and (ld % 16 == 0 or rows == 1):   # else the call reports the pitch
        end = t.storage_offset() + (rows - 1) * ld + -(-k // 16) * 16
        if end > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: the last row of {what} must be readable to a multiple "
                             "of 16 codes (allocate rows with a pitch that is one)")
    return p, ld


def matmul_int8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                b_scales: torch.Tensor, *, bias: torch.Tensor | None = None,
                out: torch.Tensor | None = None, dtype: torch.dtype = torch.float16,
                start_event=None, stop_event=None) -> torch.Tensor:
    """``(a @ b.T) * a_scales[:, None] * b_scales + bias`` of int8 codes ``a``
    (m, k) and ``b`` (n, k), one float32 scale per row of either, as a (m, n)
    tensor of ``dtype`` (float16, bfloat16 or float32; ``out``'s if given;
    ``bias`` has it too).  The sum over k (at most 131071) is exact, so a
    result depends on its row and column only."""
    name = "matmul_int8"
    _first(a, name, "a", (torch.int8,))
    _first(b, name, "b", (torch.int8,))
    dev = a.device
    m, k = a.shape
    n = b.shape[0]
    ap, lda = _code_rows(a, name, "a", m, k, dev)
    bp, ldb = _code_rows(b, name, "b", n, k, dev)
    asp = _vector(a_scales, name, "a_scales", m, torch.float32, dev)
    bsp = _vector(b_scales, name, "b_scales", n, torch.float32, dev)
    if out is None:
        if dtype not in _TYPES:
            raise TypeError(f"{name}: dtype must be float16, bfloat16 or float32, got {dtype}")
        out = torch.empty((m, n), dtype=dtype, device=dev)
        op, ldo = out.data_ptr() or None, n
    else:
        dtype = out.dtype if isinstance(out, torch.Tensor) else None
        if dtype not in _TYPES:
            raise TypeError(f"{name}: out must be a float16, bfloat16 or float32 tensor")
        op, ldo = _matrix(out, name, "out", (m, n), dtype, dev)
    biasp = None if bias is None else _vector(bias, name, "bias", n, dtype, dev)
    with _on_device(dev):
        st = lib.matmul_int8(ap, lda, asp, bp, ldb, bsp, biasp, m, n, k, op, ldo, _TYPES[dtype],
                             _events(start_event, stop_event), _stream_of(dev.index))
    _check(st, name)
    return out
