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
_HALVES = (torch.float16, torch.bfloat16)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

# A call's kernel may take no longer than its Python does, so the checks below
# read each tensor's properties once, compare dtypes by identity and devices by
# index, and check nothing of the matrices made here.


def _first(x, name: str, what: str, dtypes):
    """Shape, dtype and device index of the operand the others must match."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: {what} must be a torch.Tensor")
    dtype = x.dtype
    if dtype not in dtypes:
        raise TypeError(f"{name}: {what} must be {' or '.join(str(d) for d in dtypes)}, "
                        f"got {dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name}: {what} must be on a GPU (HIP) device")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a 2-D {what}, got {len(shape)}-D")
    return shape, dtype, x.get_device()


def _matrix(t, name: str, what: str, shape, dtype, dev: int) -> tuple[int | None, int]:
    """Pointer and row pitch of a matrix that must have this shape and type."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape \
            or t.get_device() != dev:
        raise ValueError(f"{name}: {what} must be a {tuple(shape)} {dtype} tensor on cuda:{dev}")
    rows, cols = shape
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: rows of {what} must be contiguous (stride(1) == 1)")
    return t.data_ptr() or None, pitch if rows > 1 else cols


def _vector(t, name: str, what: str, n: int, dtype, dev: int) -> int | None:
    """Pointer of n contiguous values."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.numel() != n \
            or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be {n} contiguous {dtype} values on cuda:{dev}")
    return t.data_ptr() or None


def _rows_like(x, rows: int, cols: int, multiple: int, dtype) -> tuple:
    """An uninitialised matrix on x's device whose rows start at multiples of
    `multiple` values; its pointer and pitch."""
    pitch = -(-cols // multiple) * multiple
    m = x.new_empty((rows, pitch), dtype=dtype)
    return m if pitch == cols else m[:, :cols], m.data_ptr() or None, pitch


def _call(fn, name: str, dev: int, args: tuple, start_event, stop_event) -> None:
    """fn(*args, cfg, stream) on the current stream of device `dev`."""
    cfg = None
    if start_event is not None or stop_event is not None:
        cfg = ctypes.byref(_config(start_event=start_event, stop_event=stop_event))
    if _current_device() == dev:
        st = fn(*args, cfg, _stream_of(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, cfg, _stream_of(dev))
    if st:
        _check(st, name)


def _norm_inputs(x, weight, residual, sum_out, name):
    shape, dtype, dev = _first(x, name, "x", _HALVES)
    xp, ldx = _matrix(x, name, "x", shape, dtype, dev)
    wp = _vector(weight, name, "weight", shape[1], dtype, dev)
    if residual is None:
        if sum_out is not None:
            raise ValueError(f"{name}: sum_out goes with a residual")
        return shape, dtype, dev, xp, ldx, wp, None, 0, None, None, 0
    rp, ldr = _matrix(residual, name, "residual", shape, dtype, dev)
    if sum_out is None:
        sum_out, sp, lds = _rows_like(x, *shape, 8, dtype)
    else:
        sp, lds = _matrix(sum_out, name, "sum_out", shape, dtype, dev)
    return shape, dtype, dev, xp, ldx, wp, rp, ldr, sum_out, sp, lds


def _codes_out(x, shape, out, scales, name, dev):
    """Codes and scales with their pointers and the codes' pitch, made if not given."""
    rows, cols = shape
    if out is None:
        out, op, ldo = _rows_like(x, rows, cols, 16, torch.int8)
    else:
        op, ldo = _matrix(out, name, "out", shape, torch.int8, dev)
    if scales is None:
        scales = x.new_empty(rows, dtype=torch.float32)
        cp = scales.data_ptr() or None
    else:
        cp = _vector(scales, name, "scales", rows, torch.float32, dev)
    return out, op, ldo, scales, cp


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
    shape, dtype, dev, xp, ldx, wp, rp, ldr, sum_out, sp, lds = _norm_inputs(
        x, weight, residual, sum_out, name)
    rows, cols = shape
    if out is None:
        out, op, ldo = _rows_like(x, rows, cols, 8, dtype)
    else:
        op, ldo = _matrix(out, name, "out", shape, dtype, dev)
    inv = ip = None
    if keep_inv_rms:
        inv = x.new_empty(rows, dtype=torch.float32)
        ip = inv.data_ptr() or None
    _call(lib.rms_norm_rows, name, dev, (xp, ldx, rp, ldr, wp, _TYPES[dtype], rows, cols, eps, op,
                                         ldo, sp, lds, ip), start_event, stop_event)
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
    shape, dtype, dev, xp, ldx, wp, rp, ldr, sum_out, sp, lds = _norm_inputs(
        x, weight, residual, sum_out, name)
    out, op, ldo, scales, cp = _codes_out(x, shape, out, scales, name, dev)
    _call(lib.rms_norm_rows_int8, name, dev,
          (xp, ldx, rp, ldr, wp, _TYPES[dtype], *shape, eps, op, ldo, cp, sp, lds), start_event,
          stop_event)
    return RmsNormInt8(out, scales, sum_out)


def quantize_rows_int8(x: torch.Tensor, *, out: torch.Tensor | None = None,
                       scales: torch.Tensor | None = None, start_event=None,
                       stop_event=None) -> RowCodes:
    """Rows of a float16 or bfloat16 matrix as int8 codes with one scale each:
    ``codes`` is 127 x / max|x| of the row, rounded half to even, and ``scales``
    max|x| / 127.  A linear layer's weight (one output channel per row) becomes
    ``matmul_int8``'s second operand."""
    name = "quantize_rows_int8"
    shape, dtype, dev = _first(x, name, "x", _HALVES)
    xp, ldx = _matrix(x, name, "x", shape, dtype, dev)
    out, op, ldo, scales, cp = _codes_out(x, shape, out, scales, name, dev)
    _call(lib.quantize_rows_int8, name, dev, (xp, ldx, _TYPES[dtype], *shape, op, ldo, cp),
          start_event, stop_event)
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
    shape, dtype, dev = _first(dy, name, "dy", _HALVES)
    rows, cols = shape
    yp, ldy = _matrix(dy, name, "dy", shape, dtype, dev)
    hp, ldh = _matrix(h, name, "h", shape, dtype, dev)
    wp = _vector(weight, name, "weight", cols, dtype, dev)
    ip = _vector(inv_rms, name, "inv_rms", rows, torch.float32, dev)
    dp, ldd = (None, 0) if dsum is None else _matrix(dsum, name, "dsum", shape, dtype, dev)
    if out is None:
        out, op, ldo = _rows_like(dy, rows, cols, 8, dtype)
    else:
        op, ldo = _matrix(out, name, "out", shape, dtype, dev)
    if dweight is None:
        dweight = dy.new_empty(cols, dtype=torch.float32)
        gp = dweight.data_ptr() or None
    else:
        gp = _vector(dweight, name, "dweight", cols, torch.float32, dev)
    if workspace is None:
        with _on_device(dy.device):
            need = lib.armx_workspace_bytes(OP_RMS_BACKWARD, rows, cols, None)
        # from the allocator, which knows streams and graph captures: it needs
        # no zeros, so nothing is gained by keeping one
        workspace = dy.new_empty(need, dtype=torch.uint8) if need else None
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be a contiguous tensor on cuda:{dev}")
    ws, ws_bytes = (None, 0) if workspace is None else (
        workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _call(lib.rms_norm_rows_backward, name, dev,
          (yp, ldy, hp, ldh, wp, ip, dp, ldd, _TYPES[dtype], rows, cols, op, ldo, gp, ws,
           ws_bytes), start_event, stop_event)
    return RmsNormGrads(out, dweight)


def _code_rows(t, name: str, what: str, shape, k: int, dev: int) -> tuple[int | None, int]:
    """Pointer and pitch of a matrix of codes whose rows can be read in pieces
    of 16 to their end."""
    rows = shape[0]
    if shape[1] != k:
        raise ValueError(f"{name}: {what} must have rows of {k} codes, as a has")
    p, ld = _matrix(t, name, what, shape, torch.int8, dev)
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
    shape, _, dev = _first(a, name, "a", (torch.int8,))
    m, k = shape
    ap, lda = _code_rows(a, name, "a", shape, k, dev)
    shape, _, _ = _first(b, name, "b", (torch.int8,))
    n = shape[0]
    bp, ldb = _code_rows(b, name, "b", shape, k, dev)
    asp = _vector(a_scales, name, "a_scales", m, torch.float32, dev)
    bsp = _vector(b_scales, name, "b_scales", n, torch.float32, dev)
    if out is not None:
        dtype = out.dtype if isinstance(out, torch.Tensor) else None
    type_ = _TYPES.get(dtype)
    if type_ is None:
        raise TypeError(f"{name}: the result is float16, bfloat16 or float32, not {dtype}")
    if out is None:
        out, ldo = a.new_empty((m, n), dtype=dtype), n
        op = out.data_ptr() or None
    else:
        op, ldo = _matrix(out, name, "out", (m, n), dtype, dev)
    biasp = None if bias is None else _vector(bias, name, "bias", n, dtype, dev)
    _call(lib.matmul_int8, name, dev, (ap, lda, asp, bp, ldb, bsp, biasp, m, n, k, op, ldo, type_),
          start_event, stop_event)
    return out
