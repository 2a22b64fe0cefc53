"""Refusals and workspace sizes of the layer entry points, on the CPU: every
call here fails, or has nothing to do, before a device is touched."""
import ctypes

import pytest
import torch

import arithmetic_reduction_matrix_amd as armx

lib = armx.lib
P = 1 << 20     # an aligned address; never dereferenced
NAN = float("nan")


def cfg(**kw):
    return ctypes.byref(armx._config(**kw))


BAD_CONFIGS = [dict(block_threads=256), dict(chain_r=1), dict(grid_blocks=5), dict(plain=True)]


def norm(x=P, ldx=64, res=None, ldr=0, w=P, type=0, rows=4, cols=64, eps=1e-6, out=P, ldo=64,
         sum=None, lds=0, inv=None, c=None):
    return lib.rms_norm_rows(x, ldx, res, ldr, w, type, rows, cols, eps, out, ldo, sum, lds, inv,
                             c, None)


def norm8(x=P, ldx=64, res=None, ldr=0, w=P, type=0, rows=4, cols=64, eps=1e-6, codes=P, ldc=64,
          scales=P, sum=None, lds=0, c=None):
    return lib.rms_norm_rows_int8(x, ldx, res, ldr, w, type, rows, cols, eps, codes, ldc, scales,
                                  sum, lds, c, None)


def quant(x=P, ldx=64, type=0, rows=4, cols=64, codes=P, ldc=64, scales=P, c=None):
    return lib.quantize_rows_int8(x, ldx, type, rows, cols, codes, ldc, scales, c, None)


def back(dy=P, ldy=64, h=P, ldh=64, w=P, inv=P, ds=None, ldd=0, type=0, rows=4, cols=64, dx=P,
         ldx=64, dw=P, ws=P, ws_bytes=1 << 30, c=None):
    return lib.rms_norm_rows_backward(dy, ldy, h, ldh, w, inv, ds, ldd, type, rows, cols, dx, ldx,
                                      dw, ws, ws_bytes, c, None)


def mm(a=P, lda=64, sa=P, b=P, ldb=64, sb=P, bias=None, m=4, n=4, k=64, out=P, ldo=4, type=0,
       c=None):
    return lib.matmul_int8(a, lda, sa, b, ldb, sb, bias, m, n, k, out, ldo, type, c, None)


def test_norm_refusals():
    for f in (norm, norm8):
        for kw in (dict(x=None), dict(w=None)):
            assert f(**kw) == -1, (f, kw)
        for kw in (dict(x=P + 2), dict(ldx=68), dict(res=P + 8, ldr=64), dict(w=P + 2),
                   dict(res=P, ldr=66), dict(res=P, ldr=64, sum=P + 4, lds=64),
                   dict(res=P, ldr=64, sum=P, lds=65)):
            assert f(**kw) == -2, (f, kw)
        for kw in (dict(type=2), dict(type=-1), dict(eps=-1e-9), dict(eps=NAN),
                   dict(sum=P, lds=64), *(dict(c=cfg(**b)) for b in BAD_CONFIGS)):
            assert f(**kw) == -3, (f, kw)
        for kw in (dict(ldx=56), dict(ldx=0), dict(cols=1 << 30, rows=1), dict(rows=(1 << 40) + 1),
                   dict(rows=1 << 36), dict(res=P, ldr=56)):
            assert f(**kw) == -5, (f, kw)
        # nothing to do
        assert f(x=None, rows=0) == 0
    assert norm(out=None) == -1 and norm(out=P + 8) == -2 and norm(ldo=68) == -2
    assert norm(ldo=56) == -5 and norm(inv=P + 2) == -2
    assert norm8(codes=None) == -1 and norm8(scales=None) == -1 and norm8(codes=P + 8) == -2
    assert norm8(ldc=72) == -2 and norm8(ldc=48) == -5 and norm8(scales=P + 1) == -2
    assert norm(rows=4, cols=0, x=None, w=None, out=None) == 0


def test_quantize_refusals():
    assert quant(x=None) == -1 and quant(codes=None) == -1 and quant(scales=None) == -1
    assert quant(x=P + 2) == -2 and quant(codes=P + 8) == -2 and quant(ldx=68) == -2
    assert quant(ldc=72) == -2 and quant(scales=P + 2) == -2
    assert quant(type=2) == -3 and all(quant(c=cfg(**b)) == -3 for b in BAD_CONFIGS)
    assert quant(ldx=56) == -5 and quant(ldc=48) == -5
    assert quant(rows=0, x=None, codes=None, scales=None) == 0


def test_backward_refusals():
    big = dict(rows=4096, cols=4096, ldy=4096, ldh=4096, ldx=4096)   # several blocks: a workspace
    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(inv=None), dict(dx=None),
               dict(dw=None), dict(ws=None, **big)):
        assert back(**kw) == -1, kw
    for kw in (dict(dy=P + 2), dict(h=P + 8), dict(w=P + 2), dict(inv=P + 1), dict(dx=P + 4),
               dict(dw=P + 4), dict(ws=P + 16, **big), dict(ds=P + 2, ldd=64), dict(ldy=68),
               dict(ldh=68), dict(ldx=68), dict(ds=P, ldd=68)):
        assert back(**kw) == -2, kw
    for kw in (dict(type=2), *(dict(c=cfg(**b)) for b in BAD_CONFIGS)):
        assert back(**kw) == -3, kw
    need = armx.workspace_bytes(armx.OP_RMS_BACKWARD, 4096, 4096)
    assert need > 0
    assert back(ws_bytes=need - 1, **big) == -4
    for kw in (dict(ldy=56), dict(ldh=56), dict(ldx=56), dict(ds=P, ldd=56), dict(cols=1 << 30),
               dict(cols=(1 << 26) + 1, rows=1)):
        assert back(**kw) == -5, kw
    assert back(cols=0, dy=None, h=None, dx=None, dw=None, w=None, inv=None, ws=None) == 0


def test_backward_workspace_and_plan():
    assert armx.workspace_bytes(armx.OP_RMS_BACKWARD, 0, 4096) == 0
    assert armx.workspace_bytes(armx.OP_RMS_BACKWARD, 1, 4096) == 0
    # few rows, and rows of more than 16384 values: dweight's columns in blocks of
    # their own, one launch, no workspace; otherwise every block's partial sums and
    # a launch that joins them
    for rows, cols, apart in ((2, 4096, True), (1024, 4096, True), (1025, 4096, False),
                              (1024, 128, True), (1025, 128, False), (1024, 8200, False),
                              (5000, 20000, True), (5000, 100, False), (8192, 4096, False),
                              (77, 40000, True), (5000, 40000, True)):
        p = armx.launch_plan(armx.OP_RMS_BACKWARD, rows, cols)
        pitch = (cols + 63) // 64 * 64
        blocks = p["grid_blocks"]
        assert p["workspace_bytes"] == (0 if apart else 4 * blocks * pitch), (rows, cols)
        assert p["launches"] == (1 if apart else 2)
        if apart:
            assert blocks > pitch // 64
        assert p["workspace_bytes"] == armx.workspace_bytes(armx.OP_RMS_BACKWARD, rows, cols)
    with pytest.raises(armx.ArmxError):
        armx.workspace_bytes(armx.OP_RMS_BACKWARD, 4, 64, chain_r=2)
    with pytest.raises(armx.ArmxError):
        armx.launch_plan(armx.OP_RMS_BACKWARD, 4, 1 << 31)
    with pytest.raises(armx.ArmxError):
        armx.workspace_bytes(armx.OP_RMS_BACKWARD, 4, (1 << 26) + 1)
    # the largest grid: a block per row up to half of it, column blocks the other half
    p = armx.launch_plan(armx.OP_RMS_BACKWARD, 1 << 14, 1 << 26)
    assert p["grid_blocks"] == (1 << 20) + (1 << 14) and p["workspace_bytes"] == 0
    p = armx.launch_plan(armx.OP_RMS_BACKWARD, 1 << 22, 1 << 18)
    assert p["grid_blocks"] * p["block_threads"] < 1 << 31
    assert armx.launch_plan(armx.OP_RMS_BACKWARD, 4, 0)["launches"] == 0


def test_matmul_refusals():
    for kw in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(out=None)):
        assert mm(**kw) == -1, kw
    for kw in (dict(a=P + 8), dict(b=P + 8), dict(lda=72), dict(ldb=72), dict(sa=P + 2),
               dict(sb=P + 2), dict(out=P + 1), dict(bias=P + 1), dict(type=2, out=P + 2),
               dict(type=2, bias=P + 2)):
        assert mm(**kw) == -2, kw
    for kw in (dict(type=3), dict(type=-1), *(dict(c=cfg(**b)) for b in BAD_CONFIGS)):
        assert mm(**kw) == -3, kw
    for kw in (dict(k=131072, lda=131072, ldb=131072), dict(lda=48), dict(ldb=48), dict(ldo=3),
               dict(lda=(1 << 23) + 16), dict(ldb=(1 << 23) + 16), dict(m=(1 << 30) + 1),
               dict(n=(1 << 30) + 1, ldo=1 << 31), dict(m=1 << 30, lda=1 << 23),
               dict(m=1 << 30), dict(m=2097151 * 256 + 1), dict(m=1 << 22, n=1 << 17, ldo=1 << 17)):
        assert mm(**kw) == -5, kw
    assert mm(m=0, a=None, sa=None, out=None) == 0
    assert mm(n=0, b=None, sb=None, out=None) == 0


def test_python_layer_checks():
    h = torch.zeros(2, 16, dtype=torch.float16)
    w = torch.zeros(16, dtype=torch.float16)
    q = torch.zeros(2, 16, dtype=torch.int8)
    s = torch.ones(2)
    with pytest.raises(ValueError):
        armx.rms_norm_rows(h, w)                       # not on a GPU
    with pytest.raises(ValueError):
        armx.quantize_rows_int8(h)
    with pytest.raises(ValueError):
        armx.rms_norm_rows_backward(h, h, w, s)
    with pytest.raises(ValueError):
        armx.matmul_int8(q, s, q, s)
    for bad in (h.float(), h.double(), q):
        with pytest.raises(TypeError):
            armx.rms_norm_rows(bad, w)
        with pytest.raises(TypeError):
            armx.rms_norm_rows_int8(bad, w)
        with pytest.raises(TypeError):
            armx.quantize_rows_int8(bad)
    with pytest.raises(TypeError):
        armx.matmul_int8(h, s, q, s)
    with pytest.raises(TypeError):
        armx.rms_norm_rows(None, w)
