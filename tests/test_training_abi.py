"""Refusals and workspace sizes of dropout, layer norm and the cross entropy, on the
CPU: every call here fails, or has nothing to do, before a device is touched."""
import ctypes

import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from arithmetic_reduction_matrix_amd.training import _DropoutArgs

lib = armx.lib
P = 1 << 20     # an aligned address; never dereferenced
Q = P + (1 << 16)
NAN = float("nan")
NONE = ctypes.c_size_t(-1).value


def cfg(**kw):
    return ctypes.byref(armx._config(**kw))


def drop(p=0.1, seed=1, offset=0, step=None, first_row=0):
    return ctypes.byref(_DropoutArgs(p, seed, offset, step, first_row))


BAD_CONFIGS = [dict(block_threads=256), dict(chain_r=1), dict(grid_blocks=5), dict(plain=True)]
BAD_DROPS = [(dict(p=-0.1), -3), (dict(p=1.1), -3), (dict(p=NAN), -3), (dict(step=P + 4), -2),
             (dict(first_row=(1 << 32) - 3), -5), (dict(first_row=(1 << 64) - 1), -5)]


def dropped(x=P, ldx=64, res=None, ldr=0, type=0, rows=4, cols=64, d=drop(), out=P, ldo=64, c=None):
    return lib.dropout_rows(x, ldx, res, ldr, type, rows, cols, d, out, ldo, c, None)


def norm(x=P, ldx=64, res=None, ldr=0, w=P, b=P, type=0, rows=4, cols=64, eps=1e-5, d=None, out=P,
         ldo=64, sum=None, lds=0, mean=None, inv=None, c=None):
    return lib.layer_norm_rows(x, ldx, res, ldr, w, b, type, rows, cols, eps, d, out, ldo, sum, lds,
                               mean, inv, c, None)


def back(dy=P, ldy=64, h=P, ldh=64, w=P, mean=P, inv=P, ds=None, ldd=0, type=0, rows=4, cols=64,
         d=None, dx=P, ldx=64, dr=None, ldr=0, dw=P, db=P, ws=P, ws_bytes=1 << 30, c=None):
    return lib.layer_norm_rows_backward(dy, ldy, h, ldh, w, mean, inv, ds, ldd, type, rows, cols, d,
                                        dx, ldx, dr, ldr, dw, db, ws, ws_bytes, c, None)


def loss(x=P, ldx=64, w=P, ldw=64, t=P, type=0, rows=4, vocab=100, cols=64, ignore=-100, out=P,
         lse=P, ws=P, ws_bytes=1 << 40, c=None):
    return lib.cross_entropy_rows(x, ldx, w, ldw, t, type, rows, vocab, cols, ignore, out, lse, ws,
                                  ws_bytes, c, None)


def grad(g=P, x=P, ldx=64, w=P, ldw=64, t=P, lse=P, type=0, rows=4, vocab=100, cols=64, ignore=-100,
         dx=P, lddx=64, dw=P, lddw=64, dwt=0, ws=P, ws_bytes=1 << 40, c=None):
    return lib.cross_entropy_rows_backward(g, x, ldx, w, ldw, t, lse, type, rows, vocab, cols,
                                           ignore, dx, lddx, dw, lddw, dwt, ws, ws_bytes, c, None)


def test_dropout_refusals():
    assert dropped(x=None) == -1 and dropped(out=None) == -1 and dropped(d=None) == -1
    for kw in (dict(x=P + 2), dict(ldx=68), dict(out=P + 8), dict(ldo=68), dict(res=P + 8, ldr=64),
               dict(res=P, ldr=66)):
        assert dropped(**kw) == -2, kw
    assert dropped(type=2) == -3 and all(dropped(c=cfg(**b)) == -3 for b in BAD_CONFIGS)
    assert dropped(ldx=56) == -5 and dropped(ldo=56) == -5 and dropped(cols=1 << 30, rows=1) == -5
    for kw, status in BAD_DROPS:
        assert dropped(d=drop(**kw)) == status, kw
    assert dropped(d=drop(first_row=(1 << 32) - 4), x=None) == -1   # the last rows there are
    assert dropped(rows=0, x=None, out=None) == 0 and dropped(cols=0, x=None, out=None) == 0


def test_layer_norm_refusals():
    for kw in (dict(x=None), dict(w=None), dict(out=None)):
        assert norm(**kw) == -1, kw
    for kw in (dict(x=P + 2), dict(ldx=68), dict(res=P + 8, ldr=64), dict(w=P + 2), dict(b=P + 2),
               dict(res=P, ldr=66), dict(out=P + 8), dict(ldo=68), dict(mean=P + 2), dict(inv=P + 2),
               dict(res=P, ldr=64, sum=P + 4, lds=64), dict(res=P, ldr=64, sum=Q, lds=65)):
        assert norm(**kw) == -2, kw
    for kw in (dict(type=2), dict(type=-1), dict(eps=-1e-9), dict(eps=NAN), dict(sum=Q, lds=64),
               dict(x=P, res=Q, ldr=64, out=P, sum=P, lds=64), dict(d=drop(), out=P, sum=P, lds=64),
               *(dict(c=cfg(**b)) for b in BAD_CONFIGS)):
        assert norm(**kw) == -3, kw
    for kw in (dict(ldx=56), dict(ldo=56), dict(cols=1 << 30, rows=1), dict(rows=(1 << 40) + 1),
               dict(rows=1 << 36), dict(res=P, ldr=56)):
        assert norm(**kw) == -5, kw
    for kw, status in BAD_DROPS:
        assert norm(d=drop(**kw)) == status, kw
    assert norm(rows=0, x=None, w=None, out=None) == 0
    assert norm(cols=0, x=None, w=None, out=None) == 0


def test_layer_norm_backward_refusals():
    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(mean=None), dict(inv=None),
               dict(dx=None), dict(dw=None), dict(db=None), dict(rows=2000, ws=None)):
        assert back(**kw) == -1, kw
    for kw in (dict(dy=P + 2), dict(ldy=68), dict(h=P + 8), dict(ldh=68), dict(w=P + 2),
               dict(mean=P + 2), dict(inv=P + 2), dict(ds=P + 2, ldd=64), dict(ds=P, ldd=68),
               dict(dx=P + 8), dict(ldx=68), dict(dw=P + 2), dict(db=P + 2),
               dict(d=drop(), dr=Q + 8, ldr=64), dict(rows=2000, ws=P + 128)):
        assert back(**kw) == -2, kw
    for kw in (dict(type=2), dict(dr=Q, ldr=64), dict(d=drop(), dr=P, ldr=64, dx=P),
               *(dict(c=cfg(**b)) for b in BAD_CONFIGS)):
        assert back(**kw) == -3, kw
    need = armx.workspace_bytes(armx.OP_LAYER_NORM_BACKWARD, 2000, 64)
    assert need > 0 and back(rows=2000, ws_bytes=need - 1) == -4
    for kw in (dict(ldy=56), dict(ldx=56), dict(cols=(1 << 26) + 1, rows=1),
               dict(rows=(1 << 40) + 1)):
        assert back(**kw) == -5, kw
    for kw, status in BAD_DROPS:
        assert back(d=drop(**kw)) == status, kw
    assert back(cols=0, dy=None, h=None, dw=None, db=None) == 0


def test_layer_norm_workspace_is_two_rows_of_sums_a_block():
    for rows, cols in [(1, 64), (1000, 64), (2000, 64), (8192, 4096), (8192, 3000), (513, 16385),
                       (0, 64)]:
        plan = armx.launch_plan(armx.OP_LAYER_NORM_BACKWARD, rows, cols)
        need = armx.workspace_bytes(armx.OP_LAYER_NORM_BACKWARD, rows, cols)
        assert plan["workspace_bytes"] == need
        assert need in (0, plan["grid_blocks"] * 2 * ((cols + 63) // 64 * 64) * 4)
        # few rows, and rows that the registers do not hold beside the sums, need none
        assert (need == 0) == ((rows <= 1024 and rows * cols <= 1 << 23) or cols > 16384)
        assert plan["launches"] == (2 if need else 1)


BAD_LOSS_SIZES = [dict(vocab=0), dict(cols=0), dict(cols=(1 << 21) + 1, rows=1, vocab=1),
                  dict(rows=(1 << 21) + 1), dict(vocab=(1 << 28) + 1),
                  dict(rows=1 << 21, vocab=1 << 20)]


def test_cross_entropy_refusals():
    for kw in (dict(x=None), dict(w=None), dict(t=None), dict(out=None), dict(lse=None),
               dict(ws=None)):
        assert loss(**kw) == -1, kw
    for kw in (dict(x=P + 2), dict(ldx=68), dict(w=P + 8), dict(ldw=68), dict(t=P + 4),
               dict(out=P + 2), dict(lse=P + 2), dict(ws=P + 128)):
        assert loss(**kw) == -2, kw
    assert loss(type=2) == -3 and all(loss(c=cfg(**b)) == -3 for b in BAD_CONFIGS)
    need = lib.armx_cross_entropy_workspace_bytes(4, 100, 64)
    assert need == 2 * 8 * 8 + 4 * 4 and loss(ws_bytes=need - 1) == -4
    for kw in (*BAD_LOSS_SIZES, dict(ldx=56), dict(ldw=56), dict(ldx=(1 << 22) + 8),
               dict(ldw=(1 << 22) + 8)):
        assert loss(**kw) == -5, kw
    assert loss(rows=0, x=None, w=None, t=None, out=None, lse=None, ws=None) == 0


def test_cross_entropy_backward_refusals():
    for kw in (dict(g=None), dict(x=None), dict(w=None), dict(t=None), dict(lse=None),
               dict(dx=None, dw=None), dict(ws=None)):
        assert grad(**kw) == -1, kw
    for kw in (dict(g=P + 2), dict(x=P + 2), dict(ldx=68), dict(w=P + 8), dict(ldw=68),
               dict(t=P + 4), dict(lse=P + 2), dict(dx=P + 8), dict(lddx=68), dict(dw=P + 8),
               dict(lddw=68), dict(ws=P + 128)):
        assert grad(**kw) == -2, kw
    for kw in (dict(type=2, dwt=2), dict(dwt=1), dict(type=1, dwt=0), dict(dwt=3),
               *(dict(c=cfg(**b)) for b in BAD_CONFIGS)):
        assert grad(**kw) == -3, kw
    need = lib.armx_cross_entropy_backward_workspace_bytes(4, 100, 64, 1, 1)
    assert grad(ws_bytes=need - 1) == -4
    for kw in (*BAD_LOSS_SIZES, dict(rows=1 << 21, vocab=100, cols=1 << 20), dict(ldx=56),
               dict(lddx=56), dict(lddw=56), dict(ldw=(1 << 22) + 8)):
        assert grad(**kw) == -5, kw
    assert grad(rows=0, g=None, x=None, w=None, t=None, lse=None, dx=None, dw=None, ws=None) == 0


def test_two_results_in_one_place_are_refused():
    assert norm(mean=P, inv=P) == -3 and norm(mean=P, inv=P, cols=0) == -3
    assert back(dw=P, db=P) == -3
    assert loss(out=P, lse=P) == -3
    assert grad(dx=P, dw=P) == -3
    # which is said last: what else is wrong has its own status
    assert loss(out=P, lse=P, ws_bytes=0) == -4 and grad(dx=P, dw=P, ws_bytes=0) == -4


def test_cross_entropy_workspaces():
    size = lib.armx_cross_entropy_backward_workspace_bytes
    both, dx, dw = (size(4096, 131072, 4096, *w) for w in ((1, 1), (1, 0), (0, 1)))
    # the logits alone would take 4 bytes each
    assert both < 4 * 4096 * 131072 / 2 and dx < both and dw < both
    assert size(0, 100, 64, 1, 1) == 0 == lib.armx_cross_entropy_workspace_bytes(0, 100, 64)
    for kw in BAD_LOSS_SIZES:
        s = dict(rows=4, vocab=100, cols=64) | kw
        assert lib.armx_cross_entropy_workspace_bytes(s["rows"], s["vocab"], s["cols"]) == NONE
        assert size(s["rows"], s["vocab"], s["cols"], 1, 1) == NONE
    # nothing that is taken is out of bounds or out of proportion, whatever the shape
    for rows, vocab, cols in [(1, 1, 1), (1, 1 << 28, 8), (1 << 21, 255, 8), (1, 100, 1 << 21),
                              (128, 50001, 4096), (129, 50001, 4096), (8192, 131072, 8192)]:
        assert 0 < size(rows, vocab, cols, 1, 1) < 1 << 40


def test_python_refusals():
    x, w, t = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(64, dtype=torch.float16), \
        torch.zeros(4, dtype=torch.long)
    stat = torch.zeros(4)
    d = armx.Dropout(0.1, 1)
    calls = [lambda x: armx.dropout_rows(x, d), lambda x: armx.layer_norm_rows(x, w),
             lambda x: armx.layer_norm_rows_backward(x, x, w, stat, stat),
             lambda x: armx.cross_entropy_rows(x, x, t),
             lambda x: armx.cross_entropy_rows_backward(stat, x, x, t, stat)]
    for call in calls:
        with pytest.raises(ValueError, match="on a GPU"):
            call(x)
        with pytest.raises(TypeError, match="float16 or bfloat16"):
            call(x.float())
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call(None)
