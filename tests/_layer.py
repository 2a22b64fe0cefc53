"""Helpers of the layer operators' tests: inputs, conversions and tolerances."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24                                   # half a binary32 step
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}     # half a step, relative
FLOOR = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the smallest step
TYPES = [torch.float16, torch.bfloat16]


def ids(t):
    return str(t).replace("torch.", "")


def f64(t):
    return t.detach().cpu().double().numpy()


def f32(t):
    return t.detach().cpu().float().numpy()


def make(rng, rows, cols, dtype, scale=1.0, pad=0, multiple=8, device="cpu"):
    """rows x cols normal values in `dtype`, at a pitch of whole multiples plus
    `pad` of them; what stands in the padding is NaN."""
    pitch = (-(-cols // multiple) + pad) * multiple
    m = torch.full((rows, pitch), float("nan"), dtype=dtype)
    m[:, :cols] = torch.from_numpy(rng.standard_normal((rows, cols)) * scale).to(dtype)
    return m.to(device)[:, :cols]


def make_codes(rng, rows, k, pad=0, device="cpu", low=-128):
    """rows x k codes at a pitch of whole 16s plus `pad` of them; the padding
    holds codes too."""
    pitch = (-(-k // 16) + pad) * 16
    m = torch.from_numpy(rng.integers(low, 128, (rows, pitch), dtype=np.int8))
    return m.to(device)[:, :k]


def sum_depth(cols):
    """No value meets more than this many binary32 additions in a row's sum:
    4 + 1 within a 16-byte chunk, one per chunk of a thread (at most 4, or one
    per 1024 x 8 values of a longer row), 6 across lanes, 16 across wavefronts."""
    return 5 + max(4, -(-cols // 8192)) + 6 + 16
