"""Cases that measure the row norms, the 8-bit row quantisation and the 8-bit
matrix product: a transformer layer's norm with its residual addition (forward
and backward), its 16-bit values turned into 8-bit codes with one scale per
row, and the product of such codes with the scales applied at its end.

`own` False runs each operator in plain torch operations, True through this
library's entry points; both take the same prepared inputs.  Codes are whole
numbers fixed to the last one by their definition (round half to even of
127 p / max|p| for the binary32 products p), so they are returned as they are,
with the scales beside them.
"""
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one token's residual stream, between two layers of a decode step
        {"name": "norm 1x4096 f16", "op": "norm", "rows": 1, "cols": 4096, "type": "f16",
         "residual": True, "eps": 1e-6},
        # a training micro-batch of 8192 tokens; 1/rms is kept for the backward pass
        {"name": "norm 8192x4096 bf16", "op": "norm", "rows": 8192, "cols": 4096,
         "type": "bf16", "residual": True, "eps": 1e-6},
        # a decode batch of odd size and width, before a quantised product
        {"name": "norm-int8 37x5001 f16", "op": "norm_int8", "rows": 37, "cols": 5001,
         "type": "f16", "residual": True, "eps": 1e-5},
        # a prompt chunk of a wide model, before a quantised product
        {"name": "norm-int8 8192x8192 bf16", "op": "norm_int8", "rows": 8192, "cols": 8192,
         "type": "bf16", "residual": True, "eps": 1e-6},
        # the norm's gradient on a short ragged batch, nothing else flowing in
        {"name": "norm-grad 515x2056 f16", "op": "norm_backward", "rows": 515, "cols": 2056,
         "type": "f16", "residual": False, "eps": 1e-6},
        # the norm's gradient on the training micro-batch, joined with the residual's
        {"name": "norm-grad 8192x4096 bf16", "op": "norm_backward", "rows": 8192, "cols": 4096,
         "type": "bf16", "residual": True, "eps": 1e-6},
        # a decode batch's activations before the second product of a feed-forward block
        {"name": "quantise 64x14336 f16", "op": "quantise", "rows": 64, "cols": 14336,
         "type": "f16"},
        # a weight matrix, laid out once when a model is loaded
        {"name": "quantise 16384x8192 bf16", "op": "quantise", "rows": 16384, "cols": 8192,
         "type": "bf16"},
        # a single token's projection
        {"name": "product 1x4096x4096 f16", "op": "product", "m": 1, "n": 4096, "k": 4096,
         "type": "f16", "bias": False},
        # a decode batch's projection
        {"name": "product 48x8192x4096 bf16", "op": "product", "m": 48, "n": 8192, "k": 4096,
         "type": "bf16", "bias": True},
        # a ragged batch, no side of it a multiple of a tile, sums kept in 32 bits
        {"name": "product 777x4100x5001 f32", "op": "product", "m": 777, "n": 4100, "k": 5001,
         "type": "f32", "bias": False},
        # a prompt chunk's projection
        {"name": "product 8192x8192x8192 bf16", "op": "product", "m": 8192, "n": 8192,
         "k": 8192, "type": "bf16", "bias": False},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over the logarithm."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_int8", "norm_backward", "quantise", "product", "product"])
    if op == "product":
        m, n, k = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        if rng.random() < 0.5:   # weights are mostly whole multiples of 64
            n, k = (n + 63) // 64 * 64, (k + 63) // 64 * 64
        return {"op": op, "m": m, "n": n, "k": k, "type": rng.choice(["f16", "bf16", "f32"]),
                "bias": rng.random() < 0.5}
    cols = _spread(rng, 64, 16384)
    if rng.random() < 0.5:
        cols = (cols + 63) // 64 * 64
    case = {"op": op, "rows": _spread(rng, 1, (1 << 25) // cols), "cols": cols,
            "type": rng.choice(["f16", "bf16"])}
    if op != "quantise":
        case |= {"residual": rng.random() < 0.7, "eps": rng.choice([1e-5, 1e-6])}
    return case


# ---- inputs -------------------------------------------------------------------

def _pitched(rows, cols, multiple, dtype):
    """An uninitialised matrix whose rows start at multiples of `multiple` values."""
    return torch.empty(rows, -(-cols // multiple) * multiple, dtype=dtype, device="cuda")[:, :cols]


def _codes(g, rows, cols):
    """8-bit codes and row scales of normally distributed values."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    scales = x.abs().amax(1) / 127
    q = _pitched(rows, cols, 16, torch.int8)
    q.copy_((x / scales[:, None]).round_().clamp_(-127, 127))
    return q, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "product":
        a, a_scales = _codes(g, case["m"], case["k"])
        b, b_scales = _codes(g, case["n"], case["k"])
        b_scales *= case["k"] ** -0.5
        dtype = _TYPES[case["type"]]
        bias = torch.randn(case["n"], generator=g, device="cuda").to(dtype) if case["bias"] else None
        return {"op": "product", "a": a, "a_scales": a_scales, "b": b, "b_scales": b_scales,
                "bias": bias, "dtype": dtype}
    rows, cols, dtype = case["rows"], case["cols"], _TYPES[case["type"]]

    def matrix(loud):
        m = _pitched(rows, cols, 8, dtype)
        m.copy_(torch.randn(rows, cols, generator=g, device="cuda") * loud)
        return m

    # hidden states: a few channels are much louder than the rest
    loud = 1 + 20 * (torch.rand(cols, generator=g, device="cuda") < 0.005)
    state = {"op": case["op"], "x": matrix(loud)}
    if case["op"] == "quantise":
        return state
    state["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dtype)
    state["eps"] = case["eps"]
    if case["op"] == "norm_backward":
        x = state["x"].float()
        state["inv_rms"] = torch.rsqrt(x.square().mean(1) + case["eps"])
        state["dy"] = matrix(0.01)
        state["dsum"] = matrix(0.01) if case["residual"] else None
    else:
        state["residual"] = matrix(1.0) if case["residual"] else None
    return state


# ---- the plain forms ----------------------------------------------------------

def _plain_sum(s):
    """The residual stream after the addition, in the inputs' type."""
    return s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)


def _plain_codes(p):
    """Codes and largest magnitudes of the rows of p (32 bits); the quotient in
    64 bits, where one next to a half is on its right side."""
    top = p.abs().amax(1)
    q = (127 * p.double() / top.double()[:, None]).round().to(torch.int8)
    return q, top


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = _plain_sum(s)
        f = h.float()
        inv = torch.rsqrt(f.square().mean(1) + s["eps"])
        return (f * inv[:, None] * s["weight"].float()).to(h.dtype), h, inv
    if op == "norm_int8":
        h = _plain_sum(s)
        f = h.float()
        inv = torch.rsqrt(f.square().mean(1) + s["eps"])
        q, top = _plain_codes(f * s["weight"].float())
        return q, top * inv / 127, h
    if op == "norm_backward":
        dy, x, inv = s["dy"].float(), s["x"].float(), s["inv_rms"][:, None]
        g = dy * s["weight"].float()
        dx = inv * (g - x * inv * inv * (g * x).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        return dx.to(s["x"].dtype), (dy * (x * inv)).sum(0)
    if op == "quantise":
        q, top = _plain_codes(s["x"].float())
        return q, top / 127
    y = (s["a"].float() @ s["b"].float().t()) * (s["a_scales"][:, None] * s["b_scales"])
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["dtype"])


def run(state):
    if not own:
        return _plain(state)
    import arithmetic_reduction_matrix_amd as armx

    op = state["op"]
    if op == "norm":
        r = armx.rms_norm_rows(state["x"], state["weight"], residual=state["residual"],
                               eps=state["eps"], keep_inv_rms=True)
        return r.out, state["x"] if r.sum is None else r.sum, r.inv_rms
    if op == "norm_int8":
        r = armx.rms_norm_rows_int8(state["x"], state["weight"], residual=state["residual"],
                                    eps=state["eps"])
        return r.codes, r.scales, state["x"] if r.sum is None else r.sum
    if op == "norm_backward":
        return armx.rms_norm_rows_backward(state["dy"], state["x"], state["weight"],
                                           state["inv_rms"], dsum=state["dsum"])
    if op == "quantise":
        return armx.quantize_rows_int8(state["x"])
    return armx.matmul_int8(state["a"], state["a_scales"], state["b"], state["b_scales"],
                            bias=state["bias"], dtype=state["dtype"])


# ---- what a pass cannot do without -----------------------------------------------

def work(case):
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["type"] == "f32" else 2
        return {"bytes": m * k + n * k + 4 * (m + n) + out * (m * n + (n if case["bias"] else 0)),
                "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    values = rows * cols
    if case["op"] == "quantise":
        return {"bytes": 3 * values + 4 * rows, "flops": 2 * values}
    if case["op"] == "norm_backward":
        return {"bytes": (8 if case["residual"] else 6) * values + 4 * rows + 6 * cols,
                "flops": 10 * values}
    # in and out, and with a residual the second input and the sum
    each = (2 if case["op"] == "norm" else 1) + 2 + (4 if case["residual"] else 0)
    return {"bytes": each * values + 4 * rows + 2 * cols, "flops": 5 * values}


# ---- the definitions, in 64 bits -----------------------------------------------

def _exact_codes(p):
    """Round half to even of 127 p / max|p|, decided by comparing 254 |p| with
    the odd multiples of max|p|: both sides exact in 64 bits."""
    top = p.abs().amax(1, keepdim=True)
    twice = 254 * p.abs()
    k = torch.floor(127 * p.abs() / top)
    k = k - (2 * k * top > twice).double() + (2 * (k + 1) * top <= twice).double()
    border = (2 * k + 1) * top
    up = (twice > border) | ((twice == border) & (k.remainder(2) == 1))
    return ((k + up.double()) * torch.sign(p)).to(torch.int8), top[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        y = torch.mm(s["a"].double(), s["b"].double().t().contiguous())
        y *= s["a_scales"].double()[:, None]
        y *= s["b_scales"].double()[None, :]
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["x"].double()
    if case["op"] == "quantise":
        q, top = _exact_codes(x)
        return q, top / 127
    w = s["weight"].double()
    if case["op"] == "norm_backward":
        r = s["inv_rms"].double().unsqueeze(1)
        n = x * r                                   # the normalised values
        g = s["dy"].double() * w
        dx = (g - n * ((g * n).sum(1, keepdim=True) / case["cols"])) * r
        if s["dsum"] is not None:
            dx = dx + s["dsum"].double()
        return dx, (s["dy"].double() * n).sum(0)
    if s["residual"] is not None:                   # the sum is defined as rounded once
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    r = 1 / ((x * x).sum(1) / case["cols"] + case["eps"]).sqrt()
    if case["op"] == "norm":
        return x * w * r.unsqueeze(1), x, r
    q, top = _exact_codes(x * w)
    return q, top * r / 127, x
