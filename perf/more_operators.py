"""Cases that measure what a training step needs beside the row norms and the
product: layer norm with its residual and dropout (forward and backward),
dropout by itself, and the softmax cross entropy of hidden states against a
large output weight (forward and backward).

`own` False runs each operator in plain torch operations, True through this
library's entry points; both take the same prepared inputs.

Dropout's random bits are a function of its seed, offset and step and of the
place in the matrix: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011) with the seed as key and the counter
(column / 8, row, low and high word of offset + step) gives 16 bits for each of
8 consecutive columns, low half of a word first.  A value is kept where its 16 bits
are at least t = round(65536 p), and then multiplied by 65536 / (65536 - t).
"""
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_IGNORED = -100


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one token's residual stream between two layers, as a model is sampled from
        {"name": "layer-norm 1x4096 f16", "op": "norm", "rows": 1, "cols": 4096, "type": "f16",
         "residual": True, "p": 0.0, "bias": True},
        # a ragged batch of an odd width, the first norm of a block: nothing to add
        {"name": "layer-norm 20011x1001 f16", "op": "norm", "rows": 20011, "cols": 1001,
         "type": "f16", "residual": False, "p": 0.0, "bias": False},
        # a training micro-batch: a block's output dropped out and added to the stream
        {"name": "layer-norm 8192x4096 bf16", "op": "norm", "rows": 8192, "cols": 4096,
         "type": "bf16", "residual": True, "p": 0.1, "bias": True},
        # the norm's gradient on a short ragged batch, nothing else flowing in
        {"name": "layer-norm-grad 515x2056 f16", "op": "norm_backward", "rows": 515, "cols": 2056,
         "type": "f16", "residual": False, "p": 0.0},
        # the micro-batch's gradient, joined with the stream's and through the dropout
        {"name": "layer-norm-grad 8192x4096 bf16", "op": "norm_backward", "rows": 8192,
         "cols": 4096, "type": "bf16", "residual": True, "p": 0.1},
        # a few sequences' embeddings of odd width, added to their positions'
        {"name": "dropout 37x5001 f16", "op": "dropout", "rows": 37, "cols": 5001, "type": "f16",
         "residual": True, "p": 0.25},
        # a feed-forward block's inner activations (the backward pass is the same call)
        {"name": "dropout 16384x8192 bf16", "op": "dropout", "rows": 16384, "cols": 8192,
         "type": "bf16", "residual": False, "p": 0.1},
        # the likelihood of a few tokens, as candidates are scored
        {"name": "loss 8x32768x1024 f16", "op": "loss", "rows": 8, "vocab": 32768, "cols": 1024,
         "type": "f16"},
        # a ragged evaluation batch, no side of it a multiple of a tile
        {"name": "loss 777x50001x2056 bf16", "op": "loss", "rows": 777, "vocab": 50001,
         "cols": 2056, "type": "bf16"},
        # a training micro-batch's loss over a large vocabulary
        {"name": "loss 8192x131072x4096 bf16", "op": "loss", "rows": 8192, "vocab": 131072,
         "cols": 4096, "type": "bf16"},
        # the loss's gradients on a short ragged batch of a small model
        {"name": "loss-grad 515x32003x1000 f16", "op": "loss_backward", "rows": 515,
         "vocab": 32003, "cols": 1000, "type": "f16"},
        # a training micro-batch's gradients over a large vocabulary
        {"name": "loss-grad 4096x131072x4096 bf16", "op": "loss_backward", "rows": 4096,
         "vocab": 131072, "cols": 4096, "type": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over the logarithm."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "dropout", "loss", "loss_backward"])
    kind = rng.choice(["f16", "bf16"])
    if op in ("loss", "loss_backward"):
        vocab, cols = _spread(rng, 1000, 131072), _spread(rng, 64, 4096)
        if rng.random() < 0.5:   # models mostly have whole multiples of 64
            vocab, cols = (vocab + 63) // 64 * 64, (cols + 63) // 64 * 64
        most = 8192 if op == "loss" else 4096
        return {"op": op, "rows": _spread(rng, 1, most), "vocab": min(vocab, 131072),
                "cols": cols, "type": kind}
    cols = _spread(rng, 64, 16384)
    if rng.random() < 0.5:
        cols = (cols + 63) // 64 * 64
    case = {"op": op, "rows": _spread(rng, 1, (1 << 25) // cols), "cols": cols, "type": kind,
            "residual": rng.random() < 0.7}
    if op == "dropout":
        return case | {"p": rng.choice([0.05, 0.1, 0.25, 0.5])}
    dropped = case["residual"] and rng.random() < 0.5
    case["p"] = rng.choice([0.05, 0.1, 0.25]) if dropped else 0.0
    return case | {"bias": rng.random() < 0.7} if op == "norm" else case


# ---- inputs -------------------------------------------------------------------

def _pitched(rows, cols, dtype):
    """An uninitialised matrix whose rows start at multiples of 16 bytes."""
    return torch.empty(rows, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, cols, dtype = case["rows"], case["cols"], _TYPES[case["type"]]

    def randn(*size):
        return torch.randn(*size, generator=g, device="cuda")

    def matrix(values):
        m = _pitched(values.shape[0], values.shape[1], dtype)
        m.copy_(values)
        return m

    state = {"op": case["op"]}
    if case["op"] in ("loss", "loss_backward"):
        vocab = case["vocab"]
        w = randn(vocab, cols) * cols ** -0.5
        # some tokens are far more frequent than others, and some positions have none
        u = torch.rand(rows, generator=g, device="cuda")
        targets = (vocab * u ** 3).long().clamp_(max=vocab - 1)
        # hidden states that point towards their target, some hardly and some clearly
        sure = 8 * torch.rand(rows, 1, generator=g, device="cuda")
        state["x"] = matrix(randn(rows, cols) + sure * w[targets])
        state["weight"] = matrix(w)
        del w
        if rows > 1:
            targets[torch.rand(rows, generator=g, device="cuda") < 0.05] = _IGNORED
        state["targets"] = targets
        if case["op"] == "loss_backward":
            state["lse"] = _plain_loss(state)[1]
            # a mean over tokens, with a weight for each sequence's own length and
            # scaled up as 16-bit gradients are
            each = 0.5 + torch.rand(rows, generator=g, device="cuda")
            state["dloss"] = each * (1024.0 / rows)
        return state

    # hidden states: a few channels are much louder than the rest
    loud = 1 + 20 * (torch.rand(cols, generator=g, device="cuda") < 0.005)
    state["x"] = matrix(randn(rows, cols) * loud + 0.5 * randn(cols))
    state["residual"] = matrix(randn(rows, cols)) if case["residual"] else None
    # a step's number, which lives on the device so that a captured step can advance it
    state["p"], state["seed"] = case["p"], 1000003 * seed + 17
    state["offset"], state["step"] = 7 << 32, torch.tensor([seed + 1], device="cuda")
    if case["op"] == "dropout":
        return state
    state["weight"] = (1 + 0.2 * randn(cols)).to(dtype)
    state["eps"] = 1e-5
    if case["op"] == "norm":
        state["bias"] = (0.2 * randn(cols)).to(dtype) if case["bias"] else None
        return state
    state["h"] = state.pop("x")
    state["dsum"] = state.pop("residual")
    f = state["h"].float()
    state["mean"] = f.mean(1)
    state["inv_std"] = torch.rsqrt(f.var(1, correction=0) + state["eps"])
    state["dy"] = matrix(0.01 * randn(rows, cols))
    if state["dsum"] is not None:
        state["dsum"].mul_(0.01)
    return state


# ---- the plain forms ----------------------------------------------------------

_LOW = 0xFFFFFFFF
_PIECE = 16384   # of the vocabulary


def _plain_factors(s, rows, cols):
    """What a value of a rows x cols matrix is multiplied by: the scale, or 0."""
    t = round(65536 * s["p"])
    place = (s["step"] + s["offset"]).view(1, 1)
    c0 = torch.arange(-(-cols // 8), device="cuda").view(1, -1)
    c1 = torch.arange(rows, device="cuda").view(-1, 1)
    c2, c3 = place & _LOW, place >> 32
    k0, k1 = s["seed"] & _LOW, (s["seed"] >> 32) & _LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # modulo 2^64: the bits are those of unsigned
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    words = torch.stack(torch.broadcast_tensors(c0, c1, c2, c3), 2)
    bits = torch.stack((words & 0xFFFF, words >> 16), 3).reshape(rows, -1)[:, :cols]
    return (bits >= t).float() * (65536 / (65536 - t))


def _plain_dropout(s):
    """The values that dropout and the residual's addition leave, in 32 bits."""
    f = s["x"].float()
    if s["p"] > 0:
        f = f * _plain_factors(s, *f.shape)
    return f if s["residual"] is None else f + s["residual"].float()


def _plain_loss(s):
    """Losses and log sums of exponentials, a piece of the vocabulary at a time."""
    x, w, targets = s["x"].float(), s["weight"], s["targets"]
    top = torch.full((x.shape[0],), -torch.inf, device="cuda")
    total = torch.zeros_like(top)
    hit = torch.zeros_like(top)
    for v in range(0, w.shape[0], _PIECE):
        z = x @ w[v:v + _PIECE].float().t()
        here = (targets >= v) & (targets < v + z.shape[1])
        at = z.gather(1, (targets - v).clamp(0, z.shape[1] - 1)[:, None])[:, 0]
        hit = torch.where(here, at, hit)
        most = torch.maximum(top, z.amax(1))
        total = total * torch.exp(top - most) + torch.exp(z.sub_(most[:, None])).sum(1)
        top = most
    lse = top + torch.log(total)
    return torch.where(targets == _IGNORED, 0.0, lse - hit), lse


def _plain_loss_backward(s):
    x, w, targets = s["x"].float(), s["weight"], s["targets"]
    each = torch.where(targets == _IGNORED, 0.0, s["dloss"])
    dx, dw = torch.zeros_like(x), torch.empty(w.shape, dtype=w.dtype, device="cuda")
    for v in range(0, w.shape[0], _PIECE):
        piece = w[v:v + _PIECE].float()
        dz = torch.exp((x @ piece.t()).sub_(s["lse"][:, None]))
        dz.sub_((torch.arange(v, v + piece.shape[0], device="cuda") == targets[:, None]).float())
        dz.mul_(each[:, None])
        dx += dz @ piece
        dw[v:v + _PIECE] = (dz.t() @ x).to(w.dtype)
    return dx.to(s["x"].dtype), dw


def _plain(s):
    op = s["op"]
    if op == "loss":
        return _plain_loss(s)
    if op == "loss_backward":
        return _plain_loss_backward(s)
    if op == "dropout":
        return _plain_dropout(s).to(s["x"].dtype)
    if op == "norm":
        h = _plain_dropout(s).to(s["x"].dtype)
        f = h.float()
        mean = f.mean(1)
        f = f - mean[:, None]
        inv = torch.rsqrt(f.square().mean(1) + s["eps"])
        y = f * inv[:, None] * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y.to(h.dtype), h, mean, inv
    dy, inv = s["dy"].float(), s["inv_std"][:, None]
    n = (s["h"].float() - s["mean"][:, None]) * inv
    g = dy * s["weight"].float()
    dh = inv * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dh = dh + s["dsum"].float()
    sums = (dy * n).sum(0), dy.sum(0)
    kind = s["h"].dtype
    if s["p"] == 0:
        return (dh.to(kind), *sums)
    return ((dh * _plain_factors(s, *dh.shape)).to(kind), *sums, dh.to(kind))


def run(state):
    if not own:
        return _plain(state)
    import arithmetic_reduction_matrix_amd as armx

    op, s = state["op"], state
    if op == "loss":
        return armx.cross_entropy_rows(s["x"], s["weight"], s["targets"], ignore_index=_IGNORED)
    if op == "loss_backward":
        return armx.cross_entropy_rows_backward(s["dloss"], s["x"], s["weight"], s["targets"],
                                                s["lse"], ignore_index=_IGNORED)
    drop = armx.Dropout(s["p"], s["seed"], s["offset"], step=s["step"]) if s["p"] > 0 else None
    if op == "dropout":
        return armx.dropout_rows(s["x"], drop, residual=s["residual"])
    if op == "norm":
        r = armx.layer_norm_rows(s["x"], s["weight"], s["bias"], residual=s["residual"],
                                 dropout=drop, eps=s["eps"], keep_stats=True)
        return r.out, s["x"] if r.sum is None else r.sum, r.mean, r.inv_std
    r = armx.layer_norm_rows_backward(s["dy"], s["h"], s["weight"], s["mean"], s["inv_std"],
                                      dsum=s["dsum"], dropout=drop)
    return r[:3] if drop is None else tuple(r)


# ---- what a pass cannot do without -----------------------------------------------

def work(case):
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "loss":
        vocab = case["vocab"]
        return {"bytes": 2 * (rows + vocab) * cols + 16 * rows, "flops": 2 * rows * vocab * cols}
    if case["op"] == "loss_backward":   # the logits, which nothing keeps, and two products
        vocab = case["vocab"]
        return {"bytes": 4 * (rows + vocab) * cols + 16 * rows, "flops": 6 * rows * vocab * cols}
    values = rows * cols
    each = 4 + (2 if case["residual"] else 0)
    if case["op"] == "dropout":
        return {"bytes": each * values, "flops": 2 * values}
    if case["op"] == "norm":   # in and out, and with a residual the second input and the sum
        each += 2 if case["residual"] else 0
        return {"bytes": each * values + 8 * rows + (4 if case["bias"] else 2) * cols,
                "flops": 8 * values}
    each += 4 if case["p"] > 0 else 2   # dy and h in, dx out, and the residual's apart from x's
    return {"bytes": each * values + 8 * rows + 10 * cols, "flops": 14 * values}


# ---- the definitions, in 64 bits -----------------------------------------------

def _high_low(m, c):
    """The words of m c (m a number, c a tensor, both of 32 bits), from products of
    halves, none of which leaves 63 bits."""
    m1, m0 = m >> 16, m & 0xFFFF
    low = c * m0
    mid = c * m1 + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _exact_kept(s, rows, cols):
    """Which values are kept, a column of 8 x 4 words at a time."""
    limit = int(65536 * s["p"] + 0.5)
    place = s["offset"] + int(s["step"])
    lanes = (cols + 7) // 8
    group = torch.arange(lanes, device="cuda").expand(rows, lanes)
    row = torch.arange(rows, device="cuda")[:, None].expand(rows, lanes)
    ctr = [group, row, torch.full_like(group, place % 2 ** 32), torch.full_like(group, place // 2 ** 32)]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32 % 2 ** 32]
    for _ in range(10):
        h0, l0 = _high_low(0xD2511F53, ctr[0])
        h1, l1 = _high_low(0xCD9E8D57, ctr[2])
        ctr = [h1.bitwise_xor(ctr[1]).bitwise_xor(key[0]), l1,
               h0.bitwise_xor(ctr[3]).bitwise_xor(key[1]), l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    kept = torch.empty(rows, lanes, 8, dtype=torch.bool, device="cuda")
    for i in range(8):
        kept[:, :, i] = (ctr[i // 2] // (65536 if i % 2 else 1)) % 65536 >= limit
    return kept.view(rows, lanes * 8)[:, :cols], 65536 / (65536 - limit)


def _exact_dropout(s):
    x = s["x"].double()
    if s["p"] > 0:
        kept, scale = _exact_kept(s, *x.shape)
        x = torch.where(kept, x * scale, torch.zeros_like(x))
    return x if s["residual"] is None else s["residual"].double() + x


def _exact_logits(s, first, count):
    return torch.mm(s["x"].double(), s["weight"][first:first + count].double().t().contiguous())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "loss":
        t = s["targets"]
        lse = torch.full((case["rows"],), -torch.inf, dtype=torch.float64, device="cuda")
        for v in range(0, case["vocab"], 8192):
            lse = torch.logaddexp(lse, torch.logsumexp(_exact_logits(s, v, 8192), 1))
        own_logit = (s["x"].double() * s["weight"][t.clamp(min=0)].double()).sum(1)
        return torch.where(t < 0, torch.zeros_like(lse), lse - own_logit), lse
    if case["op"] == "loss_backward":
        t, d = s["targets"], s["dloss"].double()
        d = torch.where(t < 0, torch.zeros_like(d), d)
        x = s["x"].double()
        dx = torch.zeros_like(x)
        dw = torch.empty(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        for v in range(0, case["vocab"], 8192):
            p = torch.exp(_exact_logits(s, v, 8192) - s["lse"].double().unsqueeze(1))
            rows = ((t >= v) & (t < v + p.shape[1])).nonzero()[:, 0]
            p[rows, t[rows] - v] -= 1
            p *= d.unsqueeze(1)
            dx += torch.mm(p, s["weight"][v:v + 8192].double())
            dw[v:v + 8192] = torch.mm(p.t().contiguous(), x)
        return dx, dw
    if case["op"] == "dropout":
        return _exact_dropout(s)
    if case["op"] == "norm":
        h = _exact_dropout(s).to(s["x"].dtype).double()   # the sum is defined as rounded once
        mean = h.sum(1) / case["cols"]
        c = h - mean.unsqueeze(1)
        inv = 1 / ((c * c).sum(1) / case["cols"] + s["eps"]).sqrt()
        y = c * inv.unsqueeze(1) * s["weight"].double()
        return y if s["bias"] is None else y + s["bias"].double(), h, mean, inv
    dy, w = s["dy"].double(), s["weight"].double()
    inv = s["inv_std"].double().unsqueeze(1)
    n = (s["h"].double() - s["mean"].double().unsqueeze(1)) * inv
    g = dy * w
    dh = (g - g.sum(1, keepdim=True) / case["cols"] - n * ((g * n).sum(1, keepdim=True) / case["cols"])) * inv
    if s["dsum"] is not None:
        dh = dh + s["dsum"].double()
    sums = torch.sum(dy * n, 0), torch.sum(dy, 0)
    if case["p"] == 0:
        return (dh, *sums)
    kept, scale = _exact_kept(s, *dh.shape)
    return (torch.where(kept, dh * scale, torch.zeros_like(dh)), *sums, dh)
