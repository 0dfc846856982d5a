"""Cases of the linear-layer operators: the norm that feeds a layer, the
quantisation to 8 bits with a scale per block of 128, the 8-bit product with
those scales, and the products grouped by expert, each forward and backward.

`run` computes an operator in its plain form with elementary torch operations
(`own` false) or calls the library's operator (`own` true).
"""

import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EIGHT = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
SMALLEST = 2.0 ** -100  # a block's largest magnitude counts as at least this
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token of a serving loop: the residual's sum and the layer's 8-bit input, width 1024
        dict(name="norm_token", op="norm", rows=1, width=1024, type="bf16", residual=True, keep_y=False, eight="e4m3"),
        # a training batch at width 2048: y is kept for the weight's gradient, q feeds the product
        dict(name="norm_batch", op="norm", rows=16384, width=2048, type="bf16", residual=True, keep_y=True, eight="e4m3"),
        # its backward pass, with the gradient that comes down the residual
        dict(name="norm_grad_batch", op="norm_grad", rows=16384, width=2048, type="bf16", residual=True),
        # odd sizes, fp16, no residual
        dict(name="norm_grad_odd", op="norm_grad", rows=3001, width=1337, type="f16", residual=False),
        # an MLP weight after its step (float32 master): 128 x 128 blocks, both orders (forward and row gradient)
        dict(name="quantize_weight", op="quantize", rows=8192, cols=2048, type="f32", eight="e4m3", block="square", order="both"),
        # an output gradient with a ragged number of tokens, by rows for dX and by columns for dW
        dict(name="quantize_grad", op="quantize", rows=8191, cols=1024, type="bf16", eight="e5m2", block="vector", order="both"),
        # one to a few tokens through a width-1024 up projection: latency and the weight's bytes
        dict(name="matmul_tokens", op="matmul", m=8, n=4096, k=1024, a_eight="e4m3", b_block="square", out="bf16"),
        # the width-2048 up projection over a training batch
        dict(name="matmul_forward", op="matmul", m=16384, n=8192, k=2048, a_eight="e4m3", b_block="square", out="bf16"),
        # its weight's gradient: contraction over a ragged number of tokens, float32 out
        dict(name="matmul_weight_grad", op="matmul", m=8192, n=2048, k=16383, a_eight="e5m2", b_block="vector", out="f32"),
        # 16 rows routed over 64 experts: most of them empty, latency and the used experts' bytes
        dict(name="grouped_tokens", op="grouped", experts=64, rows=16, n=2048, k=1536, type="bf16", skew=1.0, spare=0),
        # a training batch over 64 experts, uneven loads, some rows routed nowhere
        dict(name="grouped_forward", op="grouped", experts=64, rows=16384, n=2048, k=1536, type="bf16", skew=0.7, spare=100),
        # its backward pass: the rows' gradient and the experts' (float32, what the Gram update takes)
        dict(name="grouped_backward", op="grouped_grad", experts=64, rows=16384, n=2048, k=1536, type="bf16", skew=0.7, spare=100),
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm; a third of them multiples of 128, the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.33 and v > 128:
        v = v // 128 * 128
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "matmul", "matmul", "grouped", "grouped_grad"])
    if op in ("norm", "norm_grad"):
        case = dict(op=op, rows=_size(rng, 1, 16384), width=_size(rng, 64, 8192), type=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.7)
        case["rows"] = max(1, min(case["rows"], 16384 * 2048 // case["width"]))
        if op == "norm":
            case["keep_y"] = rng.random() < 0.6
            case["eight"] = rng.choice(["e4m3", "e5m2", "e4m3"]) if not case["keep_y"] or rng.random() < 0.7 else ""
        return case
    if op == "quantize":
        case = dict(op=op, rows=_size(rng, 1, 16384), cols=_size(rng, 32, 8192), type=rng.choice(["bf16", "f16", "f32"]),
                    eight=rng.choice(["e4m3", "e5m2"]), block=rng.choice(["vector", "square"]), order=rng.choice(["rows", "columns", "both"]))
        case["rows"] = max(1, min(case["rows"], 8192 * 2048 // case["cols"]))
        return case
    if op == "matmul":
        case = dict(op=op, m=_size(rng, 1, 16384), n=_size(rng, 64, 8192), k=_size(rng, 64, 16384), a_eight=rng.choice(["e4m3", "e5m2"]),
                    b_block=rng.choice(["square", "vector"]), out=rng.choice(["bf16", "f16", "f32"]))
        case["m"] = max(1, min(case["m"], 16384 * 8192 * 2048 // (case["n"] * case["k"])))
        return case
    case = dict(op=op, experts=rng.choice([1, 3, 8, 17, 32, 64]), rows=_size(rng, 1, 16384), n=_size(rng, 64, 2048), k=_size(rng, 64, 1536),
                type=rng.choice(["bf16", "f16"]), skew=round(rng.uniform(0.0, 1.2), 2), spare=0)
    if rng.random() < 0.3:
        case["spare"] = rng.randint(0, case["rows"] // 4)
    return case


# ------------------------------------------------------------------ inputs
def _padded(rows, cols, dtype, dev):
    """A rows x cols matrix whose rows start 16 bytes apart or a multiple of it, as the quantiser lays them out."""
    return torch.zeros(rows, (cols + 15) // 16 * 16, dtype=dtype, device=dev)[:, :cols]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quantized(x, eight, square):
    """An operand as a user's program has it: 8-bit values in padded rows, float32 scales per 1 x 128 or 128 x 128."""
    dtype, top = EIGHT[eight]
    m, n = x.shape
    full = torch.zeros(_blocks(m) * BLOCK if square else m, _blocks(n) * BLOCK, device=x.device)
    full[:m, :n] = x
    tall = BLOCK if square else 1
    tiles = full.view(full.shape[0] // tall, tall, _blocks(n), BLOCK)
    s = tiles.abs().amax((1, 3)).clamp_min(SMALLEST) / top
    q = _padded(m, n, dtype, x.device)
    q.copy_((tiles / s[:, None, :, None]).view(full.shape)[:m, :n].to(dtype))
    return q, s


def _activations(rows, cols, g, dev):
    """Rows of differing size and a few large channels, as hidden states have them."""
    x = torch.randn(rows, cols, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=dev))
    channels = torch.randint(0, cols, (max(1, cols // 200),), generator=g, device=dev)
    x[:, channels] *= 8.0
    return x


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    state = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if op in ("norm", "norm_grad"):
        t = TYPES[case["type"]]
        rows, width = case["rows"], case["width"]
        state["weight"] = 1.0 + 0.1 * randn(width)
        state["eps"] = 1e-6
        x = _activations(rows, width, g, dev).to(t)
        if op == "norm":
            state["x"] = x
            state["residual"] = (2.0 * randn(rows, width)).to(t) if case["residual"] else None
        else:
            state["h"] = x
            state["rstd"] = torch.rsqrt(x.float().square().mean(1) + 1e-6)
            state["dy"] = randn(rows, width).to(t)
            state["dresidual"] = randn(rows, width).to(t) if case["residual"] else None
    elif op == "quantize":
        state["x"] = _activations(case["rows"], case["cols"], g, dev).to(TYPES[case["type"]])
    elif op == "matmul":
        state["a"], state["sa"] = _quantized(_activations(case["m"], case["k"], g, dev), case["a_eight"], False)
        state["b"], state["sb"] = _quantized(randn(case["n"], case["k"]) / math.sqrt(case["k"]), "e4m3", case["b_block"] == "square")
    else:
        t = TYPES[case["type"]]
        E, rows = case["experts"], case["rows"]
        p = torch.softmax(case["skew"] * randn(E).double(), 0)
        ends = torch.cumsum(p, 0)
        routed = rows - case["spare"]
        at = torch.rand(routed, generator=g, device=dev, dtype=torch.float64)
        expert = (at[:, None] >= ends[None, :-1]).sum(1) if E > 1 else torch.zeros(routed, dtype=torch.int64, device=dev)
        sizes = torch.bincount(expert, minlength=E)
        state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(sizes, 0)]).to(torch.int32)
        state["most"] = max(1, int(sizes.max()))  # the plain form pads every expert to this many rows
        state["w"] = (randn(E, case["n"], case["k"]) / math.sqrt(case["k"])).to(t)
        state["x"] = _activations(rows, case["k"], g, dev).to(t)
        if op == "grouped_grad":
            state["dy"] = randn(rows, case["n"]).to(t)
    return state


# ------------------------------------------------------------ plain forms
def _plain_blocks(y, eight, tall):
    """(8-bit values, scales) of float32 y for blocks of `tall` x 128."""
    dtype, top = EIGHT[eight]
    m, n = y.shape
    mb, nb = (m + tall - 1) // tall, _blocks(n)
    if mb * tall != m or nb * BLOCK != n:
        y = torch.nn.functional.pad(y, (0, nb * BLOCK - n, 0, mb * tall - m))
    tiles = y.view(mb, tall, nb, BLOCK)
    s = tiles.abs().amax((1, 3)).clamp_min(SMALLEST) / top
    q = (tiles / s[:, None, :, None]).view(mb * tall, nb * BLOCK)[:m, :n]
    return q.to(dtype), s


def _plain_norm(state):
    case = state["case"]
    h = state["x"]
    if state["residual"] is not None:
        h = (h.float() + state["residual"].float()).to(h.dtype)
    v = h.float()
    rstd = torch.rsqrt(v.square().mean(1) + state["eps"])
    y = v * rstd[:, None] * state["weight"]
    out = {"rstd": rstd}
    if state["residual"] is not None:
        out["h"] = h
    if case["keep_y"]:
        out["y"] = y.to(h.dtype)
    if case["eight"]:
        out["q"], out["scales"] = _plain_blocks(y, case["eight"], 1)
    return out


def _plain_norm_grad(state):
    t = state["dy"].dtype
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    xhat = state["h"].float() * rstd
    g = dy * state["weight"]
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if state["dresidual"] is not None:
        dx = dx + state["dresidual"].float()
    return {"dx": dx.to(t), "dweight": (dy * xhat).sum(0)}


def _plain_quantize(state):
    case = state["case"]
    x = state["x"].float()
    out = {}
    tall = BLOCK if case["block"] == "square" else 1
    if case["order"] in ("rows", "both"):
        out["q"], out["scales"] = _plain_blocks(x, case["eight"], tall)
    if case["order"] in ("columns", "both"):
        out["qt"], out["scales_t"] = _plain_blocks(x.t().contiguous(), case["eight"], tall)
    return out


def _plain_spread(q, s):
    """float32 values that 8-bit q with scales s stands for."""
    m, n = q.shape
    s = s.repeat_interleave(BLOCK, 1)[:, :n]
    if s.shape[0] != m:
        s = s.repeat_interleave(BLOCK, 0)[:m]
    return q.float() * s


def _plain_matmul(state):
    a, b = _plain_spread(state["a"], state["sa"]), _plain_spread(state["b"], state["sb"])
    return torch.matmul(a, b.t()).to(TYPES[state["case"]["out"]])


def _plain_places(state):
    """Where each expert's rows are, padded to the fullest expert, and where each row went: no sizes leave the GPU."""
    off = state["offsets"].long()
    rows, E, dev = state["x"].shape[0], off.numel() - 1, off.device
    at = off[:-1, None] + torch.arange(state["most"], device=dev)
    held = at < off[1:, None]
    r = torch.arange(rows, device=dev)
    expert = (r[:, None] >= off[None, 1:]).sum(1).clamp_max(E - 1)
    place = (r - off[expert]).clamp(0, state["most"] - 1)
    inside = (r >= off[0]) & (r < off[-1])
    return at.clamp_max(rows - 1), held, expert, place, inside


def _plain_padded(x, at, held):
    return torch.where(held[:, :, None], x[at].float(), 0.0)


def _plain_grouped(state):
    at, held, expert, place, inside = _plain_places(state)
    x, w = state["x"], state["w"]
    y = torch.bmm(_plain_padded(x, at, held), w.transpose(1, 2).to(torch.float32, memory_format=torch.contiguous_format))
    return torch.where(inside[:, None], y[expert, place], 0.0).to(x.dtype)


def _plain_grouped_grad(state):
    at, held, expert, place, inside = _plain_places(state)
    dy = _plain_padded(state["dy"], at, held)
    dx = torch.bmm(dy, state["w"].float())
    dx = torch.where(inside[:, None], dx[expert, place], 0.0).to(state["dy"].dtype)
    dw = torch.bmm(dy.transpose(1, 2).contiguous(), _plain_padded(state["x"], at, held))
    return {"dx": dx, "dw": dw}


# --------------------------------------------------------------------- run
def _own(state):
    import matrix_roots_amd as mr

    case = state["case"]
    op = case["op"]
    if op == "norm":
        r = mr.rms_norm_forward(state["x"], state["weight"], state["eps"], residual=state["residual"], keep_y=case["keep_y"], eight=case["eight"] or None)
        out = {"rstd": r.rstd}
        if state["residual"] is not None:
            out["h"] = r.h
        if case["keep_y"]:
            out["y"] = r.y
        if case["eight"]:
            out["q"], out["scales"] = r.q, r.scales
        return out
    if op == "norm_grad":
        dx, dweight = mr.rms_norm_backward(state["dy"], state["h"], state["rstd"], state["weight"], dresidual=state["dresidual"])
        return {"dx": dx, "dweight": dweight}
    if op == "quantize":
        r = mr.quantize_blocks(state["x"], case["eight"], block=case["block"], order=case["order"])
        out = {}
        if case["order"] in ("rows", "both"):
            out["q"], out["scales"] = r.q, r.scales
        if case["order"] in ("columns", "both"):
            out["qt"], out["scales_t"] = r.qt, r.scales_t
        return out
    if op == "matmul":
        return mr.block_scaled_matmul(state["a"], state["sa"], state["b"], state["sb"], out_dtype=TYPES[case["out"]])
    if op == "grouped":
        return mr.grouped_matmul(state["x"], state["w"], state["offsets"])
    return {"dx": mr.grouped_matmul(state["dy"], state["w"], state["offsets"], transpose=True),
            "dw": mr.grouped_weight_grad(state["dy"], state["x"], state["offsets"])}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "quantize": _plain_quantize, "matmul": _plain_matmul,
          "grouped": _plain_grouped, "grouped_grad": _plain_grouped_grad}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    """Bytes: each input read once, each output written once (of the experts those that can hold a row). Flops: of the formulas."""
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, b = case["rows"] * case["width"], BYTES[case["type"]]
        if op == "norm":
            bytes_ = n * b * (3 if case["residual"] else 1) + (n * b if case["keep_y"] else 0) + case["width"] * 4 + case["rows"] * 4
            if case["eight"]:
                bytes_ += n + case["rows"] * _blocks(case["width"]) * 4
            return {"bytes": bytes_, "flops": 8 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + case["rows"] * 4 + case["width"] * 8, "flops": 12 * n}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        ways = 2 if case["order"] == "both" else 1
        return {"bytes": n * (BYTES[case["type"]] + ways) + ways * n * 4 // (BLOCK if case["block"] == "vector" else BLOCK * BLOCK), "flops": 3 * n}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + m * _blocks(k) * 4 + m * n * BYTES[case["out"]], "flops": 2.0 * m * n * k}
    E, r, n, k, b = case["experts"], case["rows"] - case["spare"], case["n"], case["k"], BYTES[case["type"]]
    used = min(E, r)
    if op == "grouped":
        return {"bytes": b * (case["rows"] * n + r * k + used * n * k), "flops": 2.0 * r * n * k}
    return {"bytes": b * (r * n + r * k + case["rows"] * k + used * n * k) + 4 * E * n * k, "flops": 4.0 * r * n * k}


# ------------------------------------------------------------------- exact
def _exact_blocks(y, eight, tall):
    """The definition block row by block row: scale, then the nearest 8-bit value to y / scale (ties to even), as float64."""
    dtype, top = EIGHT[eight]
    m, n = y.shape
    column = torch.arange(n, device=y.device) // BLOCK
    row = torch.arange(m, device=y.device) // tall
    s = torch.zeros(_blocks(m) if tall > 1 else m, _blocks(n), dtype=torch.float64, device=y.device)
    for j in range(_blocks(n)):
        peak = y[:, j * BLOCK:(j + 1) * BLOCK].abs().max(1).values
        s[:, j] = s[:, j].scatter_reduce(0, row, peak, "amax")
    s = torch.maximum(s, torch.full_like(s, SMALLEST)) / top
    v = y / s[row][:, column]
    fraction, lowest = (3, -6) if eight == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(lowest) - fraction)
    return torch.round(v / step) * step, s


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = state["x"].double()
        if state["residual"] is not None:
            h = (h + state["residual"].double()).to(state["x"].dtype).double()
        rstd = (torch.einsum("ij,ij->i", h, h) / case["width"] + state["eps"]) ** -0.5
        y = torch.einsum("ij,i,j->ij", h, rstd, state["weight"].double())
        out = {"rstd": rstd}
        if state["residual"] is not None:
            out["h"] = h
        if case["keep_y"]:
            out["y"] = y
        if case["eight"]:
            out["q"], out["scales"] = _exact_blocks(y, case["eight"], 1)
        return out
    if op == "norm_grad":
        dy, h, rstd, w = (state[k].double() for k in ("dy", "h", "rstd", "weight"))
        inner = torch.einsum("ij,j,ij->i", dy, w, h)
        dx = torch.einsum("i,ij,j->ij", rstd, dy, w) - torch.einsum("i,ij->ij", rstd ** 3 * inner / case["width"], h)
        if state["dresidual"] is not None:
            dx += state["dresidual"].double()
        return {"dx": dx, "dweight": torch.einsum("ij,ij,i->j", dy, h, rstd)}
    if op == "quantize":
        x = state["x"].double()
        tall = BLOCK if case["block"] == "square" else 1
        out = {}
        if case["order"] != "columns":
            out["q"], out["scales"] = _exact_blocks(x, case["eight"], tall)
        if case["order"] != "rows":
            out["qt"], out["scales_t"] = _exact_blocks(x.T, case["eight"], tall)
        return out
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        c = torch.zeros(m, n, dtype=torch.float64, device=state["a"].device)
        column = torch.arange(n, device=c.device) // (BLOCK if case["b_block"] == "square" else 1)
        for j in range(_blocks(k)):  # block by block of the contraction, the scales outside the sums
            part = state["a"][:, j * BLOCK:(j + 1) * BLOCK].double() @ state["b"][:, j * BLOCK:(j + 1) * BLOCK].double().T.contiguous()
            c += part * state["sa"][:, j].double()[:, None] * state["sb"][column, j].double()[None, :]
        return c
    off = [int(v) for v in state["offsets"].tolist()]
    x, w = state["x"], state["w"]
    if op == "grouped":
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=x.device)
        for e in range(case["experts"]):
            if off[e + 1] > off[e]:
                y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]].double() @ w[e].double().T.contiguous()
        return y
    dy = state["dy"]
    dx = torch.zeros(case["rows"], case["k"], dtype=torch.float64, device=x.device)
    dw = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    for e in range(case["experts"]):
        if off[e + 1] > off[e]:
            d = dy[off[e]:off[e + 1]].double()
            dx[off[e]:off[e + 1]] = d @ w[e].double()
            dw[e] = d.T.contiguous() @ x[off[e]:off[e + 1]].double()
    return {"dx": dx, "dw": dw}
