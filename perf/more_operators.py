"""Cases of the operators around a bank of experts and its training step: layer
norm, the choice of experts for each token, rows sorted by expert and back with
weights, each forward and backward, and the clipping of many gradients by their
common norm.

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
EPS = 1e-5


def listed():
    return [
        # one token of a serving loop: the residual's sum and the layer's 8-bit input, width 1024
        dict(name="layer_norm_token", op="norm", rows=1, width=1024, type="bf16", residual=True, keep_y=False, eight="e4m3"),
        # a training batch at width 2048
        dict(name="layer_norm_batch", op="norm", rows=16384, width=2048, type="bf16", residual=True, keep_y=True, eight=""),
        # its backward pass, with the gradient that comes down the residual
        dict(name="layer_norm_grad_batch", op="norm_grad", rows=16384, width=2048, type="bf16", residual=True),
        # the experts of a few tokens of a serving loop: latency
        dict(name="route_tokens", op="route", tokens=8, experts=64, k=8, type="f32", normalize=True, masked=0.0),
        # the experts of a training batch's tokens, out of a large bank
        dict(name="route_batch", op="route", tokens=16384, experts=384, k=8, type="f32", normalize=True, masked=0.0),
        # backward, odd sizes, shares of the softmax over all experts, some of them switched off
        dict(name="route_grad_odd", op="route_grad", tokens=8191, experts=250, k=6, type="bf16", normalize=False, masked=0.1),
        # a few tokens' rows sorted by expert: latency
        dict(name="dispatch_tokens", op="dispatch", tokens=16, k=8, experts=64, width=2048, type="bf16", dropped=0.0),
        # a training batch's rows sorted by expert, uneven loads
        dict(name="dispatch_batch", op="dispatch", tokens=16384, k=8, experts=64, width=2048, type="bf16", dropped=0.0),
        # the experts' rows of a ragged batch back to their tokens, by weights, added to the residual; some choices are of no expert here
        dict(name="combine_batch", op="combine", tokens=16383, k=8, experts=64, width=2048, type="bf16", dropped=0.03, weighted=True, residual=True),
        # its backward pass at odd sizes: the rows' gradient in expert order and the weights'
        dict(name="combine_grad_odd", op="combine_grad", tokens=4001, k=4, experts=17, width=1337, type="f16", dropped=0.05),
        # the ordinary step: the gradients of the width-1024 set with its norms' vectors, below the limit and left in place
        dict(name="clip_step", op="clip", layers=8, width=1024, experts=0, odd=0, type="f32", out=False, above=False),
        # a bank of 16-bit gradients and odd small ones above the limit, scaled into the float32 that the optimizer's step takes
        dict(name="clip_bank", op="clip", layers=1, width=1536, experts=32, odd=9, type="bf16", out=True, above=True),
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm; a third of them multiples of 128, the others as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.33 and v > 128:
        v = v // 128 * 128
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "route", "route_grad", "dispatch", "dispatch_grad", "combine", "combine_grad", "clip"])
    if op in ("norm", "norm_grad"):
        case = dict(op=op, rows=_size(rng, 1, 16384), width=_size(rng, 64, 8192), type=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.7)
        case["rows"] = max(1, min(case["rows"], 16384 * 2048 // case["width"]))
        if op == "norm":
            case["keep_y"] = rng.random() < 0.7
            case["eight"] = rng.choice(["e4m3", "e5m2", "e4m3"]) if not case["keep_y"] or rng.random() < 0.5 else ""
        return case
    if op in ("route", "route_grad"):
        return dict(op=op, tokens=_size(rng, 1, 16384), experts=_size(rng, 8, 384), k=rng.randint(1, 8), type=rng.choice(["f32", "f32", "bf16", "f16"]),
                    normalize=rng.random() < 0.6, masked=rng.choice([0.0, 0.0, 0.1]))
    if op == "clip":
        width = _size(rng, 64, 1536)
        case = dict(op=op, layers=rng.randint(1, 7), width=width, experts=rng.choice([0, 0, 4, 17]), odd=rng.randint(0, 9), type=rng.choice(["f32", "bf16", "f16"]))
        case["out"] = rng.random() < 0.5
        case["above"] = case["out"] and rng.random() < 0.8
        while work(case)["bytes"] > 6e8:
            case["width"] = case["width"] * 4 // 5
        return case
    case = dict(op=op, tokens=_size(rng, 1, 16384), k=rng.randint(1, 8), experts=rng.choice([1, 3, 8, 17, 64, 384]), width=_size(rng, 64, 4096),
                type=rng.choice(["bf16", "bf16", "f16", "f32"]), dropped=rng.choice([0.0, 0.0, 0.05, 0.4]))
    most = 16384 * 8 * 2048 * (1 if op == "combine_grad" else 2)  # bytes of the sorted rows, which a backward pass moves twice
    case["tokens"] = max(1, min(case["tokens"], most // (case["k"] * case["width"] * BYTES[case["type"]])))
    if op == "combine":
        case["weighted"] = rng.random() < 0.8
        case["residual"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _activations(rows, cols, g, dev):
    """Rows of differing size and mean with a few large channels, as hidden states have them."""
    x = torch.randn(rows, cols, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=dev))
    x += 0.3 * torch.randn(rows, 1, generator=g, device=dev)
    channels = torch.randint(0, cols, (max(1, cols // 200),), generator=g, device=dev)
    x[:, channels] *= 8.0
    return x


def _shapes(case):
    """Of a set of gradients: per layer four square matrices, up, down and the norms' vectors; a bank of experts; vectors and matrices of odd sizes."""
    w = case["width"]
    shapes = []
    for _ in range(case["layers"]):
        shapes += [(w, w)] * 4 + [(w, 4 * w), (4 * w, w), (2, w)]
    if case["experts"]:
        shapes.append((case["experts"], w, w))
    return shapes + [(17 * i + 1, 3 * i + 1) if i % 2 else (131 * i + 7,) for i in range(case["odd"])]


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    t = TYPES[case["type"]]
    state = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if op in ("norm", "norm_grad"):
        rows, width = case["rows"], case["width"]
        state["weight"] = 1.0 + 0.1 * randn(width)
        state["bias"] = 0.1 * randn(width)
        x = _activations(rows, width, g, dev).to(t)
        if op == "norm":
            state["x"] = x
            state["residual"] = (2.0 * randn(rows, width)).to(t) if case["residual"] else None
        else:
            v = x.double()
            state["h"] = x
            state["mean"] = v.mean(1).float()
            state["rstd"] = ((v - v.mean(1, keepdim=True)).square().mean(1) + EPS).rsqrt().float()
            state["dy"] = randn(rows, width).to(t)
            state["dresidual"] = randn(rows, width).to(t) if case["residual"] else None
    elif op in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        logits = (1.5 * randn(T, E) + randn(E)).to(t)
        if case["masked"] and E > 2 * k:
            off = torch.rand(T, E, generator=g, device=dev) < case["masked"]
            off[:, : k + 1] = False  # enough experts stay
            logits = torch.where(off, torch.full_like(logits, -math.inf), logits)
        state["logits"] = logits
        if op == "route_grad":
            state["dweights"] = randn(T, k)
            state["experts"], state["weights"], state["log_sum"] = _plain_route(state).values()
    elif op == "clip":
        grads = [(0.02 * randn(*s)).to(t) for s in _shapes(case)]
        state["grads"] = grads
        norm = math.sqrt(sum(float(x.double().square().sum()) for x in grads))
        state["max_norm"] = 0.37 * norm if case["above"] else 1.5 * norm
        state["outs"] = [torch.empty(x.shape, dtype=torch.float32, device=dev) for x in grads] if case["out"] else None
    else:
        T, k, E, W = case["tokens"], case["k"], case["experts"], case["width"]
        # distinct experts for each token where there are enough, popular ones more often; some choices of no expert here (-1)
        score = randn(T, E) + 0.7 * randn(E)
        chosen = torch.cat([torch.topk(score, min(k, E), dim=1).indices] + [torch.randint(0, E, (T, 1), generator=g, device=dev)] * max(0, k - E), 1)
        away = torch.rand(T, k, generator=g, device=dev) < case["dropped"]
        state["experts"] = torch.where(away, torch.full_like(chosen, -1), chosen).to(torch.int32)
        if op == "dispatch":
            state["x"] = _activations(T, W, g, dev).to(t)
        else:
            state["offsets"], state["place"] = _plain_order(state["experts"], E)
            state["rows"] = _activations(T * k, W, g, dev).to(t)
            if op == "combine_grad" or case.get("weighted"):
                state["weights"] = torch.softmax(randn(T, k), 1)
            if op == "combine_grad":
                state["dout"] = randn(T, W).to(t)
            state["residual"] = randn(T, W).to(t) if case.get("residual") else None
    return state


# ------------------------------------------------------------ plain forms
def _plain_eight(y, eight):
    """(8-bit values, scales) of float32 y for blocks of 128 of a row."""
    dtype, top = EIGHT[eight]
    m, n = y.shape
    tiles = torch.nn.functional.pad(y, (0, _blocks(n) * BLOCK - n)).view(m, _blocks(n), BLOCK)
    s = tiles.abs().amax(2).clamp_min(SMALLEST) / top
    return (tiles / s[:, :, None]).view(m, -1)[:, :n].to(dtype), s


def _plain_norm(state):
    case = state["case"]
    h = state["x"]
    if state["residual"] is not None:
        h = (h.float() + state["residual"].float()).to(h.dtype)
    v = h.float()
    mean = v.mean(1)
    c = v - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS)
    y = c * rstd[:, None] * state["weight"] + state["bias"]
    out = {"mean": mean, "rstd": rstd}
    if state["residual"] is not None:
        out["h"] = h
    if case["keep_y"]:
        out["y"] = y.to(h.dtype)
    if case["eight"]:
        out["q"], out["scales"] = _plain_eight(y, case["eight"])
    return out


def _plain_norm_grad(state):
    t = state["dy"].dtype
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    xhat = (state["h"].float() - state["mean"][:, None]) * rstd
    g = dy * state["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if state["dresidual"] is not None:
        dx = dx + state["dresidual"].float()
    return {"dx": dx.to(t), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def _plain_route(state):
    """The k largest logits of a row, ties to the lowest index, and their shares of the softmax (over all, or over themselves)."""
    case = state["case"]
    l = state["logits"].float()
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    v, i = v[:, : case["k"]], i[:, : case["k"]]
    top = v[:, :1]
    log_sum = torch.log(torch.exp((v if case["normalize"] else l) - top).sum(1)) + top[:, 0]
    return {"experts": i.to(torch.int32), "weights": torch.exp(v - log_sum[:, None]), "log_sum": log_sum}


def _plain_route_grad(state):
    case = state["case"]
    l, w, at = state["logits"].float(), state["weights"], state["experts"].long()
    mean = (w * state["dweights"]).sum(1, keepdim=True)
    if case["normalize"]:
        d = torch.zeros_like(l)
    else:
        d = -torch.exp(l - state["log_sum"][:, None]) * mean
    part = w * (state["dweights"] - mean) if case["normalize"] else w * state["dweights"]
    return {"dlogits": d.scatter_add(1, at, part).to(state["logits"].dtype)}


def _plain_order(experts, n):
    """Where each expert's rows begin, and the row of every choice: sorted by expert, then by token; choices of no expert last."""
    e = experts.reshape(-1).long()
    e = torch.where((e < 0) | (e >= n), torch.full_like(e, n), e)
    by = torch.sort(e, stable=True).indices
    place = torch.empty_like(by)
    place[by] = torch.arange(by.numel(), device=by.device)
    edges = torch.searchsorted(e[by], torch.arange(n + 1, device=by.device))
    return edges.to(torch.int32), place.view(experts.shape).to(torch.int32)


def _plain_dispatch(state):
    case = state["case"]
    offsets, place = _plain_order(state["experts"], case["experts"])
    x = state["x"]
    rows = torch.empty(place.numel(), x.shape[1], dtype=x.dtype, device=x.device)
    kept = place.reshape(-1) < offsets[-1]
    each = x[:, None, :].expand(-1, case["k"], -1).reshape(-1, x.shape[1])
    rows[place.reshape(-1).long()] = torch.where(kept[:, None], each, torch.zeros_like(each))
    return {"offsets": offsets, "place": place, "rows": rows}


def _plain_combine(state):
    kept = state["place"] < state["offsets"][-1]
    y = torch.where(kept[:, :, None], state["rows"][state["place"].long()].float(), 0.0)
    if "weights" in state:
        y = y * state["weights"][:, :, None]
    out = y.sum(1)
    if state["residual"] is not None:
        out = out + state["residual"].float()
    return {"out": out.to(state["rows"].dtype)}


def _plain_combine_grad(state):
    kept = state["place"] < state["offsets"][-1]
    dout, at = state["dout"].float(), state["place"].long()
    y = torch.where(kept[:, :, None], state["rows"][at].float(), 0.0)
    drows = torch.empty_like(state["rows"])
    each = torch.where(kept, state["weights"], 0.0)[:, :, None] * dout[:, None, :]
    drows[at] = each.to(drows.dtype)
    return {"drows": drows, "dweights": (y * dout[:, None, :]).sum(2)}


def _plain_clip(state):
    squares = torch.stack([x.double().square().sum() for x in state["grads"]])
    norm = squares.sum().sqrt()
    by = torch.where(norm > state["max_norm"], state["max_norm"] / norm, 1.0).float()
    out = {"norm": norm, "norms": squares.sqrt()}
    if state["outs"] is not None:
        out["grads"] = [x.float() * by for x in state["grads"]]
    else:  # in place; below the limit the values stay
        for x in state["grads"]:
            x.copy_(x.float() * by)
        out["grads"] = state["grads"]
    return out


# --------------------------------------------------------------------- run
def _own(state):
    import matrix_roots_amd as mr

    case = state["case"]
    op = case["op"]
    if op == "norm":
        r = mr.layer_norm_forward(state["x"], state["weight"], state["bias"], EPS, residual=state["residual"], keep_y=case["keep_y"], eight=case["eight"] or None)
        out = {"mean": r.mean, "rstd": r.rstd}
        if state["residual"] is not None:
            out["h"] = r.h
        if case["keep_y"]:
            out["y"] = r.y
        if case["eight"]:
            out["q"], out["scales"] = r.q, r.scales
        return out
    if op == "norm_grad":
        dx, dweight, dbias = mr.layer_norm_backward(state["dy"], state["h"], state["mean"], state["rstd"], state["weight"], dresidual=state["dresidual"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "route":
        r = mr.route_tokens(state["logits"], case["k"], normalize=case["normalize"])
        return {"experts": r.experts, "weights": r.weights, "log_sum": r.log_sum}
    if op == "route_grad":
        routed = mr.Routed(state["experts"], state["weights"], state["log_sum"])
        return {"dlogits": mr.route_tokens_backward(state["dweights"], state["logits"], routed, normalize=case["normalize"])}
    if op == "dispatch":
        order = mr.order_by_expert(state["experts"], case["experts"])
        return {"offsets": order.offsets, "place": order.place, "rows": mr.dispatch_rows(state["x"], order)}
    if op == "clip":
        norm, norms = mr.clip_gradients_batched(state["grads"], state["max_norm"], outs=state["outs"], return_norms=True)
        return {"norm": norm, "norms": norms, "grads": state["grads"] if state["outs"] is None else state["outs"]}
    order = mr.ExpertOrder(state["offsets"], state["place"])
    if op == "dispatch_grad":
        return {"out": mr.dispatch_rows_backward(state["rows"], order)}
    if op == "combine":
        return {"out": mr.combine_rows(state["rows"], order, weights=state.get("weights"), residual=state["residual"])}
    drows, dweights = mr.combine_rows_backward(state["dout"], state["rows"], order, state["weights"])
    return {"drows": drows, "dweights": dweights}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "route": _plain_route, "route_grad": _plain_route_grad, "dispatch": _plain_dispatch,
          "dispatch_grad": _plain_combine, "combine": _plain_combine, "combine_grad": _plain_combine_grad, "clip": _plain_clip}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    """Bytes: each input read once, each output written once. Flops: of the formulas."""
    op, b = case["op"], BYTES[case["type"]]
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["width"]
        if op == "norm":
            bytes_ = n * b * (3 if case["residual"] else 1) + (n * b if case["keep_y"] else 0) + case["width"] * 8 + case["rows"] * 8
            if case["eight"]:
                bytes_ += n + case["rows"] * _blocks(case["width"]) * 4
            return {"bytes": bytes_, "flops": 10 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + case["rows"] * 8 + case["width"] * 12, "flops": 15 * n}
    if op in ("route", "route_grad"):
        n, c = case["tokens"] * case["experts"], case["tokens"] * case["k"]
        if op == "route":
            return {"bytes": n * b + c * 8 + case["tokens"] * 4, "flops": n * (case["k"] + 3)}
        return {"bytes": n * b * (1 if case["normalize"] else 2) + c * 12 + case["tokens"] * 4, "flops": 4 * n}
    if op == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        return {"bytes": n * b + (n * 4 if case["out"] else 0), "flops": 3 * n}
    T, c, W = case["tokens"], case["tokens"] * case["k"], case["width"]
    held = int(round(c * (1 - case["dropped"])))  # rows of an expert; the others are not read
    if op == "dispatch":
        return {"bytes": c * 8 + case["experts"] * 4 + T * W * b + c * W * b, "flops": c}
    if op == "combine_grad":
        return {"bytes": c * 12 + T * W * b + (held + c) * W * b, "flops": 3 * held * W}
    return {"bytes": c * (8 if case.get("weighted") else 4) + held * W * b + T * W * b * (2 if case.get("residual") else 1), "flops": 2 * held * W}


# ------------------------------------------------------------------- exact
def _exact_eight(y, eight):
    """Block by block: scale, then the nearest 8-bit value to y / scale (ties to even), as float64."""
    top = EIGHT[eight][1]
    s = torch.stack([y[:, j * BLOCK:(j + 1) * BLOCK].abs().max(1).values for j in range(_blocks(y.shape[1]))], 1)
    s = torch.maximum(s, torch.full_like(s, SMALLEST)) / top
    v = y / s[:, torch.arange(y.shape[1], device=y.device) // BLOCK]
    fraction, lowest = (3, -6) if eight == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(lowest) - fraction)
    return torch.round(v / step) * step, s


def _exact_route(logits, k, normalize):
    """One choice after another: the largest of what is left, the first of equal ones."""
    l = logits.double()
    left = l.clone()
    number = torch.arange(l.shape[1], device=l.device)
    experts = []
    for _ in range(k):
        peak = left.max(1, keepdim=True).values
        first = torch.where(left == peak, number, l.shape[1]).min(1).values
        experts.append(first)
        left[torch.arange(l.shape[0], device=l.device), first] = -math.inf
    experts = torch.stack(experts, 1)
    chosen = torch.gather(l, 1, experts)
    log_sum = torch.logsumexp(chosen if normalize else l, 1)
    return experts, torch.exp(chosen - log_sum[:, None]), log_sum


def _exact_order(experts, n):
    """An expert's rows begin behind all choices of lower ones; a choice's row is behind those of its expert at earlier places."""
    e = experts.reshape(-1).long()
    e = torch.where((e < 0) | (e >= n), n, e)
    counts = torch.bincount(e, minlength=n + 1)
    begin = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(e)
    for i in range(n + 1):
        at = torch.nonzero(e == i)[:, 0]
        place[at] = begin[i] + torch.arange(at.numel(), device=e.device)
    return begin.to(torch.int32), place.view(experts.shape).to(torch.int32)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = state["x"].double()
        if state["residual"] is not None:
            h = (h + state["residual"].double()).to(state["x"].dtype).double()
        mean = torch.einsum("ij->i", h) / case["width"]
        rstd = (torch.einsum("ij,ij->i", h - mean[:, None], h - mean[:, None]) / case["width"] + EPS) ** -0.5
        y = torch.einsum("ij,i,j->ij", h - mean[:, None], rstd, state["weight"].double()) + state["bias"].double()
        out = {"mean": mean, "rstd": rstd}
        if state["residual"] is not None:
            out["h"] = h
        if case["keep_y"]:
            out["y"] = y
        if case["eight"]:
            out["q"], out["scales"] = _exact_eight(y, case["eight"])
        return out
    if op == "norm_grad":
        dy, h, mean, rstd, w = (state[k].double() for k in ("dy", "h", "mean", "rstd", "weight"))
        c = h - mean[:, None]
        inner = torch.einsum("ij,j,ij->i", dy, w, c)
        dx = torch.einsum("i,ij,j->ij", rstd, dy, w) - (rstd * (dy @ w) / case["width"])[:, None] - torch.einsum("i,ij->ij", rstd ** 3 * inner / case["width"], c)
        if state["dresidual"] is not None:
            dx += state["dresidual"].double()
        return {"dx": dx, "dweight": torch.einsum("ij,ij,i->j", dy, c, rstd), "dbias": torch.einsum("ij->j", dy)}
    if op == "route":
        experts, weights, log_sum = _exact_route(state["logits"], case["k"], case["normalize"])
        return {"experts": experts.to(torch.int32), "weights": weights, "log_sum": log_sum}
    if op == "route_grad":
        # the kept weights are the inputs that the pass is given
        l, w, dw, at = state["logits"].double(), state["weights"].double(), state["dweights"].double(), state["experts"].long()
        inner = torch.einsum("ij,ij->i", w, dw)
        d = torch.zeros_like(l) if case["normalize"] else -torch.einsum("ij,i->ij", torch.exp(l - state["log_sum"].double()[:, None]), inner)
        for j in range(case["k"]):
            r = torch.arange(l.shape[0], device=l.device)
            d[r, at[:, j]] += w[:, j] * (dw[:, j] - inner if case["normalize"] else dw[:, j])
        return {"dlogits": d}
    if op == "clip":
        squares = [torch.linalg.vector_norm(x.double().reshape(-1)) ** 2 for x in state["grads"]]
        norm = torch.stack(squares).sum() ** 0.5
        by = min(1.0, state["max_norm"] / float(norm))
        return {"norm": norm, "norms": torch.stack(squares) ** 0.5, "grads": [x.double() * by for x in state["grads"]]}
    offsets, place = _exact_order(state["experts"], case["experts"])
    T, k, W = case["tokens"], case["k"], case["width"]
    held = int(offsets[-1])
    token = torch.empty(T * k, dtype=torch.int64, device=place.device)
    token[place.reshape(-1).long()] = torch.arange(T * k, device=place.device) // k  # the token of each sorted row
    if op == "dispatch":
        rows = torch.zeros(T * k, W, dtype=torch.float64, device=place.device)
        rows[:held] = state["x"][token[:held]].double()
        return {"offsets": offsets, "place": place, "rows": rows}
    weight = torch.ones(T * k, dtype=torch.float64, device=place.device)
    if "weights" in state:
        weight[place.reshape(-1).long()] = state["weights"].reshape(-1).double()
    if op == "combine_grad":
        d = torch.zeros(T * k, W, dtype=torch.float64, device=place.device)
        d[:held] = weight[:held, None] * state["dout"][token[:held]].double()
        dots = torch.zeros(T * k, dtype=torch.float64, device=place.device)
        dots[:held] = torch.einsum("ij,ij->i", state["rows"][:held].double(), state["dout"][token[:held]].double())
        return {"drows": d, "dweights": dots[place.long()]}
    out = torch.zeros(T, W, dtype=torch.float64, device=place.device)
    for b in range(0, held, 1 << 15):
        e = min(held, b + (1 << 15))
        out.index_add_(0, token[b:e], state["rows"][b:e].double() * weight[b:e, None])
    if state["residual"] is not None:
        out += state["residual"].double()
    return {"out": out}
