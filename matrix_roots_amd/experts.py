"""What lies between tokens and the products of a bank of experts (linear.py's
grouped_matmul): the choice of experts, the order of rows by expert, rows to
their experts and back with weights, and the gradients of these.

    routed = route_tokens(logits, k)                  # (tokens, experts) -> experts and weights of each token
    order = order_by_expert(routed.experts, experts)  # where each choice's row goes
    rows = dispatch_rows(x, order)                    # what grouped_matmul(rows, w, order.offsets) takes
    out = combine_rows(y, order, routed.weights)      # its rows back to their tokens

Argument marshalling over libmatrix_roots.so, with linear.py's conventions:
nothing waits for the device, nothing is recorded for autograd, `stream` as
there.
"""

from __future__ import annotations

from ctypes import addressof
from typing import NamedTuple

import torch

from . import binding as B
from . import linear as L
from .binding import _check, _in_use_here, _in_use_on, _memory_of, _ptr, _workspace, library
from .linear import _device, _float_code, _ld, _same_shape, _stream


class Routed(NamedTuple):
    experts: torch.Tensor  # (tokens, k) int32, -1 for no expert
    weights: torch.Tensor  # (tokens, k) float32
    log_sum: torch.Tensor  # (tokens,) float32


class ExpertOrder(NamedTuple):
    offsets: torch.Tensor  # (experts + 1,) int32: expert e's sorted rows are offsets[e] .. offsets[e + 1] - 1
    place: torch.Tensor  # (tokens, k) int32: the sorted row of each choice


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")


def _small(name, t, shape, dtype):
    """A contiguous array of 4-byte values."""
    _same_shape(name, t, shape)
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype}")


def _experts_of(order, tokens) -> tuple:
    """(experts, k) of an order for `tokens` tokens."""
    offsets, place = order
    if place.dim() != 2 or place.shape[0] != tokens:
        raise ValueError("the order is for another number of tokens")
    if offsets.dim() != 1:
        raise ValueError("order.offsets must be a vector")
    for t in order:
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("an order is contiguous int32")
    return offsets.shape[0] - 1, place.shape[1]


def route_tokens(logits, k: int, normalize: bool = True, stream=None) -> Routed:
    """The k experts with the largest logits (tokens, experts) of each token, ties to
    the lowest index, and their weights: shares of the softmax over those k, or with
    normalize False over all experts.  -inf is never chosen; where fewer than k are
    left the expert is -1 and its weight 0.  k up to 16, experts up to 4096."""
    dev = _device(logits)
    code = _float_code(logits, "logits")
    _matrix("logits", logits)
    tokens, experts = logits.shape
    with _memory_of(stream):
        chosen = torch.empty(tokens, k, dtype=torch.int32, device=dev)
        weights = torch.empty(tokens, k, dtype=torch.float32, device=dev)
        log_sum = torch.empty(tokens, dtype=torch.float32, device=dev)
    p = B.RouteProblem(tokens, experts, k, _ptr(logits), _ld(logits), _ptr(chosen), _ptr(weights), _ptr(log_sum), code,
                       1 if normalize else 0)
    if stream is not None:
        _in_use_here(stream, chosen, weights, log_sum)
        _in_use_on(stream, chosen, weights, log_sum)
    _check(library().route_tokens(addressof(p), _stream(stream, dev)))
    return Routed(chosen, weights, log_sum)


def route_tokens_backward(dweights, logits, routed: Routed, normalize: bool = True, stream=None):
    """The logits' gradient, of their type, from that of routed.weights."""
    chosen, weights, _ = routed
    dev = _device(logits, dweights, chosen, weights)
    code = _float_code(logits, "logits")
    _matrix("logits", logits)
    _matrix("dweights", dweights)
    tokens, experts = logits.shape
    k = dweights.shape[1]
    _small("dweights", dweights, (tokens, k), torch.float32)
    _small("routed.experts", chosen, (tokens, k), torch.int32)
    _small("routed.weights", weights, (tokens, k), torch.float32)
    with _memory_of(stream):
        dlogits = torch.empty(tokens, experts, dtype=logits.dtype, device=dev)
    p = B.RouteGradProblem(tokens, experts, k, _ptr(logits), _ld(logits), _ptr(chosen), _ptr(weights), _ptr(dweights),
                           _ptr(dlogits), experts, code, 1 if normalize else 0)
    if stream is not None:
        _in_use_here(stream, dlogits)
        _in_use_on(stream, dlogits)
    _check(library().route_tokens_backward(addressof(p), _stream(stream, dev)))
    return dlogits


def order_by_expert(experts, n_experts: int, stream=None) -> ExpertOrder:
    """The tokens' choices (tokens, k), int32 or int64, sorted by expert and within
    one by token.  Numbers outside 0 .. n_experts - 1 are no expert: their rows come
    last, behind offsets[n_experts]."""
    dev = _device(experts)
    bits = {torch.int32: 32, torch.int64: 64}.get(experts.dtype)
    if bits is None:
        raise ValueError(f"experts is {experts.dtype}: int32 or int64 is needed")
    _matrix("experts", experts)
    tokens, k = experts.shape
    with _memory_of(stream):
        offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
        place = torch.empty(tokens, k, dtype=torch.int32, device=dev)
    p = B.OrderProblem(tokens, n_experts, k, _ptr(experts), _ld(experts), _ptr(offsets), _ptr(place), bits, 0)
    lib = library()
    need = lib.order_by_expert_workspace(addressof(p))
    ws = None
    if need:
        with _memory_of(stream):
            ws = _workspace(need, dev)
    if stream is not None:
        _in_use_here(stream, offsets, place)
        _in_use_on(stream, ws, offsets, place)
    _check(lib.order_by_expert(addressof(p), _ptr(ws), need, _stream(stream, dev)))
    return ExpertOrder(offsets, place)


def dispatch_rows(x, order: ExpertOrder, stream=None):
    """The rows of x (tokens, width) in the order's places (tokens k, width); zeros
    in the rows of no expert."""
    dev = _device(x, *order)
    _matrix("x", x)
    tokens, width = x.shape
    experts, k = _experts_of(order, tokens)
    with _memory_of(stream):
        out = torch.empty(tokens * k, width, dtype=x.dtype, device=dev)
    p = B.DispatchProblem(tokens, experts, k, width, _ptr(x), _ld(x), _ptr(order[1]), _ptr(order[0]), 0, 0, 0, _ptr(out),
                          width, 0, _float_code(x, "x"), 0)
    if stream is not None:
        _in_use_here(stream, out)
        _in_use_on(stream, out)
    _check(library().dispatch_rows(addressof(p), _stream(stream, dev)))
    return out


def dispatch_rows_backward(drows, order: ExpertOrder, stream=None):
    """The gradient of dispatch_rows' x: a token's rows of drows added up."""
    return combine_rows(drows, order, stream=stream)


def combine_rows(y, order: ExpertOrder, weights=None, residual=None, stream=None):
    """(tokens, width): residual_t + sum_j weights_tj y[place_tj], over a token's
    choices that an expert has; added up in float32, of y's type.  y: (tokens k,
    width) in the order's places, weights: (tokens, k) float32."""
    dev = _device(y, *order, weights, residual)
    code = _float_code(y, "y")
    _matrix("y", y)
    _matrix("order.place", order[1])
    tokens, width = order[1].shape[0], y.shape[1]
    experts, k = _experts_of(order, tokens)
    _same_shape("y", y, (tokens * k, width))
    if weights is not None:
        _small("weights", weights, (tokens, k), torch.float32)
    if residual is not None:
        _same_shape("residual", residual, (tokens, width))
        if residual.dtype != y.dtype:
            raise ValueError("residual must have y's type")
    with _memory_of(stream):
        out = torch.empty(tokens, width, dtype=y.dtype, device=dev)
    p = B.CombineProblem(tokens, experts, k, width, _ptr(y), _ld(y), _ptr(order[1]), _ptr(order[0]), _ptr(weights),
                         _ptr(residual), _ld(residual) if residual is not None else 0, _ptr(out), width, code, 0)
    if stream is not None:
        _in_use_here(stream, out)
        _in_use_on(stream, out)
    _check(library().combine_rows(addressof(p), _stream(stream, dev)))
    return out


def combine_rows_backward(dout, y, order: ExpertOrder, weights, stream=None):
    """(drows, dweights) of combine_rows from its output's gradient dout (tokens,
    width), which is the residual's too: drows of y's shape and type, zeros in the
    rows of no expert; dweights (tokens, k) float32, the dot products of dout with
    the rows.  weights None: as if they were 1."""
    dev = _device(dout, y, *order, weights)
    code = _float_code(y, "y")
    _matrix("dout", dout)
    tokens, width = dout.shape
    experts, k = _experts_of(order, tokens)
    _same_shape("y", y, (tokens * k, width))
    if dout.dtype != y.dtype:
        raise ValueError("dout must have y's type")
    if weights is not None:
        _small("weights", weights, (tokens, k), torch.float32)
    with _memory_of(stream):
        drows = torch.empty(tokens * k, width, dtype=y.dtype, device=dev)
        dweights = torch.empty(tokens, k, dtype=torch.float32, device=dev)
    p = B.DispatchProblem(tokens, experts, k, width, _ptr(dout), _ld(dout), _ptr(order[1]), _ptr(order[0]), _ptr(weights),
                          _ptr(y), _ld(y), _ptr(drows), width, _ptr(dweights), code, 0)
    if stream is not None:
        _in_use_here(stream, drows, dweights)
        _in_use_on(stream, drows, dweights)
    _check(library().dispatch_rows(addressof(p), _stream(stream, dev)))
    return drows, dweights
