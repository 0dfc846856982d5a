"""The operators of the linear layers whose weights the preconditioner steps:
norm, 8-bit quantisation, block-scaled and expert-grouped products.

Argument marshalling over libmatrix_roots.so, like binding.py: torch tensors
provide device memory and the current stream, every step of the computation
runs in the library's HIP kernels, and nothing waits for the device.
With `stream` the kernels run there, on inputs that the caller has ordered with
it; new results come from that stream's memory and are used on the current
stream once the caller has ordered that.
Matrices are 2-D with unit column stride.  Nothing here is recorded for
autograd; the gradients are calls of their own.  Weight gradients come out in
float32, as gram_ema_update and momentum_ema_batched take them.
"""

from __future__ import annotations

from ctypes import addressof
from typing import NamedTuple, Optional

import torch

from . import binding as B
from .binding import _check, _in_use_here, _in_use_on, _memory_of, _ptr, _workspace, library

_FLOATS = {torch.float32: B.MR_F32, torch.float16: B.MR_F16, torch.bfloat16: B.MR_BF16}
_EIGHTS = {torch.float8_e4m3fn: B.MR_E4M3, torch.float8_e5m2: B.MR_E5M2}
_EIGHT_NAMES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_BLOCKS = {"vector": B.MR_BLOCK_VECTOR, "square": B.MR_BLOCK_SQUARE}
BLOCK = 128


class RmsNormOut(NamedTuple):
    h: torch.Tensor  # x + residual (x itself without a residual)
    rstd: torch.Tensor
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


class Quantized(NamedTuple):
    q: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    qt: Optional[torch.Tensor]
    scales_t: Optional[torch.Tensor]


def _device(first, *others):
    """The one GPU the tensors are on, which has to be torch's current one."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one GPU")
    if index < 0:
        raise ValueError("all tensors must be on one GPU")
    if index != torch.cuda.current_device():
        raise ValueError(f"tensors are on GPU {index}, not on the current one")
    return first.device


# The current stream's handle without a Stream object around it (2 us of a 10 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    return _raw_stream(dev.index) if _raw_stream is not None else int(torch.cuda.current_stream(dev).cuda_stream)


def _ld(t) -> int:
    """Leading dimension in elements (any that fits, where there is one row at most)."""
    if t.dim() != 2:
        raise ValueError("matrices must be 2-D with unit column stride")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError("matrices must be 2-D with unit column stride")
    return ld if rows > 1 else (cols + 15) // 16 * 16


def _same_shape(name, t, shape):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")


def _float_code(t, name="the operand") -> int:
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is {t.dtype}: float32, float16 or bfloat16 is needed")
    return code


def _norm_weight(weight, x):
    if weight.dim() != 1 or weight.shape[0] != x.shape[1] or (weight.stride(0) != 1 and weight.shape[0] > 1):
        raise ValueError("weight must be contiguous, one value per column")
    if weight.dtype != torch.float32 and weight.dtype != x.dtype:
        raise ValueError("weight must be float32 or of x's type")
    return _FLOATS[weight.dtype]


def _eight(rows, cols, name, dev):
    """Uninitialised 8-bit matrix whose rows are whole 16-byte units."""
    if name not in _EIGHT_NAMES:
        raise ValueError(f"unknown 8-bit type {name!r}: 'e4m3' or 'e5m2'")
    t = torch.empty(rows, (cols + 15) // 16 * 16, dtype=_EIGHT_NAMES[name], device=dev)
    return t if t.shape[1] == cols else t[:, :cols]


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def rms_norm_forward(x, weight, eps: float, residual=None, keep_y: bool = True, eight: Optional[str] = None,
                     stream=None) -> RmsNormOut:
    """Root-mean-square norm of the rows of x (+ residual), y = h rstd weight.

    x, residual: (rows, width) of one type, float32, float16 or bfloat16;
    weight: (width,), float32 or of that type.  keep_y: return y.  eight
    ("e4m3" or "e5m2"): return y in 8 bits with float32 scales (rows,
    ceil(width / 128)), quantised from the float32 y.
    """
    dev = _device(x, weight, residual)
    code = _float_code(x, "x")
    rows, width = x.shape
    w_code = _norm_weight(weight, x)
    if residual is not None:
        _same_shape("residual", residual, x.shape)
        if residual.dtype != x.dtype:
            raise ValueError("residual must have x's type")
    if not keep_y and eight is None:
        raise ValueError("keep_y or eight: one output at least")
    with _memory_of(stream):
        h = torch.empty(rows, width, dtype=x.dtype, device=dev) if residual is not None else None
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        y = torch.empty(rows, width, dtype=x.dtype, device=dev) if keep_y else None
        q = _eight(rows, width, eight, dev) if eight is not None else None
        scales = torch.empty(rows, _blocks(width), dtype=torch.float32, device=dev) if eight is not None else None
    p = B.RmsNormProblem(rows, width, _ptr(x), _ld(x), _ptr(residual), _ld(residual) if residual is not None else 0,
                         _ptr(weight), _ptr(h), width, _ptr(rstd), _ptr(y), width, _ptr(q),
                         (width + 15) // 16 * 16, _ptr(scales), _blocks(width), code, w_code,
                         _EIGHTS[q.dtype] if q is not None else 0, 0, float(eps))
    if stream is not None:
        _in_use_here(stream, h, rstd, y, q, scales)
        _in_use_on(stream, h, rstd, y, q, scales)
    _check(library().rms_norm_forward(addressof(p), _stream(stream, dev)))
    return RmsNormOut(h if residual is not None else x, rstd, y, q, scales)


def rms_norm_backward(dy, h, rstd, weight, dresidual=None, weight_grad: bool = True, stream=None):
    """(dx, dweight) of rms_norm_forward: dx of dy's type is the gradient of x and
    of the residual, with dresidual (what reaches h by the residual path)
    added; dweight (width,) float32, or None without weight_grad."""
    dev = _device(dy, h, rstd, weight, dresidual)
    code = _float_code(dy, "dy")
    rows, width = dy.shape
    for name, t in (("h", h), ("dresidual", dresidual)):
        if t is not None:
            _same_shape(name, t, dy.shape)
            if t.dtype != dy.dtype:
                raise ValueError(f"{name} must have dy's type")
    if rstd.dtype != torch.float32 or rstd.dim() != 1 or rstd.shape[0] != rows or (rows > 1 and rstd.stride(0) != 1):
        raise ValueError("rstd must be contiguous float32, one value per row")
    w_code = _norm_weight(weight, dy)
    with _memory_of(stream):
        dx = torch.empty(rows, width, dtype=dy.dtype, device=dev)
        dweight = torch.empty(width, dtype=torch.float32, device=dev) if weight_grad else None
    p = B.RmsNormGradProblem(rows, width, _ptr(dy), _ld(dy), _ptr(h), _ld(h), _ptr(rstd), _ptr(weight),
                             _ptr(dresidual), _ld(dresidual) if dresidual is not None else 0, _ptr(dx), width,
                             _ptr(dweight), code, w_code)
    lib = library()
    need = lib.rms_norm_backward_workspace(addressof(p))
    with _memory_of(stream):
        ws = _workspace(need, dev)
    if stream is not None:
        _in_use_here(stream, dx, dweight)
        _in_use_on(stream, ws, dx, dweight)
    _check(lib.rms_norm_backward(addressof(p), _ptr(ws), need, _stream(stream, dev)))
    return dx, dweight


def quantize_blocks(x, eight: str = "e4m3", block: str = "vector", order: str = "rows", stream=None) -> Quantized:
    """x (m, n) in 8 bits with float32 scales, one per block of 128.

    order "rows": q (m, n) with scales; "columns": qt = the transposed (n, m)
    with scales_t; "both": both from one reading.  block "vector": 128
    consecutive values of a row of q (of qt), scales (m, ceil(n / 128));
    "square": 128 x 128, scales (ceil(m / 128), ceil(n / 128)).
    """
    dev = _device(x)
    code = _float_code(x, "x")
    if block not in _BLOCKS:
        raise ValueError(f"unknown block {block!r}: 'vector' or 'square'")
    if order not in ("rows", "columns", "both"):
        raise ValueError(f"unknown order {order!r}: 'rows', 'columns' or 'both'")
    m, n = x.shape
    square = block == "square"
    q = s = qt = st = None
    with _memory_of(stream):
        if order != "columns":
            q = _eight(m, n, eight, dev)
            s = torch.empty(_blocks(m) if square else m, _blocks(n), dtype=torch.float32, device=dev)
        if order != "rows":
            qt = _eight(n, m, eight, dev)
            st = torch.empty(_blocks(n) if square else n, _blocks(m), dtype=torch.float32, device=dev)
    p = B.QuantizeProblem(m, n, _ptr(x), _ld(x), _ptr(q), (n + 15) // 16 * 16, _ptr(s), _blocks(n), _ptr(qt),
                          (m + 15) // 16 * 16, _ptr(st), _blocks(m), code, _EIGHTS[(q if q is not None else qt).dtype],
                          _BLOCKS[block], 0)
    if stream is not None:
        _in_use_here(stream, q, s, qt, st)
        _in_use_on(stream, q, s, qt, st)
    _check(library().quantize_blocks(addressof(p), _stream(stream, dev)))
    return Quantized(q, s, qt, st)


def _scales(name, s, rows, k):
    """(block code, leading dimension) of a scale matrix for `rows` rows."""
    if s.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    if s.shape == (rows, _blocks(k)):
        return B.MR_BLOCK_VECTOR, _ld(s)
    _same_shape(name, s, torch.Size((_blocks(rows), _blocks(k))))
    return B.MR_BLOCK_SQUARE, _ld(s)


def _padded(t, ld) -> bool:
    """Whether the last row's bytes up to a multiple of 16 lie in t's memory too."""
    end = t.storage_offset() + (t.shape[0] - 1) * ld + (t.shape[1] + 15) // 16 * 16
    return end <= t.untyped_storage().nbytes()


def block_scaled_matmul(a, sa, b, sb, out_dtype=torch.bfloat16, out=None, accumulate: bool = False, stream=None):
    """a b^T for 8-bit a (m, k) and b (n, k) with scales per block of 128 of k:
    sa (m, ceil(k / 128)) or (ceil(m / 128), ceil(k / 128)), sb alike.  a: e4m3
    or e5m2, b: e4m3.  With `out` (m, n) the result goes there (is added there
    with accumulate), else into a new tensor of out_dtype."""
    dev = _device(a, sa, b, sb, out)
    if a.dtype not in _EIGHTS or b.dtype not in _EIGHTS:
        raise ValueError("a and b must be float8_e4m3fn or float8_e5m2")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError("a and b must be (m, k) and (n, k)")
    m, k = a.shape
    n = b.shape[0]
    a_block, ldsa = _scales("sa", sa, m, k)
    b_block, ldsb = _scales("sb", sb, n, k)
    own = out is None
    if own:
        if accumulate:
            raise ValueError("accumulate needs out")
        with _memory_of(stream):
            out = torch.empty(m, n, dtype=out_dtype, device=dev)
    else:
        _same_shape("out", out, (m, n))
    lda, ldb = _ld(a), _ld(b)
    padded = k % 16 != 0 and _padded(a, lda) and _padded(b, ldb)
    p = B.ScaledMatmulProblem(m, n, k, _ptr(a), lda, _ptr(sa), ldsa, _ptr(b), ldb, _ptr(sb), ldsb, _ptr(out),
                              _ld(out), _EIGHTS[a.dtype], _EIGHTS[b.dtype], _float_code(out, "out"), a_block, b_block,
                              1 if accumulate else 0, 1 if padded else 0, 0)
    lib = library()
    need = lib.block_scaled_matmul_workspace(addressof(p))
    ws = None
    if need:
        with _memory_of(stream):
            ws = _workspace(need, dev)
    if stream is not None:
        _in_use_here(stream, out if own else None)
        _in_use_on(stream, ws, out if own else None)
    _check(lib.block_scaled_matmul(addressof(p), _ptr(ws), need, _stream(stream, dev)))
    return out


def _bank(name, w):
    """(leading dimension, expert stride) of a bank of matrices (experts, n, k)."""
    if w.dim() != 3 or (w.stride(2) != 1 and w.shape[2] > 1):
        raise ValueError(f"{name} must be (experts, n, k) with unit column stride")
    ld = int(w.stride(1)) if w.shape[1] > 1 else (w.shape[2] + 7) // 8 * 8
    least = (w.shape[1] - 1) * ld + w.shape[2]
    return ld, int(w.stride(0)) if w.shape[0] > 1 else (least + 7) // 8 * 8


def _offset_bits(offsets, experts):
    bits = {torch.int32: 32, torch.int64: 64}.get(offsets.dtype)
    if bits is None or offsets.dim() != 1 or offsets.shape[0] != experts + 1 or offsets.stride(0) != 1:
        raise ValueError("offsets must be contiguous int32 or int64, one more than the experts")
    return bits


def grouped_matmul(x, w, offsets, transpose: bool = False, out_dtype=None, out=None, stream=None):
    """Rows of x by their expert's weight: expert e's rows are offsets[e] ..
    offsets[e + 1] - 1 (device integers, never read by the host), w is (experts,
    n, k).  y_r = w_e x_r (rows, n), or with transpose y_r = w_e^T x_r (rows, k),
    the gradient of the rows.  Rows of no expert get zeros.  float16 or
    bfloat16; out_dtype: that type (default) or float32."""
    dev = _device(x, w, offsets, out)
    ldw, w_stride = _bank("w", w)
    experts, n, k = w.shape
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows = x.shape[0]
    if x.dtype != w.dtype:
        raise ValueError("x and w must have one type")
    _same_shape("x", x, (rows, n if transpose else k))
    bits = _offset_bits(offsets, experts)
    own = out is None
    if own:
        with _memory_of(stream):
            out = torch.empty(rows, k if transpose else n, dtype=out_dtype or x.dtype, device=dev)
    else:
        _same_shape("out", out, (rows, k if transpose else n))
    p = B.GroupedProblem(experts, rows, n, k, _ptr(x), _ld(x), _ptr(w), ldw, w_stride, _ptr(offsets), _ptr(out),
                         _ld(out), _float_code(x, "x"), _float_code(out, "out"), bits, 1 if transpose else 0)
    if stream is not None and own:
        _in_use_here(stream, out)
        _in_use_on(stream, out)
    _check(library().grouped_matmul(addressof(p), _stream(stream, dev)))
    return out


def grouped_weight_grad(dy, x, offsets, out_dtype=torch.float32, out=None, accumulate: bool = False, stream=None):
    """(experts, n, k): for each expert the sum over its rows of dy_r x_r^T, dy
    (rows, n), x (rows, k) of one 16-bit type; zeros for an expert without
    rows.  float32 (default) or that type; with `out` it goes there (is added
    there with accumulate)."""
    dev = _device(dy, x, offsets, out)
    if dy.dtype != x.dtype:
        raise ValueError("dy and x must have one type")
    if dy.dim() != 2 or x.dim() != 2 or offsets.dim() != 1:
        raise ValueError("dy and x must be matrices, offsets a vector")
    rows, n = dy.shape
    _same_shape("x", x, (rows, x.shape[1]))
    k = x.shape[1]
    experts = offsets.shape[0] - 1
    bits = _offset_bits(offsets, experts)
    own = out is None
    if own:
        if accumulate:
            raise ValueError("accumulate needs out")
        with _memory_of(stream):
            out = torch.empty(experts, n, k, dtype=out_dtype, device=dev)
    else:
        _same_shape("out", out, (experts, n, k))
    ld, stride = _bank("out", out)
    p = B.GroupedGradProblem(experts, rows, n, k, _ptr(dy), _ld(dy), _ptr(x), _ld(x), _ptr(offsets), _ptr(out), ld,
                             stride, _float_code(dy, "dy"), _float_code(out, "out"), bits, 1 if accumulate else 0)
    if stream is not None and own:
        _in_use_here(stream, out)
        _in_use_on(stream, out)
    _check(library().grouped_weight_grad(addressof(p), _stream(stream, dev)))
    return out
