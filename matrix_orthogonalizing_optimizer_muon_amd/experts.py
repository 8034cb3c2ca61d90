"""Operators of a mixture-of-experts layer: routing, products grouped by expert,
the way back to the tokens, the gated activation and 8-bit activation
checkpoints, each with its backward pass (include/muon.h, "Operators of a
mixture-of-experts layer").  Training a layer's matrices with MuonPlan takes
the gradients these give.

    r = route(logits, k)                                 # T x E -> choices and row order
    gu = grouped_matmul(x, w_gate_up, r.offsets, rows=r.rows)
    h, kept = gated(gu, checkpoint="int8")               # gu may be dropped now
    y = grouped_matmul(h, w_down, r.offsets)
    out = combine(y, r.slots, r.weights)

Autograd does not see these calls: the backward functions here are called by
the program (or by its own torch.autograd.Function).  So that no gradient is
lost unnoticed, a tensor that requires grad is refused while grad mode is on;
pass it detached, or call under torch.no_grad().

Tensors are contiguous, on one GPU, float32 or bfloat16; outputs are new
tensors.  Calls are asynchronous on the current stream, or on ``stream`` (of the
tensors' GPU; a Stream or a handle), which then owns the outputs; inputs made on another stream have to be waited for
before, and kept until this one is done with them, as with any tensor.
"""
import ctypes
import functools
from typing import NamedTuple

import torch

from . import _lib as L

__all__ = ["route", "route_backward", "Routing", "grouped_matmul", "grouped_input_grad", "grouped_weight_grad",
           "combine", "combine_backward", "checkpoint", "restore", "Checkpoint", "gated", "gated_backward"]

BLOCK = 32   # columns of one row that share a checkpoint scale

_CODE = {torch.float32: L.MUON_F32, torch.bfloat16: L.MUON_BF16}
_KIND = {"int8": (L.MUON_INT8, torch.int8), "e4m3": (L.MUON_E4M3, torch.float8_e4m3fn)}
_KIND_OF = {torch.int8: L.MUON_INT8, torch.float8_e4m3fn: L.MUON_E4M3}
_I32 = torch.int32


class Routing(NamedTuple):
    """What route() returns; rows are the (token, choice) pairs sorted by expert."""
    weights: torch.Tensor   # T x k float32
    experts: torch.Tensor   # T x k int32, -1 where nothing was left to choose
    slots: torch.Tensor     # T x k int32: the row of each choice, -1
    rows: torch.Tensor      # T k int32: the token of each row, -1 past the last
    offsets: torch.Tensor   # E + 1 int32: expert e has rows offsets[e] to offsets[e + 1]


class Checkpoint:
    """A matrix kept in 8 bits: q (int8 or float8_e4m3fn) times 2^(scale - 127)
    for each block of 32 columns of a row; dtype is what it restores to."""
    __slots__ = ("q", "scale", "dtype", "kind")

    def __init__(self, q, scale, dtype):
        if not isinstance(q, torch.Tensor) or not isinstance(scale, torch.Tensor):
            raise TypeError("q and scale must be tensors")
        if q.dtype not in _KIND_OF:
            raise ValueError(f"q must be int8 or float8_e4m3fn, not {q.dtype}")
        if dtype not in _CODE:
            raise ValueError(f"unsupported dtype {dtype}")
        if q.dim() != 2 or scale.dtype != torch.uint8 or scale.shape != (q.shape[0], -(-q.shape[1] // BLOCK)):
            raise ValueError("q must be rows x cols and scale rows x ceil(cols / 32) uint8")
        self.q, self.scale, self.dtype, self.kind = q, scale, dtype, _KIND_OF[q.dtype]

    @property
    def shape(self):
        return self.q.shape

    @property
    def nbytes(self):
        return self.q.numel() + self.scale.numel()


# ---------------------------------------------------------------------- checks

def _matrix(name, t, dims=2):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} is not a tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _like(name, t, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} is not a tensor")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, not {t.dtype} of {tuple(t.shape)}")


def _offsets(t, experts=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("offsets is not a tensor")
    if t.dtype != _I32 or t.dim() != 1 or t.shape[0] < 2:
        raise ValueError("offsets must be int32 of experts + 1 entries")
    if experts is not None and t.shape[0] != experts + 1:
        raise ValueError(f"offsets has {t.shape[0]} entries for {experts} experts")


def _rows(t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("rows is not a tensor")
    if t.dtype != _I32 or t.dim() != 1:
        raise ValueError("rows must be int32 with one dimension")


def _placed(*named):
    """The GPU all tensors of (name, tensor, ...) are on, by index; they must be contiguous, and
    not require grad while grad mode is on."""
    dev = named[1].get_device()
    for t in named[1::2]:
        if t.get_device() != dev or dev < 0 or not t.is_contiguous() or t.requires_grad:
            _misplaced(named)
    return dev


def _misplaced(named):
    """Raises for what _placed found, if it is wrong (a tensor that requires grad is not under no_grad)."""
    dev = named[1].device
    if torch.is_grad_enabled():
        for name, t in zip(named[::2], named[1::2]):
            if t.requires_grad:
                raise ValueError(f"{name} requires grad, which autograd would lose here: call under torch.no_grad(), "
                                 "or pass it detached, and call the backward functions")
    for name, t in zip(named[::2], named[1::2]):
        if not t.is_cuda:
            raise ValueError(f"{name} is not on the GPU")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {named[0]} on {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} is not contiguous")


def _device(values):
    """Where the first tensor or Checkpoint of an operator's arguments is, None without one."""
    for t in values:
        if isinstance(t, Checkpoint):
            t = t.q
        if isinstance(t, torch.Tensor):
            return t.device
    return None


def _on(fn):
    """Adds ``stream`` to an operator: it runs, and allocates, on that stream."""
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        dev = _device((*args, *kw.values()))
        if dev is None or dev.type != "cuda":
            return fn(*args, **kw)            # which refuses it
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        elif stream.device != dev:
            raise ValueError(f"stream is of {stream.device}, the tensors are on {dev}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    call.__name__, call.__qualname__, call.__doc__ = fn.__name__, fn.__name__, fn.__doc__
    return call


def _call(dev, fn, *args):
    """fn(*args, stream) on dev's current stream, with dev the current device (the library launches there)."""
    if dev == torch.cuda.current_device():
        code = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _stream(dev))
    if code:
        L.check(code)


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# the stream's handle without a Stream object around it, where this torch has it: a third of a small call's time
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)


def _ptr(t):
    return t.data_ptr()


# --------------------------------------------------------------------- routing

@functools.lru_cache(maxsize=256)
def _route_workspace(tokens, experts):
    need = ctypes.c_uint64()
    L.check(L.lib().muon_route_workspace(tokens, experts, ctypes.byref(need)))
    return need.value


@_on
def route(logits, k, *, normalize=True):
    """The k largest of each token's logits (T x E), ties to the lowest expert, and the
    order of the rows by expert (muon_route).  -inf masks an expert; NaN counts as
    -inf.  normalize: weights over the chosen, else over all experts."""
    code = _matrix("logits", logits)
    tokens, experts = logits.shape
    k = int(k)
    if not 1 <= k <= experts:
        raise ValueError(f"k must be in [1, {experts}], not {k}")
    dev = _placed("logits", logits)
    lib = L.lib()
    weights = logits.new_empty((tokens, k), dtype=torch.float32)
    chosen = logits.new_empty((tokens, k), dtype=_I32)
    slots = torch.empty_like(chosen)
    rows = logits.new_empty(tokens * k, dtype=_I32)
    offsets = logits.new_empty(experts + 1, dtype=_I32)
    need = _route_workspace(tokens, experts)
    ws = logits.new_empty(need, dtype=torch.uint8) if need else None
    _call(dev, lib.muon_route, _ptr(logits), code, tokens, experts, k, 1 if normalize else 0, _ptr(weights),
          _ptr(chosen), _ptr(slots), _ptr(rows), _ptr(offsets), _ptr(ws) if ws is not None else None, need)
    return Routing(weights, chosen, slots, rows, offsets)


@_on
def route_backward(dweights, logits, routing, *, normalize=True):
    """The logits' gradient from that of the weights (muon_route_backward); routing
    is what route() gave for these logits with the same ``normalize``."""
    code = _matrix("logits", logits)
    tokens, experts = logits.shape
    k = routing.weights.shape[1] if routing.weights.dim() == 2 else 0
    _like("weights", routing.weights, torch.float32, (tokens, k))
    _like("experts", routing.experts, _I32, (tokens, k))
    _like("dweights", dweights, torch.float32, (tokens, k))
    dev = _placed("logits", logits, "dweights", dweights, "weights", routing.weights, "experts", routing.experts)
    out = torch.empty_like(logits)
    _call(dev, L.lib().muon_route_backward, _ptr(dweights), _ptr(logits), _ptr(routing.weights),
          _ptr(routing.experts), code, tokens, experts, k, 1 if normalize else 0, _ptr(out))
    return out


# -------------------------------------------------------------------- products

@_on
def grouped_matmul(x, w, offsets, *, rows=None):
    """y[r] = x[rows[r]] W_e^T for the rows r of expert e, zero past the last expert's
    (muon_grouped_matmul).  x: rows x inner; w: E x outer x inner; rows None: x[r]."""
    code = _matrix("x", x)
    if _matrix("w", w, 3) != code:
        raise ValueError(f"x is {x.dtype}, w {w.dtype}")
    experts, outer, inner = w.shape
    if x.shape[1] != inner:
        raise ValueError(f"x has {x.shape[1]} columns, w {inner}")
    _offsets(offsets, experts)
    n = x.shape[0]
    if rows is None:
        dev = _placed("x", x, "w", w, "offsets", offsets)
    else:
        _rows(rows)
        n = rows.shape[0]
        dev = _placed("x", x, "w", w, "offsets", offsets, "rows", rows)
    y = x.new_empty((n, outer))
    _call(dev, L.lib().muon_grouped_matmul, _ptr(x), _ptr(w), _ptr(offsets), None if rows is None else _ptr(rows),
          code, n, x.shape[0], experts, outer, inner, _ptr(y))
    return y


@_on
def grouped_input_grad(dy, w, offsets):
    """dx[r] = dy[r] W_e for the rows r of expert e, zero past the last expert's
    (muon_grouped_input_grad).  dy: n x outer; w: E x outer x inner."""
    code = _matrix("dy", dy)
    if _matrix("w", w, 3) != code:
        raise ValueError(f"dy is {dy.dtype}, w {w.dtype}")
    experts, outer, inner = w.shape
    if dy.shape[1] != outer:
        raise ValueError(f"dy has {dy.shape[1]} columns, w {outer} rows a matrix")
    _offsets(offsets, experts)
    dev = _placed("dy", dy, "w", w, "offsets", offsets)
    n = dy.shape[0]
    dx = dy.new_empty((n, inner))
    _call(dev, L.lib().muon_grouped_input_grad, _ptr(dy), _ptr(w), _ptr(offsets), code, n, experts, outer, inner,
          _ptr(dx))
    return dx


@_on
def grouped_weight_grad(dy, x, offsets, *, rows=None):
    """dW_e = sum over the rows r of expert e of dy[r]^T x[rows[r]], zero for an expert
    without rows (muon_grouped_weight_grad).  dy: n x outer; x: rows x inner, a tensor or
    its Checkpoint; rows None: x[r].  Returns E x outer x inner in dy's dtype."""
    code = _matrix("dy", dy)
    kept = isinstance(x, Checkpoint)
    if not kept:
        _matrix("x", x)
    if x.dtype != dy.dtype:
        raise ValueError(f"dy is {dy.dtype}, x {x.dtype}")
    _offsets(offsets)
    experts, (n, outer), (x_rows, inner) = offsets.shape[0] - 1, dy.shape, x.shape
    placed = ["dy", dy, "offsets", offsets]
    placed += ["q", x.q, "scale", x.scale] if kept else ["x", x]
    if rows is not None:
        _rows(rows)
        placed += ["rows", rows]
    if n != (x_rows if rows is None else rows.shape[0]):
        raise ValueError(f"dy has {n} rows, x or rows {x_rows if rows is None else rows.shape[0]}")
    dev = _placed(*placed)
    lib = L.lib()
    dw = dy.new_empty((experts, outer, inner))
    need = ctypes.c_uint64()
    L.check(lib.muon_grouped_weight_grad_workspace(code, n, x_rows, experts, outer, inner, 1 if kept else 0,
                                                   ctypes.byref(need)))
    ws = dy.new_empty(need.value, dtype=torch.uint8) if need.value else None
    _call(dev, lib.muon_grouped_weight_grad, _ptr(dy), None if kept else _ptr(x), _ptr(x.q) if kept else None,
          _ptr(x.scale) if kept else None, x.kind if kept else 0, _ptr(offsets), None if rows is None else _ptr(rows),
          code, n, x_rows, experts, outer, inner, _ptr(dw), _ptr(ws) if ws is not None else None, need.value)
    return dw


# --------------------------------------------------------------------- combine

def _choices(y, slots, weights):
    code = _matrix("y", y)
    if not isinstance(slots, torch.Tensor):
        raise TypeError("slots is not a tensor")
    if slots.dim() != 2 or slots.dtype != _I32 or slots.shape[1] < 1:
        raise ValueError("slots must be int32, tokens x k")
    _like("weights", weights, torch.float32, slots.shape)
    if y.shape[0] != slots.numel():
        raise ValueError(f"y has {y.shape[0]} rows for {slots.numel()} choices")
    return code


@_on
def combine(y, slots, weights):
    """out[t] = sum_j weights[t][j] y[slots[t][j]] (muon_combine).  y: T k x cols, the rows'
    outputs; slots and weights: T x k, as route() gives them."""
    code = _choices(y, slots, weights)
    dev = _placed("y", y, "slots", slots, "weights", weights)
    (tokens, k), cols = slots.shape, y.shape[1]
    out = y.new_empty((tokens, cols))
    _call(dev, L.lib().muon_combine, _ptr(y), _ptr(slots), _ptr(weights), code, tokens, k, cols, _ptr(out))
    return out


@_on
def combine_backward(dout, y, slots, weights, offsets):
    """(dy, dweights) of combine (muon_combine_backward): dy[slots[t][j]] = weights[t][j] dout[t],
    zero past the last expert's rows; dweights[t][j] = <y[slots[t][j]], dout[t]>."""
    code = _choices(y, slots, weights)
    (tokens, k), cols = slots.shape, y.shape[1]
    _like("dout", dout, y.dtype, (tokens, cols))
    _offsets(offsets)
    dev = _placed("dout", dout, "y", y, "slots", slots, "weights", weights, "offsets", offsets)
    dy, dw = torch.empty_like(y), torch.empty_like(weights)
    _call(dev, L.lib().muon_combine_backward, _ptr(dout), _ptr(y), _ptr(slots), _ptr(weights), _ptr(offsets), code,
          tokens, k, offsets.shape[0] - 1, cols, _ptr(dy), _ptr(dw))
    return dy, dw


# ----------------------------------------------------------------- checkpoints

def _kept(kind, rows, cols, dtype, src):
    q = src.new_empty((rows, cols), dtype=_KIND[kind][1])
    scale = src.new_empty((rows, -(-cols // BLOCK)), dtype=torch.uint8)
    c = Checkpoint.__new__(Checkpoint)
    c.q, c.scale, c.dtype, c.kind = q, scale, dtype, _KIND[kind][0]
    return c


def _kind(kind):
    if kind not in _KIND:
        raise ValueError(f"kind must be 'int8' or 'e4m3', not {kind!r}")


@_on
def checkpoint(x, kind="int8"):
    """x (rows x cols) in 8 bits (muon_checkpoint).  kind: "int8" or "e4m3"."""
    _kind(kind)
    code = _matrix("x", x)
    dev = _placed("x", x)
    rows, cols = x.shape
    c = _kept(kind, rows, cols, x.dtype, x)
    _call(dev, L.lib().muon_checkpoint, _ptr(x), code, rows, cols, c.kind, _ptr(c.q), _ptr(c.scale))
    return c


@_on
def restore(c):
    """The dense matrix of a Checkpoint, in its dtype (muon_restore)."""
    if not isinstance(c, Checkpoint):
        raise TypeError("restore takes a Checkpoint")
    dev = _placed("q", c.q, "scale", c.scale)
    rows, cols = c.shape
    x = c.scale.new_empty((rows, cols), dtype=c.dtype)
    _call(dev, L.lib().muon_restore, _ptr(c.q), _ptr(c.scale), c.kind, rows, cols, _CODE[c.dtype], _ptr(x))
    return x


@_on
def gated(gu, checkpoint=None):
    """h = g sigmoid(g) u of gu = [g | u] (rows x 2 cols) (muon_gated).  checkpoint "int8" or
    "e4m3": returns (h, Checkpoint of gu), from one pass over gu."""
    code = _matrix("gu", gu)
    rows, cols = gu.shape[0], gu.shape[1] // 2
    if gu.shape[1] != 2 * cols or not cols:
        raise ValueError(f"gu must have an even number of columns, not {gu.shape[1]}")
    if checkpoint is not None:
        _kind(checkpoint)
    dev = _placed("gu", gu)
    h = gu.new_empty((rows, cols))
    if checkpoint is None:
        _call(dev, L.lib().muon_gated, _ptr(gu), code, rows, cols, 0, _ptr(h), None, None)
        return h
    c = _kept(checkpoint, rows, 2 * cols, gu.dtype, gu)
    _call(dev, L.lib().muon_gated, _ptr(gu), code, rows, cols, c.kind, _ptr(h), _ptr(c.q), _ptr(c.scale))
    return h, c


@_on
def gated_backward(dh, gu):
    """(dgu, h) of gated (muon_gated_backward): gu's gradient from that of h, and h again
    (the next product's weight gradient reads it).  gu: the tensor, or its Checkpoint."""
    code = _matrix("dh", dh)
    kept = isinstance(gu, Checkpoint)
    if not kept:
        _matrix("gu", gu)
    rows, cols = dh.shape
    if gu.dtype != dh.dtype or tuple(gu.shape) != (rows, 2 * cols) or not cols:
        raise ValueError(f"gu must be {dh.dtype} of shape {(rows, 2 * cols)}, not {gu.dtype} of {tuple(gu.shape)}")
    dev = _placed("dh", dh, "q", gu.q, "scale", gu.scale) if kept else _placed("dh", dh, "gu", gu)
    dgu = dh.new_empty((rows, 2 * cols))
    h = torch.empty_like(dh)
    _call(dev, L.lib().muon_gated_backward, _ptr(dh), None if kept else _ptr(gu), _ptr(gu.q) if kept else None,
          _ptr(gu.scale) if kept else None, gu.kind if kept else 0, code, rows, cols, _ptr(dgu), _ptr(h))
    return dgu, h
