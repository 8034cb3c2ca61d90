"""Operators over a vocabulary: the embedding of tokens and the classifier's losses
(cross entropy, distillation from a teacher's top logits) without the logits in
memory, each with its gradients (include/muon.h, "Operators over a vocabulary").
They give the gradients that AdamWPlan takes for a model's embedding and
classifier.

    h = embed(tokens, table)
    loss, lse, dx, dw = classifier_loss_grads(dloss, x, w, targets)   # a training step
    loss, lse = classifier_loss(x, w, targets)                        # log-probabilities
    dtable = embed_backward(dh, tokens, vocab)

Tokens, targets and ids are int32 or int64; one outside [0, vocab) names
nothing: its embedding is zeros, and a row whose target (or whole teacher)
names nothing has loss and lse 0, gradient zero, and costs nothing (but in a
small call without gradients, where all rows are computed).

Tensors, streams and autograd are treated as the expert-layer operators treat
them (experts.py): contiguous float32 or bfloat16 tensors on one GPU, outputs
new, the backward functions called by the program.
"""
import ctypes
import functools

import torch

from . import _lib as L
from .experts import _call, _like, _matrix, _on, _placed, _ptr

__all__ = ["embed", "embed_backward", "classifier_loss", "classifier_loss_grads", "classifier_loss_backward",
           "distill_loss", "distill_loss_grads", "distill_loss_backward"]

_INDEX = {torch.int32: 4, torch.int64: 8}
_F32 = torch.float32


# ---------------------------------------------------------------------- checks

def _indices(name, t, dims=1):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} is not a tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimension{'s' * (dims > 1)}, not {t.dim()}")
    size = _INDEX.get(t.dtype)
    if size is None:
        raise ValueError(f"{name} must be int32 or int64, not {t.dtype}")
    return size


def _classifier(x, w, targets, name, dims):
    """(dtype code, index bytes) of the arguments that all losses share."""
    code = _matrix("x", x)
    if _matrix("w", w) != code:
        raise ValueError(f"x is {x.dtype}, w {w.dtype}")
    if x.shape[1] != w.shape[1]:
        raise ValueError(f"x has {x.shape[1]} columns, w {w.shape[1]}")
    size = _indices(name, targets, dims)
    if targets.shape[0] != x.shape[0]:
        raise ValueError(f"{name} has {targets.shape[0]} rows, x {x.shape[0]}")
    return code, size


def _teacher(teacher, ids, temperature):
    code = _matrix("teacher", teacher)
    if teacher.shape != ids.shape:
        raise ValueError(f"teacher has shape {tuple(teacher.shape)}, ids {tuple(ids.shape)}")
    temperature = float(temperature)
    if not 0 < temperature < float("inf"):
        raise ValueError(f"temperature must be positive and finite, not {temperature}")
    if not 2.0 ** -63 <= temperature <= 2.0 ** 63:
        raise ValueError(f"temperature must be in [2^-63, 2^63], not {temperature}")
    return code, temperature


@functools.lru_cache(maxsize=256)
def _workspace(name, *args):
    need = ctypes.c_uint64()
    L.check(getattr(L.lib(), name)(*args, ctypes.byref(need)))
    return need.value


def _room(like, need):
    return like.new_empty(need, dtype=torch.uint8) if need else None


def _at(t):
    return None if t is None else _ptr(t)


# ------------------------------------------------------------------- embedding

@_on
def embed(tokens, table, *, scale=1.0):
    """out[t] = scale table[tokens[t]], zeros where tokens[t] names no row (muon_embed).
    tokens: n; table: vocab x dim."""
    size = _indices("tokens", tokens)
    code = _matrix("table", table)
    dev = _placed("tokens", tokens, "table", table)
    out = table.new_empty((tokens.shape[0], table.shape[1]))
    _call(dev, L.lib().muon_embed, _ptr(tokens), size, _ptr(table), code, tokens.shape[0], *table.shape, scale,
          _ptr(out))
    return out


@_on
def embed_backward(dout, tokens, vocab, *, scale=1.0):
    """dtable[v] = scale times the sum of dout[t] over the t with tokens[t] = v, in dout's
    dtype (muon_embed_backward).  dout: n x dim; tokens: n."""
    code = _matrix("dout", dout)
    size = _indices("tokens", tokens)
    n, dim = dout.shape
    if tokens.shape[0] != n:
        raise ValueError(f"dout has {n} rows for {tokens.shape[0]} tokens")
    vocab = int(vocab)
    if vocab < 1:
        raise ValueError(f"vocab must be >= 1, not {vocab}")
    dev = _placed("dout", dout, "tokens", tokens)
    need = _workspace("muon_embed_backward_workspace", n, vocab, dim)
    dtable, ws = dout.new_empty((vocab, dim)), _room(dout, need)
    _call(dev, L.lib().muon_embed_backward, _ptr(dout), _ptr(tokens), size, code, n, vocab, dim, scale, _ptr(dtable),
          _at(ws), need)
    return dtable


# --------------------------------------------------------------- cross entropy

def _losses(x):
    out = x.new_empty((2, x.shape[0]), dtype=_F32)
    return out[0], out[1]


@_on
def classifier_loss(x, w, targets):
    """(loss, lse): lse[t] the log of the sum over v of exp(<x[t], w[v]>), loss[t] =
    lse[t] - <x[t], w[targets[t]]>, both float32 (muon_classifier_loss).  x: n x dim;
    w: vocab x dim; targets: n."""
    code, size = _classifier(x, w, targets, "targets", 1)
    dev = _placed("x", x, "w", w, "targets", targets)
    dims = (x.shape[0], *w.shape)
    need = _workspace("muon_classifier_loss_workspace", code, *dims, 0)
    (loss, lse), ws = _losses(x), _room(x, need)
    _call(dev, L.lib().muon_classifier_loss, _ptr(x), _ptr(w), _ptr(targets), size, code, *dims, _ptr(loss), _ptr(lse),
          _at(ws), need)
    return loss, lse


@_on
def classifier_loss_grads(dloss, x, w, targets):
    """(loss, lse, dx, dw): classifier_loss, and the gradients of x and w for the loss's
    gradient dloss (n, float32), from one pass (muon_classifier_loss_grads)."""
    code, size = _classifier(x, w, targets, "targets", 1)
    _like("dloss", dloss, _F32, (x.shape[0],))
    dev = _placed("x", x, "dloss", dloss, "w", w, "targets", targets)
    dims = (x.shape[0], *w.shape)
    need = _workspace("muon_classifier_loss_workspace", code, *dims, 1)
    (loss, lse), ws = _losses(x), _room(x, need)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    _call(dev, L.lib().muon_classifier_loss_grads, _ptr(dloss), _ptr(x), _ptr(w), _ptr(targets), size, code, *dims,
          _ptr(loss), _ptr(lse), _ptr(dx), _ptr(dw), _at(ws), need)
    return loss, lse, dx, dw


@_on
def classifier_loss_backward(dloss, x, w, targets, lse):
    """(dx, dw) of classifier_loss from its lse; the logits are computed again
    (muon_classifier_loss_backward).  Where dloss is known before the loss,
    classifier_loss_grads does less."""
    code, size = _classifier(x, w, targets, "targets", 1)
    _like("dloss", dloss, _F32, (x.shape[0],))
    _like("lse", lse, _F32, (x.shape[0],))
    dev = _placed("x", x, "dloss", dloss, "w", w, "targets", targets, "lse", lse)
    dims = (x.shape[0], *w.shape)
    need = _workspace("muon_classifier_loss_workspace", code, *dims, 2)
    ws, dx, dw = _room(x, need), torch.empty_like(x), torch.empty_like(w)
    _call(dev, L.lib().muon_classifier_loss_backward, _ptr(dloss), _ptr(x), _ptr(w), _ptr(targets), _ptr(lse), size,
          code, *dims, _ptr(dx), _ptr(dw), _at(ws), need)
    return dx, dw


# ---------------------------------------------------------------- distillation

@_on
def distill_loss(x, w, teacher, ids, *, temperature=1.0):
    """(loss, lse) of x's logits against a teacher's k largest: teacher (n x k, float32 or
    bfloat16) the teacher's logits at ids (n x k).  With q their softmax over temperature,
    loss[t] = temperature^2 sum_j q_j (log q_j - l_j / temperature + lse[t]), lse that of
    the logits over temperature (muon_distill_loss).  An entry whose id names nothing, or
    whose logit is -inf or NaN, is not there."""
    code, size = _classifier(x, w, ids, "ids", 2)
    tcode, tau = _teacher(teacher, ids, temperature)
    dev = _placed("x", x, "w", w, "teacher", teacher, "ids", ids)
    dims = (x.shape[0], *w.shape, ids.shape[1])
    need = _workspace("muon_distill_loss_workspace", code, *dims, 0)
    (loss, lse), ws = _losses(x), _room(x, need)
    _call(dev, L.lib().muon_distill_loss, _ptr(x), _ptr(w), _ptr(teacher), tcode, _ptr(ids), size, code, *dims, tau,
          _ptr(loss), _ptr(lse), _at(ws), need)
    return loss, lse


@_on
def distill_loss_grads(dloss, x, w, teacher, ids, *, temperature=1.0):
    """(loss, lse, dx, dw): distill_loss, and the gradients of x and w for the loss's
    gradient dloss (n, float32), from one pass (muon_distill_loss_grads)."""
    code, size = _classifier(x, w, ids, "ids", 2)
    tcode, tau = _teacher(teacher, ids, temperature)
    _like("dloss", dloss, _F32, (x.shape[0],))
    dev = _placed("x", x, "dloss", dloss, "w", w, "teacher", teacher, "ids", ids)
    dims = (x.shape[0], *w.shape, ids.shape[1])
    need = _workspace("muon_distill_loss_workspace", code, *dims, 1)
    (loss, lse), ws = _losses(x), _room(x, need)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    _call(dev, L.lib().muon_distill_loss_grads, _ptr(dloss), _ptr(x), _ptr(w), _ptr(teacher), tcode, _ptr(ids), size,
          code, *dims, tau, _ptr(loss), _ptr(lse), _ptr(dx), _ptr(dw), _at(ws), need)
    return loss, lse, dx, dw


@_on
def distill_loss_backward(dloss, x, w, teacher, ids, lse, *, temperature=1.0):
    """(dx, dw) of distill_loss from its lse; the logits are computed again
    (muon_distill_loss_backward)."""
    code, size = _classifier(x, w, ids, "ids", 2)
    tcode, tau = _teacher(teacher, ids, temperature)
    _like("dloss", dloss, _F32, (x.shape[0],))
    _like("lse", lse, _F32, (x.shape[0],))
    dev = _placed("x", x, "dloss", dloss, "w", w, "teacher", teacher, "ids", ids, "lse", lse)
    dims = (x.shape[0], *w.shape, ids.shape[1])
    need = _workspace("muon_distill_loss_workspace", code, *dims, 2)
    ws, dx, dw = _room(x, need), torch.empty_like(x), torch.empty_like(w)
    _call(dev, L.lib().muon_distill_loss_backward, _ptr(dloss), _ptr(x), _ptr(w), _ptr(teacher), tcode, _ptr(ids),
          _ptr(lse), size, code, *dims, tau, _ptr(dx), _ptr(dw), _at(ws), need)
    return dx, dw
