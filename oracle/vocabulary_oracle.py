"""fp64 oracle of the vocabulary operators, from their definitions (torch tensors
in, float64 tensors out on the same device; no code of the library)."""
import math

import torch


def named(index, vocab):
    """index as int64, -1 where it names nothing."""
    i = index.long()
    return torch.where((i >= 0) & (i < vocab), i, -1)


def embed(tokens, table, scale=1.0):
    t = named(tokens, table.shape[0])
    out = torch.zeros(t.shape[0], table.shape[1], dtype=torch.float64, device=table.device)
    out[t >= 0] = table[t[t >= 0]].double() * scale
    return out


def embed_backward(dout, tokens, vocab, scale=1.0):
    t = named(tokens, vocab)
    out = torch.zeros(vocab + 1, dout.shape[1], dtype=torch.float64, device=dout.device)
    out.index_add_(0, torch.where(t < 0, vocab, t), dout.double())
    return out[:vocab] * scale


def teacher_weights(teacher, ids, vocab, temperature):
    """(ids, q): the entries that are there, and their softmax; q is 0 elsewhere."""
    l = teacher.double()
    at = named(ids, vocab)
    at = torch.where(torch.isnan(l) | (l == -math.inf), -1, at)
    l = l.clamp(max=float(torch.finfo(torch.float32).max))
    l = torch.where(at >= 0, l, -math.inf)
    top = l.max(1, keepdim=True).values
    e = torch.where(at >= 0, torch.exp((l - torch.where(top > -math.inf, top, 0.0)) / temperature), 0.0)
    total = e.sum(1, keepdim=True)
    return at, torch.where(total > 0, e / total, 0.0)


def target_weights(targets, vocab):
    at = named(targets, vocab)[:, None]
    return at, (at >= 0).double()


def loss(x, w, at, q, temperature=1.0):
    """(loss, lse) of the targets at (rows x k, -1: none) with weights q."""
    rows = torch.nonzero((at >= 0).any(1))[:, 0]
    out = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    lse = torch.zeros_like(out)
    z = x[rows].double() @ w.double().t() / temperature
    s = torch.logsumexp(z, 1)
    picked = torch.gather(z, 1, at[rows].clamp_min(0))
    part = torch.where(at[rows] >= 0, torch.xlogy(q[rows], q[rows]) + q[rows] * (s[:, None] - picked), 0.0)
    out[rows] = temperature ** 2 * part.sum(1)
    lse[rows] = s
    return out, lse


def logits_grad(dloss, x, w, at, q, temperature=1.0, lse=None):
    """The gradient of the logits, zero for rows without targets."""
    vocab = w.shape[0]
    z = x.double() @ w.double().t() / temperature
    s = torch.logsumexp(z, 1) if lse is None else lse.double()
    p = torch.exp(z - s[:, None])
    p = torch.cat([p, p.new_zeros(p.shape[0], 1)], 1)
    p.scatter_add_(1, torch.where(at < 0, vocab, at), -q)
    return torch.where((at >= 0).any(1)[:, None], p[:, :vocab], 0.0) * (dloss.double() * temperature)[:, None]


def grads(dloss, x, w, at, q, temperature=1.0, lse=None):
    """(dx, dw)."""
    live = (at >= 0).any(1)[:, None]
    dl = logits_grad(dloss, torch.where(live, x.double(), 0.0), w, at, q, temperature, lse)
    return dl @ w.double(), dl.t() @ torch.where(live, x.double(), 0.0)
