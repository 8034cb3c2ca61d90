"""Measured cases of the vocabulary operators: the embedding and its gradient,
the classifier's cross entropy and distillation from a teacher's top logits,
with their gradients, both without the logits in memory.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits; with ``own`` true it makes the calls a user makes of the
framework.  ``exact`` gives the same outputs from the definition in 64 bits.

The sizes come from the repository's 32000 x 1024 embedding and classifier, from
the widths of its matrix workloads, and from odd neighbours of them.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
IT = {"i32": torch.int32, "i64": torch.int64}
IS = {"i32": 4, "i64": 8}


# ----------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token on its way into the model
        {"name": "embed, one token", "op": "embed", "dtype": "bf16", "index": "i64", "tokens": 1, "vocab": 32000,
         "dim": 1024, "scale": 1.0, "absent": 0.0},
        # a training batch, scaled by the root of the width
        {"name": "embed, training batch", "op": "embed", "dtype": "bf16", "index": "i64", "tokens": 16384,
         "vocab": 32000, "dim": 2048, "scale": 45.25, "absent": 0.0},
        # that batch's gradient: a few tokens make up much of a text, most of the vocabulary is not in it
        {"name": "embedding gradient", "op": "embed_grad", "dtype": "bf16", "index": "i64", "tokens": 16384,
         "vocab": 32000, "dim": 2048, "scale": 45.25, "absent": 0.0},
        # a small fp32 model with odd sizes and padding among its tokens
        {"name": "embedding gradient, fp32 and odd", "op": "embed_grad", "dtype": "f32", "index": "i32", "tokens": 5003,
         "vocab": 4099, "dim": 515, "scale": 1.0, "absent": 0.25},
        # one token's log-probability
        {"name": "loss, one token", "op": "loss", "dtype": "bf16", "index": "i64", "tokens": 1, "vocab": 32000,
         "dim": 1024, "form": "forward", "absent": 0.0},
        # scoring answers behind prompts, whose tokens do not count
        {"name": "loss, scoring", "op": "loss", "dtype": "bf16", "index": "i64", "tokens": 2048, "vocab": 32000,
         "dim": 4096, "form": "forward", "absent": 0.5},
        # the small fp32 model's training step
        {"name": "loss and gradients, fp32 and odd", "op": "loss", "dtype": "f32", "index": "i32", "tokens": 389,
         "vocab": 4099, "dim": 515, "form": "both", "absent": 0.1},
        # gradients of a batch whose losses came before, from the log of the sum that was kept
        {"name": "loss gradients", "op": "loss", "dtype": "bf16", "index": "i64", "tokens": 4096, "vocab": 32000,
         "dim": 1024, "form": "backward", "absent": 0.0},
        # a training step of a wide model
        {"name": "loss and gradients, training batch", "op": "loss", "dtype": "bf16", "index": "i64", "tokens": 8192,
         "vocab": 32000, "dim": 4096, "form": "both", "absent": 0.0},
        # a large vocabulary, padded rows
        {"name": "loss and gradients, large vocabulary", "op": "loss", "dtype": "bf16", "index": "i64", "tokens": 3000,
         "vocab": 131072, "dim": 2048, "form": "both", "absent": 0.1},
        # a few tokens measured against a teacher
        {"name": "distillation, few tokens", "op": "distill", "dtype": "bf16", "index": "i64", "tokens": 24,
         "vocab": 32000, "dim": 1024, "form": "forward", "k": 16, "tau": 1.0, "absent": 0.0},
        # a training step on a teacher's 32 top logits, vocabulary of odd size
        {"name": "distillation, training batch", "op": "distill", "dtype": "bf16", "index": "i64", "tokens": 4096,
         "vocab": 50257, "dim": 2048, "form": "both", "k": 32, "tau": 2.0, "absent": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly multiples of 64 or 8, now and then any number."""
    v = _log(rng, lo, hi)
    step = rng.choice([64, 64, 64, 8, 1])
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "loss", "loss", "loss", "distill", "distill"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = {"op": op, "dtype": dtype, "index": rng.choice(["i32", "i64"]), "absent": rng.choice([0.0, 0.1, 0.5])}
    if op in ("embed", "embed_grad"):
        c["tokens"], c["vocab"], c["dim"] = _log(rng, 1, 32768), _log(rng, 16, 131072), _width(rng, 16, 4096)
        c["scale"] = rng.choice([1.0, round(math.sqrt(c["dim"]), 2)])
        return c
    c["form"] = rng.choice(["forward", "backward", "both"])
    c["vocab"], c["dim"] = _log(rng, 16, 131072), _width(rng, 16, 4096)
    most = 2.0 ** 40 if dtype == "bf16" else 2.0 ** 35    # fp32 products: a sixteenth of the rate, and less
    if c["vocab"] * c["dim"] > most / 16:
        c["vocab"] = int(most / 16 / c["dim"])
    c["tokens"] = _log(rng, 1, max(1, min(8192, int(most / (c["vocab"] * c["dim"])))))
    if op == "distill":
        c["k"] = rng.randint(1, min(128, c["vocab"], _log(rng, 1, 128)))
        c["tau"] = rng.choice([1.0, 2.0, 0.7])
    return c


# ---------------------------------------------------------------------- inputs

def _words(g, n, vocab, dev):
    """Tokens as texts have them: rank r about as often as 1 / r, ranks spread over the vocabulary."""
    u = torch.rand(n, generator=g, device=dev, dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1)).long().clamp(1, vocab) - 1
    stride = int(vocab * 0.618) | 1
    while math.gcd(stride, vocab) > 1:
        stride += 2
    return (rank * stride) % vocab


def _holes(g, t, part, dev):
    """Every so many places set to -1 (padding, prompts)."""
    return torch.where(torch.rand(t.shape[0], generator=g, device=dev) < part, -1, t) if part else t


def _acts(g, rows, cols, dev):
    """Activations behind a norm: normal, with a spread of channel scales."""
    scale = torch.exp(0.3 * torch.randn(cols, generator=g, device=dev))
    return torch.randn(rows, cols, generator=g, device=dev) * scale


def _grads(g, rows, cols, dtype, dev):
    """Gradients: normal rows whose scales spread over tokens."""
    scale = 1e-3 * torch.exp(torch.randn(rows, 1, generator=g, device=dev))
    return (torch.randn(rows, cols, generator=g, device=dev) * scale).to(dtype)


def _make(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt, it = case["op"], DT[case["dtype"]], IT[case["index"]]
    n, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    s = {"case": case}
    words = _words(g, n, vocab, dev)
    if op in ("embed", "embed_grad"):
        s["tokens"] = _holes(g, words, case["absent"], dev).to(it)
        if op == "embed":
            s["table"] = torch.randn(vocab, dim, generator=g, device=dev).mul_(0.02).to(dt)
        else:
            s["dout"] = _grads(g, n, dim, dt, dev)
        return s
    s["w"] = torch.randn(vocab, dim, generator=g, device=dev).mul_(1 / math.sqrt(dim)).to(dt)
    # a trained model: the right token's logit stands out, more or less
    lead = 16 * torch.rand(n, 1, generator=g, device=dev)
    s["x"] = (_acts(g, n, dim, dev) + lead * s["w"][words].float()).to(dt)
    live = _holes(g, words, case["absent"], dev)
    s["dloss"] = torch.rand(n, generator=g, device=dev).add_(0.5) / max(1, int((live >= 0).sum()))
    if op == "loss":
        s["targets"] = live.to(it)
    else:
        # the teacher's k largest, all different, the right one mostly first; some rows have fewer
        k = case["k"]
        gaps = torch.randint(1, max(2, vocab // k + 1), (n, k), generator=g, device=dev)
        gaps[:, 0] = 0
        ids = (words[:, None] + gaps.cumsum(1)) % vocab
        few = torch.rand(n, 1, generator=g, device=dev) < case["absent"]
        count = torch.where(few, torch.randint(1, k + 1, (n, 1), generator=g, device=dev), k)
        ids = torch.where(torch.arange(k, device=dev) < count, ids, -1)
        s["ids"] = torch.where((live < 0)[:, None], -1, ids).to(it)
        t = 2 * torch.randn(n, k, generator=g, device=dev)
        t[:, 0] += 8 * torch.rand(n, generator=g, device=dev)
        s["teacher"] = torch.sort(t, dim=1, descending=True).values
    if case["form"] == "backward":    # what the forward pass kept
        logits = s["x"].float() @ s["w"].float().t()
        lse = torch.logsumexp(logits / case.get("tau", 1.0), 1)
        s["lse"] = torch.where(live < 0, 0.0, lse)
    return s


def prepare(case, seed):
    return _make(case, seed)


# ----------------------------------------------------------------- plain forms

def _plain_embed(s, c):
    t = s["tokens"].long()
    rows = s["table"][t.clamp_min(0)].float() * c["scale"]
    return torch.where((t >= 0)[:, None], rows, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s, c):
    t, d = s["tokens"].long(), s["dout"].float()
    out = torch.zeros(c["vocab"], c["dim"], device=d.device)
    out.index_add_(0, t.clamp_min(0), torch.where((t >= 0)[:, None], d, 0.0))
    return (out * c["scale"]).to(s["dout"].dtype)


def _plain_classifier(s, c):
    """loss, log of the sum, and the gradients; cross entropy is a teacher with one entry."""
    x, w = s["x"].float(), s["w"].float()
    tau = c.get("tau", 1.0)
    if c["op"] == "loss":
        ids = s["targets"].long()[:, None]
        there = ids >= 0
        q = there.float()
        logq = torch.zeros_like(q)
    else:
        ids = s["ids"].long()
        there = ids >= 0
        t = torch.where(there, s["teacher"] / tau, -math.inf)
        top = t.max(1, keepdim=True).values.clamp_min(-1e30)
        e = torch.exp(t - top)
        total = e.sum(1, keepdim=True)
        live = total > 0
        q = torch.where(live, e / total, 0.0)
        logq = torch.where(there, t - top - torch.log(torch.where(live, total, 1.0)), 0.0)
    at = ids.clamp_min(0)
    live = there.any(1)
    l = (x @ w.t()) / tau
    out = []
    if c["form"] == "backward":
        lse = s["lse"]
    else:
        top = l.max(1, keepdim=True).values
        lse = (top + torch.log(torch.exp(l - top).sum(1, keepdim=True)))[:, 0]
        picked = torch.gather(l, 1, at)
        part = torch.where(there, q * (logq - picked + lse[:, None]), 0.0)
        loss = tau * tau * part.sum(1)
        lse = torch.where(live, lse, 0.0)
        out += [torch.where(live, loss, 0.0), lse]
    if c["form"] != "forward":
        p = torch.exp(l - lse[:, None])
        p = p.scatter_add_(1, at, -q)
        dl = torch.where(live[:, None], p, 0.0) * (s["dloss"] * tau)[:, None]
        out += [(dl @ w).to(s["x"].dtype), (dl.t() @ x).to(s["w"].dtype)]
    return out


def _plain(s):
    c = s["case"]
    if c["op"] == "embed":
        return _plain_embed(s, c)
    return _plain_embed_grad(s, c) if c["op"] == "embed_grad" else _plain_classifier(s, c)


# ------------------------------------------------------------- the framework's

def _own(s):
    import matrix_orthogonalizing_optimizer_muon_amd as M
    c = s["case"]
    op = c["op"]
    if op == "embed":
        return M.embed(s["tokens"], s["table"], scale=c["scale"])
    if op == "embed_grad":
        return M.embed_backward(s["dout"], s["tokens"], c["vocab"], scale=c["scale"])
    if op == "loss":
        if c["form"] == "forward":
            return list(M.classifier_loss(s["x"], s["w"], s["targets"]))
        if c["form"] == "backward":
            return list(M.classifier_loss_backward(s["dloss"], s["x"], s["w"], s["targets"], s["lse"]))
        return list(M.classifier_loss_grads(s["dloss"], s["x"], s["w"], s["targets"]))
    if c["form"] == "forward":
        return list(M.distill_loss(s["x"], s["w"], s["teacher"], s["ids"], temperature=c["tau"]))
    if c["form"] == "backward":
        return list(M.distill_loss_backward(s["dloss"], s["x"], s["w"], s["teacher"], s["ids"], s["lse"],
                                            temperature=c["tau"]))
    return list(M.distill_loss_grads(s["dloss"], s["x"], s["w"], s["teacher"], s["ids"], temperature=c["tau"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------ work

def work(case):
    es, ix = ES[case["dtype"]], IS[case["index"]]
    n, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    live = n * (1 - case["absent"])
    if case["op"] == "embed":
        return {"bytes": n * ix + (live + n) * dim * es, "flops": live * dim}
    if case["op"] == "embed_grad":
        return {"bytes": n * ix + (live + vocab) * dim * es, "flops": live * dim}
    k = case.get("k", 1)
    read = live * dim * es + vocab * dim * es + n * k * (ix + (4 if case["op"] == "distill" else 0)) + n * 8
    flops = 2.0 * live * vocab * dim
    if case["form"] == "forward":
        return {"bytes": read, "flops": flops}
    return {"bytes": read + (n + vocab) * dim * es, "flops": 3 * flops}


# ----------------------------------------------------------------------- exact

def exact(case, seed):
    s = _make(case, seed)
    op, vocab = case["op"], case["vocab"]
    if op == "embed":
        t = s["tokens"].long()
        out = torch.zeros(t.shape[0], case["dim"], dtype=torch.float64, device="cuda")
        out[t >= 0] = s["table"][t[t >= 0]].double() * case["scale"]
        return out
    if op == "embed_grad":
        t = s["tokens"].long()
        out = torch.zeros(vocab + 1, case["dim"], dtype=torch.float64, device="cuda")
        out.index_add_(0, torch.where(t < 0, vocab, t), s["dout"].double())
        return out[:vocab] * case["scale"]
    tau = case.get("tau", 1.0)
    # rows that count, and their targets as a matrix of probabilities with the rest of the vocabulary zero
    if op == "loss":
        ids, weight = s["targets"].long()[:, None], torch.zeros(s["x"].shape[0], 1, dtype=torch.float64, device="cuda")
    else:
        ids, weight = s["ids"].long(), s["teacher"].double() / tau
    rows = torch.nonzero((ids >= 0).any(1))[:, 0]
    n, dim = s["x"].shape
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    kept = torch.zeros_like(loss)
    dx = torch.zeros(n, dim, dtype=torch.float64, device="cuda")
    w = s["w"].double()
    dw = torch.zeros_like(w)
    for i in range(0, rows.shape[0], 2048):
        r = rows[i:i + 2048]
        x, id_r = s["x"][r].double(), ids[r]
        q = torch.softmax(torch.where(id_r >= 0, weight[r], -math.inf), 1)
        soft = torch.zeros(r.shape[0], vocab + 1, dtype=torch.float64, device="cuda")
        soft.scatter_add_(1, torch.where(id_r < 0, vocab, id_r), q)
        soft = soft[:, :vocab]
        z = (x @ w.t()) / tau
        logp = torch.log_softmax(z, 1)
        kept[r] = z[:, 0] - logp[:, 0]
        loss[r] = tau ** 2 * ((torch.xlogy(q, q)).sum(1) - (soft * logp).sum(1))
        if case["form"] != "forward":
            if case["form"] == "backward":     # with the log of the sum that was handed in
                logp = z - s["lse"][r].double()[:, None]
            dz = (torch.exp(logp) - soft) * (s["dloss"][r].double() * tau)[:, None]
            dx[r] = dz @ w
            dw += dz.t() @ x
    if case["form"] == "forward":
        return [loss, kept]
    return [dx, dw] if case["form"] == "backward" else [loss, kept, dx, dw]
