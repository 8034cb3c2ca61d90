"""Measured cases of the expert-layer operators: routing, products grouped by
expert, 8-bit activation checkpoints.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits; with ``own`` true it makes the calls a user makes of the
framework.  ``exact`` gives the same outputs from the definition in 64 bits.

The sizes come from the repository's mixture-of-experts workload (64 experts,
gate and up 1408 x 2048, down 2048 x 1408), from its smaller fp32 and bf16
matrices, and from odd neighbours of them.
"""
import math

import torch

own = False

BLOCK = 32        # columns of one row that share a checkpoint scale
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
F32_MAX = torch.finfo(torch.float32).max


# ----------------------------------------------------------------------- cases

def listed():
    return [
        # one token of decoding through gate and up: eight experts' weights are read for eight rows
        {"name": "product, one token", "op": "product", "dtype": "bf16", "tokens": 1, "k": 8, "experts": 64,
         "inner": 2048, "outer": 2816, "idle": 0, "skew": 0.5, "gather": True},
        # a small serving batch through the down projection, some experts idle
        {"name": "product, small batch", "op": "product", "dtype": "bf16", "tokens": 37, "k": 6, "experts": 64,
         "inner": 1408, "outer": 2048, "idle": 5, "skew": 0.5, "gather": False},
        # a small fp32 layer with odd sizes, as a test or a research model has
        {"name": "product, fp32 and odd", "op": "product", "dtype": "f32", "tokens": 389, "k": 2, "experts": 8,
         "inner": 513, "outer": 257, "idle": 1, "skew": 1.0, "gather": True},
        # a training batch through gate and up
        {"name": "product, training batch", "op": "product", "dtype": "bf16", "tokens": 8192, "k": 8, "experts": 64,
         "inner": 2048, "outer": 2816, "idle": 0, "skew": 0.5, "gather": True},
        # the same batch's gradient with respect to the rows
        {"name": "input gradient", "op": "input_grad", "dtype": "bf16", "tokens": 4096, "k": 8, "experts": 64,
         "inner": 2048, "outer": 2816, "idle": 2, "skew": 0.5},
        # the down projection's weight gradient, uneven experts
        {"name": "weight gradient", "op": "weight_grad", "dtype": "bf16", "tokens": 4096, "k": 8, "experts": 64,
         "inner": 1408, "outer": 2048, "idle": 2, "skew": 1.0, "gather": False, "kind": "none"},
        # gate and up's weight gradient from the tokens kept in 8 bits
        {"name": "weight gradient, 8 bits", "op": "weight_grad", "dtype": "bf16", "tokens": 8192, "k": 8, "experts": 64,
         "inner": 2048, "outer": 2816, "idle": 0, "skew": 0.5, "gather": True, "kind": "int8"},
        # tokens into an 8-bit checkpoint and back, ragged
        {"name": "checkpoint and back", "op": "checkpoint", "dtype": "bf16", "rows": 4099, "cols": 2056, "kind": "e4m3"},
        # the gated activation of a training batch, forward and, from its 8-bit checkpoint, backward
        {"name": "gated activation", "op": "gated", "dtype": "bf16", "rows": 32768, "cols": 1408, "kind": "int8"},
        # the router of one decoded token
        {"name": "route, one token", "op": "route", "dtype": "f32", "tokens": 1, "k": 8, "experts": 64,
         "masked": 0, "normalize": True, "grad": False},
        # the router of a training batch with its gradient, some experts masked
        {"name": "route, training batch", "op": "route", "dtype": "f32", "tokens": 16384, "k": 8, "experts": 64,
         "masked": 3, "normalize": True, "grad": True},
        # expert outputs back to their tokens, and the gradient of that
        {"name": "combine", "op": "combine", "dtype": "bf16", "tokens": 8192, "k": 8, "experts": 64, "cols": 2048,
         "masked": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A matrix side: mostly multiples of 64 or 8, now and then any number."""
    v = _log(rng, lo, hi)
    step = rng.choice([64, 64, 64, 8, 1])
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["product", "product", "input_grad", "weight_grad", "weight_grad", "checkpoint", "gated", "route",
                     "combine"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("product", "input_grad", "weight_grad"):
        experts = _log(rng, 2, 64)
        c = {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 8192), "k": rng.randint(1, min(8, experts)),
             "experts": experts, "inner": _width(rng, 64, 2048), "outer": _width(rng, 64, 2816),
             "idle": rng.choice([0, 0, 1]) if experts > 8 else 0, "skew": round(rng.uniform(0, 1), 2)}
        if dtype == "f32":   # a sixteenth of the rate: as much less work
            c["tokens"], c["inner"], c["outer"] = min(c["tokens"], 2048), min(c["inner"], 1408), min(c["outer"], 1408)
        if op != "input_grad":
            c["gather"] = rng.random() < 0.5
        if op == "weight_grad":
            c["kind"] = rng.choice(["none", "int8", "e4m3"])
        return c
    if op == "checkpoint":
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, 16384), "cols": _width(rng, 8, 4096),
                "kind": rng.choice(["int8", "e4m3"])}
    if op == "gated":
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, 32768), "cols": _width(rng, 32, 1408),
                "kind": rng.choice(["int8", "e4m3", "none"])}
    experts = _log(rng, 2, 64 if op == "combine" else 256)
    k = rng.randint(1, min(8, experts))
    if op == "route":
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 16384), "k": k, "experts": experts,
                "masked": rng.choice([0, 1, experts - 1]), "normalize": rng.random() < 0.5,
                "grad": rng.random() < 0.5}
    return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 8192), "k": k, "experts": experts,
            "cols": _width(rng, 64, 2048), "masked": rng.choice([0, 1])}


# ---------------------------------------------------------------------- inputs

def _logits(g, tokens, experts, skew, idle, dev):
    """Router logits: a popularity of the experts, noise of the tokens; the last ``idle`` experts masked."""
    pop = torch.randn(experts, generator=g, device=dev) * skew
    l = pop + torch.randn(tokens, experts, generator=g, device=dev)
    if idle:
        l[:, experts - idle:] = -math.inf
    return l


def _order(l, k):
    """(experts, slots, rows, offsets) of logits without NaN: the k largest of each row, ties to the lowest
    expert, sorted by expert and then by place; what is masked has expert and slot -1."""
    tokens, n_exp = l.shape
    val, ids = torch.sort(l, dim=1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    gone = val == -math.inf
    key = torch.where(gone, n_exp, ids).reshape(-1)
    order = torch.argsort(key, stable=True)
    place = torch.arange(tokens * k, device=l.device)
    slots = torch.empty_like(order)
    slots[order] = place
    slots = torch.where(gone, -1, slots.view(tokens, k)).int()
    count = (key[:, None] == torch.arange(n_exp, device=l.device)).sum(0)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    rows = torch.where(place < offsets[-1], order // k, -1).int()
    return torch.where(gone, -1, ids).int(), slots, rows, offsets


def _acts(g, rows, cols, dtype, dev):
    """Activations: normal, with a spread of channel scales and a few strong channels."""
    scale = torch.exp(0.5 * torch.randn(cols, generator=g, device=dev))
    scale = torch.where(torch.rand(cols, generator=g, device=dev) < 0.005, 20 * scale, scale)
    return (torch.randn(rows, cols, generator=g, device=dev) * scale).to(dtype)


def _grads(g, rows, cols, dtype, dev):
    """Gradients: normal rows whose scales spread over tokens."""
    scale = 1e-3 * torch.exp(torch.randn(rows, 1, generator=g, device=dev))
    return (torch.randn(rows, cols, generator=g, device=dev) * scale).to(dtype)


def _make(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt = case["op"], DT[case["dtype"]]
    s = {"case": case}
    if op in ("product", "input_grad", "weight_grad"):
        l = _logits(g, case["tokens"], case["experts"], case["skew"], case["idle"], dev)
        _, _, rows, offsets = _order(l, case["k"])
        n = case["tokens"] * case["k"]
        s["offsets"] = offsets
        s["cap"] = int((offsets[1:] - offsets[:-1]).max())   # the plain form's padded length
        s["rows"] = rows if case.get("gather") else None
        xr = case["tokens"] if case.get("gather") else n
        if op != "weight_grad":
            s["w"] = torch.randn(case["experts"], case["outer"], case["inner"], generator=g, device=dev,
                                 dtype=dt) * 0.02
        if op != "product":
            s["dy"] = _grads(g, n, case["outer"], dt, dev)
        if op != "input_grad":
            s["x"] = _acts(g, xr, case["inner"], dt, dev)
            if case.get("kind", "none") != "none":   # what the forward pass kept
                s["q"], s["scale"] = _pack(s["x"], case["kind"])
                del s["x"]
    elif op == "checkpoint":
        s["x"] = _acts(g, case["rows"], case["cols"], dt, dev)
    elif op == "gated":
        s["gu"] = _acts(g, case["rows"], 2 * case["cols"], dt, dev)
        s["dh"] = _grads(g, case["rows"], case["cols"], dt, dev)
    else:
        l = _logits(g, case["tokens"], case["experts"], 0.5, case["masked"], dev)
        if op == "route":
            s["logits"] = l.to(dt)
            s["dw"] = torch.randn(case["tokens"], case["k"], generator=g, device=dev)
        else:
            _, s["slots"], _, s["offsets"] = _order(l, case["k"])
            s["weights"] = torch.rand(case["tokens"], case["k"], generator=g, device=dev) / case["k"]
            s["y"] = torch.randn(case["tokens"] * case["k"], case["cols"], generator=g, device=dev, dtype=dt)
            s["dout"] = _grads(g, case["tokens"], case["cols"], dt, dev)
    return s


def prepare(case, seed):
    return _make(case, seed)


# ----------------------------------------------------------------- plain forms

def _pow2(n):
    """2^n in fp32, exactly (n a whole number in [-126, 127])."""
    return ((n.int() + 127) << 23).view(torch.float32)


def _pack(x, kind):
    """(int8 or e4m3 values, scale codes) of blocks of 32 columns; the scale is a power of two."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    m, e = torch.frexp(v.abs().amax(2))          # amax = m 2^e, 0.5 <= m < 1
    e = torch.where(m == 0, -300, e)             # a block of zeros takes the smallest scale
    s = e - 7 if kind == "int8" else torch.where(m <= 0.875, e - 9, e - 8)
    s = s.clamp_min(-126)
    t = v * _pow2(-s)[..., None]
    if kind == "int8":
        q = t.round().clamp(-127, 127).to(torch.int8)
    else:
        q = t.to(torch.float8_e4m3fn)
    return q.view(rows, blocks * BLOCK)[:, :cols].contiguous(), (s + 127).to(torch.uint8)


def _unpack(q, scale):
    return q.float() * _pow2(scale.int() - 127).repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _expert_of(offsets, n, dev):
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(n, device=dev, dtype=offsets.dtype), right=True)


def _padded(v, offsets, cap):
    """Rows sorted by expert as (experts, cap, columns), zero past each expert's rows."""
    at = offsets[:-1, None] + torch.arange(cap, device=v.device)
    return torch.where((at < offsets[1:, None])[..., None], v[at.clamp_max(v.shape[0] - 1)], 0.0)


def _unpadded(p, offsets, n):
    e = _expert_of(offsets, n, p.device)
    inside = e < p.shape[0]
    e = e.clamp_max(p.shape[0] - 1)
    at = (torch.arange(n, device=p.device) - offsets[e]).clamp(0, p.shape[1] - 1)
    return torch.where(inside[:, None], p[e, at], 0.0)


def _rows_of(x, rows):
    return x if rows is None else x[rows.clamp_min(0)]


def _plain_product(v, w, offsets, cap):
    """v[r] W_e^T for the rows r of expert e."""
    n = v.shape[0]
    if n < w.shape[0]:     # few rows: each with its own expert's weights
        e = _expert_of(offsets, n, v.device)
        y = torch.bmm(w[e.clamp_max(w.shape[0] - 1)].float(), v[:, :, None])[:, :, 0]
        return torch.where((e < w.shape[0])[:, None], y, 0.0)
    return _unpadded(torch.bmm(_padded(v, offsets, cap), w.float().transpose(1, 2)), offsets, n)


def _plain_gated(g, u, dh):
    s = 1 / (1 + torch.exp(-g))
    return g * s * u, torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)


def _plain_route(s, c):
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp_max(F32_MAX)
    ids, slots, rows, offsets = _order(l, c["k"])
    top = torch.where(ids < 0, -math.inf, torch.gather(l, 1, ids.clamp_min(0).long()))
    base = top[:, :1].clamp_min(-F32_MAX)
    ex = torch.exp(top - base)
    p = torch.exp(l - base)
    total = (ex if c["normalize"] else p).sum(1, keepdim=True)
    w = torch.where(total > 0, ex / total, 0.0)
    out = [w, ids, slots, rows, offsets]
    if c["grad"]:
        dot = (w * s["dw"]).sum(1, keepdim=True)
        d = torch.zeros_like(l) if c["normalize"] else torch.where(total > 0, -p / total, 0.0) * dot
        add = w * (s["dw"] - dot) if c["normalize"] else w * s["dw"]
        d.scatter_add_(1, ids.clamp_min(0).long(), torch.where(ids < 0, 0.0, add))
        out.append(d.to(s["logits"].dtype))
    return out


def _plain_combine(s, c):
    y, slots, w, dout = s["y"].float(), s["slots"].long(), s["weights"], s["dout"].float()
    n = y.shape[0]
    live = slots >= 0
    yk = y[slots.clamp_min(0)]                                           # T, k, D
    out = torch.where(live[..., None], w[..., None] * yk, 0.0).sum(1)
    dw = torch.where(live, (yk * dout[:, None]).sum(2), 0.0)
    dy = torch.zeros(n + 1, y.shape[1], device=y.device)
    dy[torch.where(live, slots, n).reshape(-1)] = (w[..., None] * dout[:, None]).reshape(n, -1)
    return [out.to(s["y"].dtype), dy[:n].to(s["y"].dtype), dw]


def _plain(s):
    c = s["case"]
    op, dt = c["op"], DT[c["dtype"]]
    if op == "product":
        return _plain_product(_rows_of(s["x"], s["rows"]).float(), s["w"], s["offsets"], s["cap"]).to(dt)
    if op == "input_grad":
        return _plain_product(s["dy"].float(), s["w"].transpose(1, 2), s["offsets"], s["cap"]).to(dt)
    if op == "weight_grad":
        x = s["x"].float() if c["kind"] == "none" else _unpack(s["q"], s["scale"])
        dy = _padded(s["dy"].float(), s["offsets"], s["cap"])
        return torch.bmm(dy.transpose(1, 2), _padded(_rows_of(x, s["rows"]), s["offsets"], s["cap"])).to(dt)
    if op == "checkpoint":
        return _unpack(*_pack(s["x"], c["kind"])).to(dt)
    if op == "gated":
        f = c["cols"]
        gu, dh = s["gu"].float(), s["dh"].float()
        h, d = _plain_gated(gu[:, :f], gu[:, f:], dh)
        back = h
        if c["kind"] != "none":
            kept = _unpack(*_pack(s["gu"], c["kind"]))
            back, d = _plain_gated(kept[:, :f], kept[:, f:], dh)
        return [h.to(dt), d.to(dt), back.to(dt)]
    return _plain_route(s, c) if op == "route" else _plain_combine(s, c)


# ------------------------------------------------------------- the framework's

def _own(s):
    import matrix_orthogonalizing_optimizer_muon_amd as M
    c = s["case"]
    op = c["op"]
    if op == "product":
        return M.grouped_matmul(s["x"], s["w"], s["offsets"], rows=s["rows"])
    if op == "input_grad":
        return M.grouped_input_grad(s["dy"], s["w"], s["offsets"])
    if op == "weight_grad":
        x = s["x"] if c["kind"] == "none" else M.Checkpoint(s["q"], s["scale"], DT[c["dtype"]])
        return M.grouped_weight_grad(s["dy"], x, s["offsets"], rows=s["rows"])
    if op == "checkpoint":
        return M.restore(M.checkpoint(s["x"], c["kind"]))
    if op == "gated":
        if c["kind"] == "none":
            h, kept = M.gated(s["gu"]), s["gu"]
        else:
            h, kept = M.gated(s["gu"], checkpoint=c["kind"])
        d, back = M.gated_backward(s["dh"], kept)
        return [h, d, back]
    if op == "route":
        r = M.route(s["logits"], c["k"], normalize=c["normalize"])
        out = [r.weights, r.experts, r.slots, r.rows, r.offsets]
        if c["grad"]:
            out.append(M.route_backward(s["dw"], s["logits"], r, normalize=c["normalize"]))
        return out
    out = M.combine(s["y"], s["slots"], s["weights"])
    dy, dw = M.combine_backward(s["dout"], s["y"], s["slots"], s["weights"], s["offsets"])
    return [out, dy, dw]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------ work

def work(case):
    op, es = case["op"], ES[case["dtype"]]
    if op in ("product", "input_grad", "weight_grad"):
        n, i, o = case["tokens"] * case["k"], case["inner"], case["outer"]
        xr = case["tokens"] if case.get("gather") else n
        used = min(n, case["experts"] - case["idle"])
        flops = 2.0 * n * i * o
        if op == "product":
            return {"bytes": (xr * i + used * o * i + n * o) * es, "flops": flops}
        if op == "input_grad":
            return {"bytes": (n * o + used * o * i + n * i) * es, "flops": flops}
        x = xr * i * es if case["kind"] == "none" else xr * i * (1 + 1 / BLOCK)
        return {"bytes": n * o * es + x + case["experts"] * o * i * es, "flops": flops}
    if op == "checkpoint":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * (es + 1 + 1 / BLOCK), "flops": 4.0 * n}
    if op == "gated":
        n = case["rows"] * case["cols"]
        kept = 2 * 2 * n * (1 + 1 / BLOCK) if case["kind"] != "none" else 2 * n * es   # written and read, or read again
        return {"bytes": n * es * (2 + 1 + 1 + 2 + 1) + kept, "flops": 24.0 * n}
    t, k = case["tokens"], case["k"]
    if op == "route":
        b = t * case["experts"] * es + t * k * 16
        if case["grad"]:
            b += t * case["experts"] * es + t * k * 4
        return {"bytes": b, "flops": 4.0 * t * case["experts"]}
    d = case["cols"]
    return {"bytes": (t * k * d + t * d) * es + (2 * t * k * d + t * d) * es, "flops": 5.0 * t * k * d}


# ----------------------------------------------------------------------- exact

def _exact_two_to(n):
    """2^n in 64 bits (n whole, in the normal range)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_lead(v):
    """The whole number e with 2^e <= |v| < 2^(e + 1); far below every value's for 0."""
    m, e = torch.frexp(v.abs())
    return torch.where(m == 0, -1000, e.long() - 1)


def _exact_values(q, scale):
    return q.double() * torch.repeat_interleave(_exact_two_to(scale.long() - 127), BLOCK, 1)[:, :q.shape[1]]


def _exact_kept(x, kind):
    """The values a checkpoint of x stands for, from the definition in 64 bits."""
    rows, cols = x.shape
    v = x.double()
    v = torch.cat([v, v.new_zeros(rows, -cols % BLOCK)], 1).view(rows, -1, BLOCK)
    top = v.abs().max(2, keepdim=True).values
    lead = _exact_lead(top)
    if kind == "int8":
        unit = _exact_two_to((lead - 6).clamp_min(-126))
        q = torch.clamp(torch.round(v / unit), -127, 127)
    else:
        fits = top <= 1.75 * _exact_two_to(lead.clamp_min(-1000))
        unit = _exact_two_to(torch.where(fits, lead - 8, lead - 7).clamp_min(-126))
        t = v / unit
        grid = _exact_two_to(_exact_lead(t).clamp_min(-6) - 3)   # e4m3: 3 bits of fraction, normal from 2^-6
        q = torch.round(t / grid) * grid
    return (q * unit).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = _make(case, seed)
    op = case["op"]
    if op in ("product", "input_grad", "weight_grad"):
        o = s["offsets"].tolist()
        if op == "weight_grad":
            x = s["x"].double() if case["kind"] == "none" else _exact_values(s["q"], s["scale"])
            dy = s["dy"].double()
            res = torch.zeros(case["experts"], case["outer"], case["inner"], dtype=torch.float64, device="cuda")
            for e in range(case["experts"]):
                if o[e + 1] > o[e]:
                    xe = x[o[e]:o[e + 1]] if s["rows"] is None else x[s["rows"][o[e]:o[e + 1]].long()]
                    res[e] = dy[o[e]:o[e + 1]].t() @ xe
            return res
        v = s["x"].double() if op == "product" else s["dy"].double()
        if s["rows"] is not None:
            v = v[s["rows"].clamp_min(0).long()]
        res = torch.zeros(v.shape[0], case["outer"] if op == "product" else case["inner"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            if o[e + 1] > o[e]:
                we = s["w"][e].double()
                res[o[e]:o[e + 1]] = v[o[e]:o[e + 1]] @ (we.t() if op == "product" else we)
        return res
    if op == "checkpoint":
        return _exact_kept(s["x"], case["kind"])
    if op == "gated":
        f = case["cols"]

        def act(gu, dh):
            g, u = gu[:, :f], gu[:, f:]
            sg = torch.sigmoid(g)
            return g * sg * u, torch.cat([dh * u * (sg + g * sg * (1 - sg)), dh * g * sg], 1)
        full = s["gu"].double()
        kept = full if case["kind"] == "none" else _exact_kept(s["gu"], case["kind"])
        d_back = act(kept, s["dh"].double())
        return [act(full, s["dh"].double())[0], d_back[1], d_back[0]]
    if op == "route":
        l = s["logits"].double()
        ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        hot = torch.zeros_like(l).scatter_(1, ids, 1.0) * torch.isfinite(l)
        p = torch.softmax(torch.where(hot > 0, l, -math.inf) if case["normalize"] else l, 1)
        p = torch.nan_to_num(p) * torch.isfinite(l)
        w = torch.gather(p, 1, ids) * torch.gather(hot, 1, ids)
        out = [w, None, None, None, None]
        if case["grad"]:
            up = torch.zeros_like(l).scatter_(1, ids, s["dw"].double()) * hot
            out.append(p * (up - (p * up).sum(1, keepdim=True)))
        return out
    y, w, dout = s["y"].double(), s["weights"].double(), s["dout"].double()
    slots = s["slots"].long()
    out, dy, dw = torch.zeros_like(dout), torch.zeros_like(y), torch.zeros_like(w)
    for j in range(case["k"]):
        live = (slots[:, j] >= 0)[:, None]
        at = slots[:, j].clamp_min(0)
        out += torch.where(live, w[:, j:j + 1] * y[at], 0.0)
        dw[:, j] = torch.where(live, y[at] * dout, 0.0).sum(1)
        dy.index_add_(0, at, torch.where(live, w[:, j:j + 1] * dout, 0.0))
    return [out, dy, dw]
