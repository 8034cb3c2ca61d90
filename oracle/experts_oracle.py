"""fp64 CPU oracle of the expert-layer operators, from their definitions (torch
tensors in, float64 tensors out; no code of the library)."""
import math

import torch


def clean(logits):
    l = logits.double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l)
    return l.clamp(max=float(torch.finfo(torch.float32).max))


def route(logits, k, normalize=True):
    """(weights, experts, slots, rows, offsets), the integers as Python lists."""
    l = clean(logits)
    tokens, n_exp = l.shape
    w = torch.zeros(tokens, k, dtype=torch.float64)
    ids = [[-1] * k for _ in range(tokens)]
    by_expert = [[] for _ in range(n_exp)]
    for t in range(tokens):
        row = l[t].tolist()
        order = sorted((e for e in range(n_exp) if row[e] != -math.inf), key=lambda e: (-row[e], e))[:k]
        if not order:
            continue
        base = row[order[0]]
        total = sum(math.exp(v - base) for v in ([row[e] for e in order] if normalize else row))
        for j, e in enumerate(order):
            ids[t][j] = e
            w[t, j] = math.exp(row[e] - base) / total
            by_expert[e].append((t, j))
    slots = [[-1] * k for _ in range(tokens)]
    rows, offsets = [], [0]
    for pairs in by_expert:
        for t, j in pairs:
            slots[t][j] = len(rows)
            rows.append(t)
        offsets.append(len(rows))
    rows += [-1] * (tokens * k - len(rows))
    return w, ids, slots, rows, offsets


def route_backward(dw, logits, k, normalize=True):
    w, ids, *_ = route(logits, k, normalize)
    l = clean(logits)
    d = torch.zeros_like(l)
    for t in range(l.shape[0]):
        live = [j for j in range(k) if ids[t][j] >= 0]
        if not live:
            continue
        dot = sum(float(w[t, j]) * float(dw[t, j]) for j in live)
        if normalize:
            p = torch.zeros(l.shape[1], dtype=torch.float64)
            for j in live:
                p[ids[t][j]] = w[t, j]
        else:
            p = torch.softmax(l[t], 0)
        d[t] = -p * dot
        for j in live:
            d[t, ids[t][j]] += float(w[t, j]) * float(dw[t, j])
    return d


def spans(offsets, n):
    """[(begin, end)] of the experts: offsets as their running maximum within [0, n]."""
    out, at = [], 0
    for v in offsets[1:]:
        end = min(max(v, at), n)
        out.append((at, end))
        at = end
    return out


def gathered(x, rows):
    """x[rows], a row of zeros where the index names none."""
    if rows is None:
        return x
    ok = (rows >= 0) & (rows < x.shape[0])
    if x.shape[0] == 0:
        return x.new_zeros(rows.shape[0], x.shape[1])
    return torch.where(ok[:, None], x[rows.long().clamp(0, x.shape[0] - 1)], torch.zeros((), dtype=x.dtype))


def matmul(x, w, offsets, rows=None):
    v = gathered(x.double(), rows)
    y = torch.zeros(v.shape[0], w.shape[1], dtype=torch.float64)
    for e, (b, end) in enumerate(spans(offsets, v.shape[0])):
        y[b:end] = v[b:end] @ w[e].double().t()
    return y


def input_grad(dy, w, offsets):
    dx = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64)
    for e, (b, end) in enumerate(spans(offsets, dy.shape[0])):
        dx[b:end] = dy[b:end].double() @ w[e].double()
    return dx


def weight_grad(dy, x, offsets, rows=None):
    v = gathered(x.double(), rows)
    dw = torch.zeros(len(offsets) - 1, dy.shape[1], x.shape[1], dtype=torch.float64)
    for e, (b, end) in enumerate(spans(offsets, dy.shape[0])):
        dw[e] = dy[b:end].double().t() @ v[b:end]
    return dw


def combine(y, slots, weights):
    out = torch.zeros(slots.shape[0], y.shape[1], dtype=torch.float64)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            s = int(slots[t, j])
            if 0 <= s < y.shape[0]:
                out[t] += weights[t, j].double() * y[s].double()
    return out


def combine_backward(dout, y, slots, weights):
    dy = torch.zeros(y.shape, dtype=torch.float64)
    dw = torch.zeros(slots.shape, dtype=torch.float64)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            s = int(slots[t, j])
            if 0 <= s < y.shape[0]:
                dy[s] = weights[t, j].double() * dout[t].double()
                dw[t, j] = float(y[s].double() @ dout[t].double())
    return dy, dw


# magnitudes e4m3 can hold: subnormals m 2^-9, normals (8 + m) 2^(e - 10) up to 448
_E4M3 = sorted({m * 2.0 ** -9 for m in range(8)} |
               {(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)} - {480.0})


def _nearest_e4m3(v):
    """Round to nearest, ties to the even mantissa (every second entry of the list)."""
    import bisect
    a = abs(v)
    i = min(bisect.bisect_left(_E4M3, a), len(_E4M3) - 1)
    if i and (a - _E4M3[i - 1] < _E4M3[i] - a or (a - _E4M3[i - 1] == _E4M3[i] - a and (i - 1) % 2 == 0)):
        i -= 1
    return math.copysign(_E4M3[i], v)


def checkpoint(x, kind):
    """(values in 8 bits as float64, scale codes, restored values) of blocks of 32 columns."""
    rows, cols = x.shape
    q = torch.zeros(rows, cols, dtype=torch.float64)
    scale = torch.zeros(rows, -(-cols // 32), dtype=torch.int64)
    back = torch.zeros(rows, cols, dtype=torch.float64)
    for r in range(rows):
        for b in range(scale.shape[1]):
            v = [float(t) for t in x[r, 32 * b:32 * b + 32]]
            if any(not math.isfinite(t) for t in v):
                scale[r, b] = 255
                back[r, 32 * b:32 * b + 32] = math.nan
                continue
            top = max(abs(t) for t in v)
            lead = math.frexp(top)[1] - 1 if top else -1000
            s = lead - 6 if kind == "int8" else (lead - 8 if top <= 1.75 * 2.0 ** max(lead, -1000) else lead - 7)
            s = max(s, -126)
            scale[r, b] = s + 127
            for i, t in enumerate(v):
                u = t / 2.0 ** s
                p = max(-127, min(127, round(u))) if kind == "int8" else _nearest_e4m3(u)
                q[r, 32 * b + i] = p
                back[r, 32 * b + i] = p * 2.0 ** s
    return q, scale, back


def gated(gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f].double(), gu[:, f:].double()
    return g * torch.sigmoid(g) * u


def gated_backward(dh, gu):
    f = gu.shape[1] // 2
    g, u, d = gu[:, :f].double(), gu[:, f:].double(), dh.double()
    s = torch.sigmoid(g)
    return torch.cat([d * u * (s + g * s * (1 - s)), d * g * s], 1)
