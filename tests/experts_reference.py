"""The heads' norm with rotation, the routing, the grouped products and the combination of experts' results in
64 bits on the CPU, from their definitions, with the rounding bounds that the GPU tests hold the kernels to.
Shares no code with the library."""
import numpy as np

import block_reference as ref

U32, UNIT = ref.U32, ref.UNIT


def _mates(x, split):
    """The other element of each element's pair."""
    n, h, d = x.shape
    if split:
        return np.concatenate([x[..., d // 2:], x[..., :d // 2]], axis=-1)
    return x.reshape(n, h, d // 2, 2)[..., ::-1].reshape(n, h, d)


def head_weights(weight, heads, q_heads):
    """The weight [rows, D] as [heads, D], and the row each head takes."""
    owner = np.zeros(heads, dtype=int)
    if q_heads:
        owner[q_heads:] = 1
    elif weight.shape[0] == heads:
        owner = np.arange(heads)
    return weight[owner], owner


def head_norm(x, weight, q_heads, positions, freqs, sections, eps, split, unit):
    """y, 1/rms and the error bound of y.

    The sum of squares has d terms of one sign: d/2 roundings of 1/rms and a few more; the two products two; a
    turn 16 roundings of its pair (sine and cosine 8 each, products and sum)."""
    n, h, d = x.shape
    w, _ = head_weights(weight, h, q_heads)
    rstd = 1.0 / np.sqrt((x * x).mean(axis=2) + eps)
    z = x * rstd[..., None] * w
    y = ref.rotary(z, positions, freqs, sections, False, split)
    return y, rstd, unit * np.abs(y) + (d / 2 + 24) * U32 * (np.abs(z) + np.abs(_mates(z, split)))


def head_norm_backward(g, x, weight, q_heads, positions, freqs, sections, eps, split, unit, unit_w):
    """(dx, dweight) and their bounds."""
    n, h, d = x.shape
    w, owner = head_weights(weight, h, q_heads)
    rstd = 1.0 / np.sqrt((x * x).mean(axis=2) + eps)[..., None]
    hat = x * rstd
    u = ref.rotary(g, positions, freqs, sections, True, split)
    eu = 16 * U32 * (np.abs(g) + np.abs(_mates(g, split)))
    rel = (d / 2 + 24) * U32                                   # of hat and rstd, and the products they are in
    s = (u * w * hat).mean(axis=2, keepdims=True)
    es = (eu * np.abs(w * hat) + (d + rel / U32) * U32 * np.abs(u * w * hat)).mean(axis=2, keepdims=True)
    dx = rstd * (u * w - hat * s)
    bx = rstd * (eu * np.abs(w) + np.abs(hat) * es + rel * (np.abs(u * w) + np.abs(hat * s))) + unit * np.abs(dx)
    dw, bw = np.zeros_like(weight), np.zeros_like(weight)
    many = n * np.bincount(owner, minlength=weight.shape[0])
    for i in range(h):
        dw[owner[i]] += (u[:, i] * hat[:, i]).sum(axis=0)
        bw[owner[i]] += (eu[:, i] * np.abs(hat[:, i]) + (rel + (many[owner[i]] + 2) * U32) * np.abs(u[:, i] * hat[:, i])).sum(axis=0)
    return (dx, dw), (bx, bw + unit_w * np.abs(dw))


def route(logits, k, normalize):
    """experts, gates, offsets, rows, slots and the bound of the gates, row by row and pair by pair."""
    n, e = logits.shape
    experts = np.full((n, k), -1, dtype=np.int32)
    gates, bound = np.zeros((n, k)), np.zeros((n, k))
    for i in range(n):
        order = sorted(range(e), key=lambda j: (0 if np.isnan(logits[i, j]) else 1, -logits[i, j] if not np.isnan(logits[i, j]) else 0, j))
        chosen = [j for j in order if not logits[i, j] == -np.inf][:k]
        experts[i, :len(chosen)] = chosen
        if not chosen:
            continue
        v = logits[i, chosen]
        with np.errstate(invalid="ignore"):
            over = v if normalize else logits[i][logits[i] != -np.inf]
            t = np.exp(over - v[0])
            gates[i, :len(chosen)] = np.exp(v - v[0]) / t.sum()
            # an exponential: 3 roundings and its argument's; a sum of positive terms: one a term; the quotient one
            far = np.abs(over - v[0]).max() if len(over) else 0.0
            bound[i, :len(chosen)] = gates[i, :len(chosen)] * (len(over) + 2 * far + 12) * U32
    flat = experts.reshape(-1)
    keys = np.where(flat < 0, e, flat)
    order = np.array(sorted(range(n * k), key=lambda p: (keys[p], p)), dtype=np.int64)
    slots = np.empty(n * k, dtype=np.int32)
    slots[order] = np.arange(n * k)
    offsets = np.array([(keys < j).sum() for j in range(e + 1)], dtype=np.int32)
    return experts, gates, offsets, (order // k).astype(np.int32), slots.reshape(n, k), bound


def route_backward(grad, logits, experts, gates, normalize, unit):
    """dlogits and its bound, for the gates as they are stored."""
    n, e = logits.shape
    out, bound = np.zeros((n, e)), np.zeros((n, e))
    for i in range(n):
        d = grad[i] * gates[i]
        if normalize:
            p, rel = np.zeros(e), 2.0
            for j, x in enumerate(experts[i]):
                if 0 <= x < e:
                    p[x] += gates[i, j]
        else:
            open_ = logits[i] > -np.inf
            if not open_.any():
                p, rel = np.zeros(e), 0.0
            else:
                top = logits[i].max()
                p = np.where(open_, np.exp(logits[i] - top), 0.0)
                p, rel = p / p.sum(), e + 12 + 2 * np.abs(logits[i][open_] - top).max()
        out[i] = -p * d.sum()
        bound[i] = p * (len(d) + 6 + rel) * U32 * np.abs(d).sum()
        for j, x in enumerate(experts[i]):
            if 0 <= x < e:
                out[i, x] += d[j]
                bound[i, x] += 6 * U32 * (np.abs(d[j]) + np.abs(d).sum() * p[x])
    return out, bound + unit * np.abs(out)


def bounds_of(offsets, n):
    """Offsets as the library counts them: the largest so far, clamped to [0, n]."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, n))


def grouped_linear(x, weight, bias, offsets, rows, many, unit):
    """out and its bound.  A sum of cin products: cin roundings of the sum of their sizes."""
    groups, cout, cin = weight.shape
    ends = bounds_of(offsets, many)
    xr = _taken(x, rows, many)
    out, bound = np.zeros((many, cout)), np.zeros((many, cout))
    for g in range(groups):
        p = slice(ends[g], ends[g + 1])
        b = np.zeros(cout) if bias is None else bias[g]
        out[p] = xr[p] @ weight[g].T + b
        bound[p] = (cin + 8) * U32 * (np.abs(xr[p]) @ np.abs(weight[g]).T + np.abs(b))
    return out, bound + unit * np.abs(out)


def _taken(x, rows, many):
    if rows is None:
        return x
    rows = np.asarray(rows, dtype=np.int64)
    there = (rows >= 0) & (rows < x.shape[0])
    out = np.zeros((many, x.shape[1]))
    out[there] = x[rows[there]]
    return out


def grouped_linear_backward(g, x, weight, offsets, rows, unit):
    """(dx, dweight, dbias) and their bounds."""
    groups, cout, cin = weight.shape
    many = g.shape[0]
    ends = bounds_of(offsets, many)
    xr = _taken(x, rows, many)
    dx, dw, db = np.zeros((many, cin)), np.zeros_like(weight), np.zeros((groups, cout))
    bx, bw, bb = np.zeros_like(dx), np.zeros_like(dw), np.zeros_like(db)
    for i in range(groups):
        p = slice(ends[i], ends[i + 1])
        n = ends[i + 1] - ends[i]
        dx[p], bx[p] = g[p] @ weight[i], (cout + 8) * U32 * (np.abs(g[p]) @ np.abs(weight[i]))
        dw[i], bw[i] = g[p].T @ xr[p], (n + 8) * U32 * (np.abs(g[p]).T @ np.abs(xr[p]))
        db[i], bb[i] = g[p].sum(axis=0), (n + 8) * U32 * np.abs(g[p]).sum(axis=0)
    return (dx, dw, db), (bx + unit * np.abs(dx), bw + unit * np.abs(dw), bb + U32 * np.abs(db))


def combine(y, slots, gates, unit):
    n, k = slots.shape
    out, size = np.zeros((n, y.shape[1])), np.zeros((n, y.shape[1]))
    for j in range(k):
        at = slots[:, j].astype(np.int64)
        there = (at >= 0) & (at < y.shape[0])
        f = np.ones(n) if gates is None else gates[:, j]
        out[there] += f[there, None] * y[at[there]]
        size[there] += np.abs(f[there, None] * y[at[there]])
    return out, unit * np.abs(out) + (k + 2) * U32 * size


def combine_backward(g, y, slots, rows, gates, unit):
    """(dy, dgates) and their bounds."""
    n, k = slots.shape
    many, c = y.shape
    dy, dgates, bg = np.zeros((many, c)), np.zeros((n, k)), np.zeros((n, k))
    size = np.zeros((many, c))
    for i in range(n):
        for j in range(k):
            p = slots[i, j]
            if not 0 <= p < many:
                continue
            f = 1.0 if gates is None else gates[i, j]
            dgates[i, j], bg[i, j] = g[i] @ y[p], (c + 8) * U32 * (np.abs(g[i]) @ np.abs(y[p]))
            if rows[p] == i:
                dy[p] += f * g[i]
                size[p] += np.abs(f * g[i])
    return (dy, dgates), (unit * np.abs(dy) + 2 * k * U32 * size, bg)
