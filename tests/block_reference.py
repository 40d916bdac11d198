"""The transformer-block operators in 64 bits on the CPU, from their definitions, and the
rounding bounds that the GPU tests hold the kernels to.  Shares no code with the library."""
import numpy as np

U32 = 2.0 ** -24                       # unit roundoff of fp32
UNIT = {"f32": U32, "bf16": 2.0 ** -8}  # of the output type


def layer_norm(x, w, b, eps):
    mean = x.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    return (x - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]


def layer_norm_backward(g, x, w, eps):
    _, mean, rstd = layer_norm(x, 1.0, 0.0, eps)
    h = (x - mean[:, None]) * rstd[:, None]
    gw = g * w
    dx = rstd[:, None] * (gw - gw.mean(axis=1, keepdims=True) - h * (gw * h).mean(axis=1, keepdims=True))
    return dx, (g * h).sum(axis=0), g.sum(axis=0)


def rotary(x, positions, freqs, sections, inverse, split):
    n, h, d = x.shape
    out = x.copy()
    p = 0
    for axis, count in enumerate(sections):
        for _ in range(count):
            t = positions[:, axis].astype(np.float64) * np.float64(freqs[p]) * (-1.0 if inverse else 1.0)
            i, j = (p, p + d // 2) if split else (2 * p, 2 * p + 1)
            c, s = np.cos(t)[:, None], np.sin(t)[:, None]
            out[:, :, i] = x[:, :, i] * c - x[:, :, j] * s
            out[:, :, j] = x[:, :, i] * s + x[:, :, j] * c
            p += 1
    return out


def attention(q, k, v, q_off, k_off, scale, unit):
    """out, lse and the error bound of out, for heads [N,H,D] in 64 bits.

    `unit` is the roundoff of the tensors' type; where it is not fp32's, weights are rounded
    to it before the product with v."""
    nq, h, d = q.shape
    hk = k.shape[1]
    out, lse, bound = np.zeros_like(q), np.full((nq, h), -np.inf), np.zeros_like(q)
    lse_err = np.zeros((nq, h))
    for e in range(len(q_off) - 1):
        a, b = slice(q_off[e], q_off[e + 1]), slice(k_off[e], k_off[e + 1])
        n = k_off[e + 1] - k_off[e]
        if n == 0 or q_off[e + 1] == q_off[e]:
            continue
        for i in range(h):
            kk, vv, qq = k[b, i // (h // hk)], v[b, i // (h // hk)], q[a, i]
            s = scale * qq @ kk.T
            top = s.max(axis=1, keepdims=True)
            with np.errstate(invalid="ignore"):
                w = np.where(top == -np.inf, 0.0, np.exp(s - np.where(top == -np.inf, 0.0, top)))
            total = w.sum(axis=1, keepdims=True)
            p = w / np.where(total == 0, 1.0, total)
            out[a, i] = p @ vv
            with np.errstate(divide="ignore"):
                lse[a, i] = (top + np.log(total))[:, 0]
            # a score: d products and sums; its exponent and the reference: a few roundings of its size
            with np.errstate(invalid="ignore"):
                es = ((d + 16) * U32 * scale * (np.abs(qq) @ np.abs(kk).T)).max(axis=1, keepdims=True)
            lse_err[a, i] = (es + (n + 64) * U32)[:, 0] + 4 * U32 * np.abs(np.where(np.isfinite(lse[a, i]), lse[a, i], 0))
            rel = 2 * es + (2 * n + 64) * U32 + (unit if unit != U32 else 0.0)
            bound[a, i] = (p @ np.abs(vv)) * rel
    return out, lse, bound + unit * np.abs(out), lse_err


def attention_backward(g, q, k, v, q_off, k_off, scale, unit):
    """(dq, dk, dv) and their error bounds, given out and lse within attention()'s bounds."""
    out, lse, out_err, lse_err = attention(q, k, v, q_off, k_off, scale, unit)
    h, d = q.shape[1:]
    group = h // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    low = unit if unit != U32 else 0.0
    for e in range(len(q_off) - 1):
        a, b = slice(q_off[e], q_off[e + 1]), slice(k_off[e], k_off[e + 1])
        n, m = k_off[e + 1] - k_off[e], (q_off[e + 1] - q_off[e]) * group
        if n == 0 or m == 0:
            continue
        for i in range(h):
            j = i // group
            kk, vv, qq, gg = k[b, j], v[b, j], q[a, i], g[a, i]
            p = np.exp(scale * qq @ kk.T - lse[a, i][:, None])
            es = (d + 16) * U32 * scale * (np.abs(qq) @ np.abs(kk).T)
            rel = es + lse_err[a, i][:, None] + 8 * U32 * (1 + np.abs(lse[a, i])[:, None])   # of a weight
            dp, delta = gg @ vv.T, (gg * out[a, i]).sum(axis=1, keepdims=True)
            ds = p * (dp - delta)
            dp_err = (d + 2) * U32 * (np.abs(gg) @ np.abs(vv).T)
            delta_err = (np.abs(gg) * (out_err[a, i] + (d + 2) * U32 * np.abs(out[a, i]))).sum(axis=1, keepdims=True)
            ds_err = p * (dp_err + delta_err) * (1 + rel) + np.abs(ds) * (2 * rel + low + 4 * U32)
            dq[a, i] = scale * ds @ kk
            bq[a, i] = scale * (ds_err + np.abs(ds) * (n + 4) * U32) @ np.abs(kk)
            dk[b, j] += scale * ds.T @ qq
            bk[b, j] += scale * (ds_err + np.abs(ds) * (m + 4) * U32).T @ np.abs(qq)
            dv[b, j] += p.T @ gg
            bv[b, j] += (p * (2 * rel + low + (m + 4) * U32)).T @ np.abs(gg)
    return (dq, dk, dv), (bq + unit * np.abs(dq), bk + unit * np.abs(dk), bv + unit * np.abs(dv))
