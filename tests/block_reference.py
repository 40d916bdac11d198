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
