"""Plain fp64 NumPy forms of the operators around the expert layer: token
embedding, layer norm with the residual sum, vocabulary cross entropy, each
with its gradient.  Written from the formulas; used by the tests only."""
from __future__ import annotations

import numpy as np


def round_bf16(a: np.ndarray) -> np.ndarray:
    """fp32 values rounded to the nearest bfloat16 (ties to even), as fp64."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(a), r, a).astype(np.float64)


# ------------------------------------------------------------------ embedding
def embedding(tokens, table, scale=1.0):
    ok = (tokens >= 0) & (tokens < len(table))
    return np.where(ok[:, None], table[np.where(ok, tokens, 0)] * scale, 0.0)


def embedding_grad(tokens, dy, V, scale=1.0, base=None):
    """(dtable, the sum of magnitudes behind each value, tokens per row)."""
    ok = (tokens >= 0) & (tokens < V)
    out = np.zeros((V, dy.shape[1]))
    mag = np.zeros_like(out)
    np.add.at(out, tokens[ok], scale * dy[ok])
    np.add.at(mag, tokens[ok], abs(scale) * np.abs(dy[ok]))
    count = np.bincount(tokens[ok], minlength=V)
    if base is not None:
        out += base
        mag += np.abs(base)
    return out, mag, count


# ----------------------------------------------------------------- layer norm
def layer_norm(s, weight, bias=None, eps=1e-5):
    mean = s.mean(1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(1) + eps)
    xh = (s - mean[:, None]) * rstd[:, None]
    return {"y": xh * weight + (0.0 if bias is None else bias), "mean": mean, "rstd": rstd}


def layer_norm_grad(dy, s, weight, mean, rstd, dsum=None):
    xh = (s - mean[:, None]) * rstd[:, None]
    g = dy * weight
    m1, m2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - m1 - xh * m2)
    mag = rstd[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
        mag = mag + np.abs(dsum)
    return {"dx": dx, "dx_mag": mag, "dweight": (dy * xh).sum(0), "dweight_mag": np.abs(dy * xh).sum(0),
            "dbias": dy.sum(0), "dbias_mag": np.abs(dy).sum(0)}


# -------------------------------------------------------------- cross entropy
def cross_entropy(x, w, labels):
    z = x @ w.T
    m = z.max(1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(1))
    ok = (labels >= 0) & (labels < len(w))
    loss = np.where(ok, lse - z[np.arange(len(x)), np.where(ok, labels, 0)], 0.0)
    return {"z": z, "lse": lse, "loss": loss, "z_mag": (np.abs(x) @ np.abs(w).T).max(1)}


def cross_entropy_grad(x, w, labels, dloss, lse=None):
    """Rows without a label give nothing, whatever they hold."""
    V = len(w)
    ok = (labels >= 0) & (labels < V)
    xs = np.where(ok[:, None], x, 0.0)
    z = xs @ w.T
    if lse is None:
        lse = cross_entropy(xs, w, labels)["lse"]
    d = np.exp(z - np.where(ok, lse, 0.0)[:, None])
    d[np.arange(len(x)), np.where(ok, labels, 0)] -= 1.0
    d = np.where(ok[:, None], d * np.where(ok, dloss, 0.0)[:, None], 0.0)
    return {"d": d, "dx": d @ w, "dw": d.T @ xs,
            # root of the sum of squares and sum of magnitudes of the terms, for error bounds
            "dx_sq": np.sqrt((d * d) @ (w * w)), "dw_sq": np.sqrt((d * d).T @ (xs * xs)),
            "dx_mag": np.abs(d) @ np.abs(w), "dw_mag": np.abs(d).T @ np.abs(xs)}
