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


# ------------------------------------------------------------------ attention
def _sequences(cu, T):
    return [(int(a), int(b)) for a, b in zip(cu, cu[1:]) if b > a]


def attention(q, k, v, cu, scale):
    """Causal attention of each sequence: out, lse (0 in rows of no sequence), and sums of magnitudes for bounds."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag = np.zeros((T, Hq, v.shape[2])), np.zeros((T, Hq, v.shape[2]))
    lse, s_mag = np.zeros((Hq, T)), np.zeros((Hq, T))
    for a, b in _sequences(cu, T):
        seen = np.tril(np.ones((b - a, b - a), bool))
        for h in range(Hq):
            s = np.where(seen, scale * q[a:b, h] @ k[a:b, h // G].T, -np.inf)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(1, keepdims=True)
            p = e / l
            out[a:b, h], lse[h, a:b] = p @ v[a:b, h // G], (m + np.log(l))[:, 0]
            mag[a:b, h] = p @ np.abs(v[a:b, h // G])
            s_mag[h, a:b] = (np.where(seen, np.abs(q[a:b, h]) @ np.abs(k[a:b, h // G]).T, 0.0)).max(1) * scale
    return {"out": out, "lse": lse, "out_mag": mag, "s_mag": s_mag}


def attention_grad(q, k, v, cu, scale, dout):
    """dq, dk, dv, and for each the sums of magnitudes behind its error bounds.

    *_mag: the terms' magnitudes; *_delta: what an error of one part in <|dout|, |out|> moves; *_delta_sq: the
    variance from independent errors of variance 1 in each of the row's products dout out.
    """
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    f = attention(q, k, v, cu, scale)
    r = {n: np.zeros(t.shape) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dq_mag", q), ("dk_mag", k), ("dv_mag", v),
                                           ("dq_delta", q), ("dk_delta", k), ("dq_delta_sq", q), ("dk_delta_sq", k))}
    for a, b in _sequences(cu, T):
        seen = np.tril(np.ones((b - a, b - a), bool))
        for h in range(Hq):
            qs, ks, vs, do = q[a:b, h], k[a:b, h // G], v[a:b, h // G], dout[a:b, h]
            p = np.where(seen, np.exp(np.where(seen, scale * qs @ ks.T, -np.inf) - f["lse"][h, a:b, None]), 0.0)
            delta = (do * f["out"][a:b, h]).sum(1, keepdims=True)
            ds = p * (do @ vs.T - delta)
            mag = p * (np.abs(do) @ np.abs(vs).T + np.abs(delta))
            dl = p * (np.abs(do) * np.abs(f["out"][a:b, h])).sum(1, keepdims=True)
            for name, w in (("", ds), ("_mag", mag), ("_delta", dl)):
                aq, ak = (qs, ks) if name == "" else (np.abs(qs), np.abs(ks))
                r["dq" + name][a:b, h] += scale * w @ ak
                r["dk" + name][a:b, h // G] += scale * w.T @ aq
            var = ((do * f["out"][a:b, h]) ** 2).sum(1, keepdims=True)
            r["dq_delta_sq"][a:b, h] += scale ** 2 * var * (p @ ks) ** 2
            r["dk_delta_sq"][a:b, h // G] += scale ** 2 * (p ** 2 * var).T @ qs ** 2
            r["dv"][a:b, h // G] += p.T @ do
            r["dv_mag"][a:b, h // G] += p.T @ np.abs(do)
    return {**r, **f}


# --------------------------------------------------------------------- rotary
def rotary(x, positions, freq, interleaved=False, scale=1.0, inverse=False):
    """x [T, heads, width]; the first 2 len(freq) values of each head turned by positions * freq."""
    n = len(freq)
    angle = positions.astype(np.float64)[:, None, None] * freq * (-1.0 if inverse else 1.0)
    turn = scale * np.exp(1j * angle)
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    z = (a + 1j * b) * turn
    y = x.astype(np.float64).copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


# --------------------------------------------------------------- balance loss
def _shares(logits, sigmoid):
    """Probabilities of each row (0 in a row of -infinity) and 1 - sigmoid."""
    m = logits.max(1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        if sigmoid:
            log_s = -np.logaddexp(0.0, -logits)
            e = np.exp(log_s - log_s.max(1, keepdims=True))
        else:
            e = np.exp(logits - m)
        p = e / e.sum(1, keepdims=True)
        rest = np.exp(-np.logaddexp(0.0, logits))
    return np.where(np.isneginf(m), 0.0, p), rest


def balance_loss(logits, topk, k, tokens=None, sigmoid=False):
    T, E = logits.shape
    on = np.ones(T, bool) if tokens is None else tokens >= 0
    ids = topk[on].reshape(-1)
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    n = int(on.sum())
    slope = E * counts / (k * n * n) if n else np.zeros(E)
    p, rest = _shares(logits[on], sigmoid)
    grad = np.zeros((T, E))
    grad[on] = p * (slope - (p * slope).sum(1, keepdims=True)) * (rest if sigmoid else 1.0)
    mag = np.zeros((T, E))
    mag[on] = p * (slope + (p * slope).sum(1, keepdims=True))
    return {"loss": float((slope * p.sum(0)).sum()), "counts": counts, "slope": slope, "grad": grad, "grad_mag": mag}


# -------------------------------------------------------------- gradient norm
def clip(grads, limit):
    """(norm, every gradient times min(1, limit / (norm + 1e-6)))."""
    norm = np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads))
    c = min(1.0, limit / (norm + 1e-6))
    return norm, [g * c for g in grads]
