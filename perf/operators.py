"""The operators around the expert layer in a training step, as measured cases.

Token embedding, layer norm with the residual sum, and the softmax cross
entropy of a vocabulary head: each case is one pass through one of them, in
plain torch (``own = False``) or through the library's entry points
(``own = True``).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5


def listed():
    return [
        # one decoding step of a small batch: the lookup is all latency
        dict(name="embed_decode", op="embed", direction="fwd", n=8, V=32000, H=4096, scale=1.0),
        # a training batch's tokens looked up in a large vocabulary, scaled by sqrt(H)
        dict(name="embed_batch", op="embed", direction="fwd", n=16384, V=131072, H=4096, scale=64.0),
        # gradient of an untied table at a wide hidden size: a whole batch sorted by token
        dict(name="embed_grad", op="embed", direction="bwd", n=16384, V=32000, H=7168, scale=1.0, tied=False),
        # gradient of a table tied to the vocabulary head (added to the head's gradient), a ragged short batch
        dict(name="embed_grad_tied", op="embed", direction="bwd", n=1003, V=50001, H=1024, scale=32.0, tied=True),
        # the norm in front of the expert layer in one decoding step, residual added on the way
        dict(name="norm_decode", op="norm", direction="fwd", T=4, H=4096, residual=True),
        # the same over a training batch at the widest layer
        dict(name="norm_batch", op="norm", direction="fwd", T=16384, H=7168, residual=True),
        # its backward, the gradient of the residual stream joined in
        dict(name="norm_grad", op="norm", direction="bwd", T=16384, H=7168, residual=True),
        # a ragged batch at a narrow odd width, first norm of a model (no residual)
        dict(name="norm_grad_odd", op="norm", direction="bwd", T=1003, H=1000, residual=False),
        # scoring a single token: the head's weight is read once
        dict(name="loss_token", op="loss", direction="fwd", T=1, H=4096, V=32000, ignored=0.0),
        # evaluation of a batch: losses only
        dict(name="loss_eval", op="loss", direction="fwd", T=8192, H=4096, V=32000, ignored=0.0),
        # a ragged training step on an odd vocabulary, a third of the labels ignored
        dict(name="loss_train_odd", op="loss", direction="train", T=1003, H=1000, V=5003, ignored=0.33),
        # a training step over a large vocabulary: loss and both gradients
        dict(name="loss_train", op="loss", direction="train", T=4096, H=4096, V=131072, ignored=0.05),
    ]


def _log_int(rng, lo, hi, multiple=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of `multiple`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / multiple)) * multiple
    return min(max(v, lo), hi)


def draw(rng):
    H = _log_int(rng, 64, 7168, 8)
    if H == 3072:
        H += 8
    kind = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "loss_fwd", "loss_train"])
    if kind == "embed_fwd":
        return dict(op="embed", direction="fwd", n=_log_int(rng, 1, 16384), V=_log_int(rng, 1000, 131072), H=H,
                    scale=rng.choice([1.0, math.sqrt(H)]))
    if kind == "embed_bwd":
        return dict(op="embed", direction="bwd", n=_log_int(rng, 1, 16384),
                    V=_log_int(rng, 1000, min(131072, 32000 * 7168 // H)), H=H,
                    scale=rng.choice([1.0, math.sqrt(H)]), tied=rng.random() < 0.5)
    if kind.startswith("norm"):
        return dict(op="norm", direction=kind[5:], T=_log_int(rng, 1, 16384), H=H, residual=rng.random() < 0.5)
    T = _log_int(rng, 1, 8192)
    V = _log_int(rng, 1000, min(131072, 4096 * 4096 * 131072 // (T * H)))
    return dict(op="loss", direction=kind[5:], T=T, H=H, V=V, ignored=rng.choice([0.0, 0.05, 0.4]))


def _token_shares(V):
    """Share of each token id: a Zipf law, the low ids the frequent ones."""
    p = 1.0 / (np.arange(V) + 2.7)
    return p / p.sum()


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(mean, std, generator=g)
    return t.to(torch.bfloat16)


def _tokens(g, n, V, missing):
    """n token ids; a share `missing` of them is -1 (padding, or a label that is not scored)."""
    cdf = torch.from_numpy(np.cumsum(_token_shares(V))).to(DEV)
    u = torch.rand(n, device=DEV, dtype=torch.float64, generator=g)
    t = torch.searchsorted(cdf, u).clamp(max=V - 1).to(torch.int32)
    if missing > 0:
        t = torch.where(torch.rand(n, device=DEV, generator=g) < missing, torch.full_like(t, -1), t)
    return t


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV)


def _f32(*shape):
    return torch.empty(shape, dtype=torch.float32, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    H = case["H"]
    if case["op"] == "embed":
        n, V = case["n"], case["V"]
        s["tokens"] = _tokens(g, n, V, 0.03 if n > 16 else 0.0)
        if case["direction"] == "fwd":
            s["table"] = _normal(g, V, H, std=0.02)
            s["out"] = _bf16(n, H)
        else:
            s["dy"] = _normal(g, n, H)
            s["base"] = _normal(g, V, H, std=0.01) if case["tied"] else None
            s["dtable"] = _f32(V, H)
    elif case["op"] == "norm":
        T = case["T"]
        s["weight"] = _normal(g, H, std=0.1, mean=1.0)
        s["bias"] = _normal(g, H, std=0.1)
        spread = torch.empty(H, device=DEV).normal_(0.0, 0.5, generator=g).exp()    # channels of unlike size
        x = (torch.randn(T, H, device=DEV, generator=g) * spread + 0.3).to(torch.bfloat16)
        if case["direction"] == "fwd":
            s["x"] = x
            s["residual"] = _normal(g, T, H, std=2.0) if case["residual"] else None
            s["sum"] = _bf16(T, H) if case["residual"] else None
            s["y"], s["mean"], s["rstd"] = _bf16(T, H), _f32(T), _f32(T)
        else:
            s["s"] = x
            s["mean"] = x.float().mean(1)
            s["rstd"] = torch.rsqrt(x.float().var(1, unbiased=False) + EPS)
            s["dy"] = _normal(g, T, H)
            s["dsum"] = _normal(g, T, H) if case["residual"] else None
            s["dx"], s["dweight"], s["dbias"] = _bf16(T, H), _f32(H), _f32(H)
    else:
        T, V = case["T"], case["V"]
        s["x"] = _normal(g, T, H)
        s["w"] = _normal(g, V, H, std=0.02)
        s["labels"] = _tokens(g, T, V, case["ignored"])
        s["loss"], s["lse"] = _f32(T), _f32(T)
        if case["direction"] == "train":
            scored = (s["labels"] >= 0).sum().clamp(min=1).float()
            s["dloss"] = (torch.rand(T, device=DEV, generator=g) + 0.5) / scored    # weighted mean over the batch
            s["dx"], s["dw"] = _bf16(T, H), _bf16(V, H)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_embed_fwd(s):
    t = s["tokens"].long()
    rows = s["table"][t.clamp(min=0)].float() * s["scale"]
    return (rows * (t >= 0)[:, None]).to(torch.bfloat16)


def _plain_embed_bwd(s):
    t = s["tokens"].long()
    d = s["dy"].float() * s["scale"] * (t >= 0)[:, None]
    out = s["base"].float() if s["base"] is not None else torch.zeros_like(s["dtable"])
    return out.index_add_(0, t.clamp(min=0), d)


def _plain_norm_fwd(s):
    x = s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(torch.bfloat16)
    f = x.float()
    mean = f.mean(1, keepdim=True)
    c = f - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    y = (c * rstd * s["weight"].float() + s["bias"].float()).to(torch.bfloat16)
    out = {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["residual"] is not None:
        out["sum"] = x
    return out


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    xh = (s["s"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain_loss(s):
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"].long()
    scored = labels >= 0
    at = labels.clamp(min=0)[:, None]
    z = x @ w.T
    m = z.max(1, keepdim=True).values
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    loss = torch.where(scored, (lse - z.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    out = {"loss": loss, "lse": lse[:, 0]}
    if s["direction"] == "train":
        d = torch.exp_(z.sub_(lse))                     # the probabilities, in the logits' place
        d.scatter_add_(1, at, torch.full_like(lse, -1.0))
        d.mul_((s["dloss"] * scored)[:, None])
        out["dx"] = (d @ w).to(torch.bfloat16)
        out["dw"] = (d.T @ x).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the library's entry points
_workspace = None


def _ws(api, nbytes):
    """The program's one workspace, grown to the largest call so far."""
    global _workspace
    if _workspace is None or _workspace.numel() < nbytes:
        _workspace = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        api.moe_workspace_init(_workspace)
    return _workspace


def _own(s):
    from moe_expert_layer_05_gb300 import api
    H = s["H"]
    if s["op"] == "embed":
        ws = _ws(api, api.moe_embedding_workspace_bytes(s["n"], s["V"], H))
        if s["direction"] == "fwd":
            api.moe_embedding_forward(s["tokens"], s["table"], s["out"], ws, scale=s["scale"])
            return s["out"]
        api.moe_embedding_backward(s["tokens"], s["dy"], s["dtable"], ws, scale=s["scale"], base=s["base"])
        return s["dtable"]
    if s["op"] == "norm":
        if s["direction"] == "fwd":
            api.moe_layer_norm_forward(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"],
                                       residual=s["residual"], sum_out=s["sum"], eps=EPS)
            out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
            if s["residual"] is not None:
                out["sum"] = s["sum"]
            return out
        ws = _ws(api, api.moe_layer_norm_workspace_bytes(s["T"], H))
        api.moe_layer_norm_backward(s["dy"], s["s"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"],
                                    s["dbias"], ws, dsum=s["dsum"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    ws = _ws(api, api.moe_cross_entropy_workspace_bytes(s["T"], H, s["V"]))
    api.moe_cross_entropy_forward(s["x"], s["w"], s["labels"], s["loss"], s["lse"], ws)
    out = {"loss": s["loss"], "lse": s["lse"]}
    if s["direction"] == "train":
        api.moe_cross_entropy_backward(s["x"], s["w"], s["labels"], s["lse"], s["dloss"], s["dx"], s["dw"], ws)
        out["dx"], out["dw"] = s["dx"], s["dw"]
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"] == "embed":
        return _plain_embed_fwd(state) if state["direction"] == "fwd" else _plain_embed_bwd(state)
    if state["op"] == "norm":
        return _plain_norm_fwd(state) if state["direction"] == "fwd" else _plain_norm_bwd(state)
    return _plain_loss(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    H = case["H"]
    if case["op"] == "embed":
        n, V = case["n"], case["V"]
        if case["direction"] == "fwd":
            distinct = float((1.0 - np.power(1.0 - _token_shares(V), n)).sum())    # table rows read, on average
            return {"bytes": distinct * H * 2 + n * H * 2 + 4 * n, "flops": n * H}
        return {"bytes": n * H * 2 + 4 * n + V * H * (6 if case["tied"] else 4), "flops": 2 * n * H}
    if case["op"] == "norm":
        T, r = case["T"], 1 if case["residual"] else 0
        if case["direction"] == "fwd":      # x, residual -> sum, y, mean, rstd
            return {"bytes": T * H * 2 * (2 + 2 * r) + 8 * T + 4 * H, "flops": 8 * T * H}
        return {"bytes": T * H * 2 * (3 + r) + 8 * T + 2 * H + 8 * H, "flops": 14 * T * H}
    T, V = case["T"], case["V"]
    # losses: the logits' product; a training step: the logits again (they are not kept) and two products more
    if case["direction"] == "fwd":
        return {"bytes": (T + V) * H * 2 + 12 * T, "flops": 2 * T * H * V}
    return {"bytes": (T + V) * H * 4 + 16 * T, "flops": 8 * T * H * V}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns, from the definitions, in float64."""
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "embed":
        tok = s["tokens"].long()
        keep = tok >= 0
        if case["direction"] == "fwd":
            out = torch.zeros(case["n"], case["H"], dtype=d, device=DEV)
            out[keep] = s["table"].index_select(0, tok[keep]).to(d) * case["scale"]
            return out
        out = torch.zeros(case["V"], case["H"], dtype=d, device=DEV)
        out.index_put_((tok[keep],), s["dy"][keep].to(d), accumulate=True)
        out *= case["scale"]
        return out if s["base"] is None else out + s["base"].to(d)
    if case["op"] == "norm":
        w, b = s["weight"].to(d), s["bias"].to(d)
        if case["direction"] == "fwd":
            x = s["x"].to(d)
            if s["residual"] is not None:
                x = (x + s["residual"].to(d)).to(torch.float32).to(torch.bfloat16).to(d)   # the stream is held in bf16
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS).pow(-0.5)
            out = {"y": torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w), "mean": mean, "rstd": rstd}
            return out if s["residual"] is None else {**out, "sum": x}
        # through the Jacobian of the normalised row: dx = rstd (I - 11^T/H - xh xh^T/H) (w dy)
        rstd, H = s["rstd"].to(d)[:, None], case["H"]
        xh, dy = (s["s"].to(d) - s["mean"].to(d)[:, None]) * rstd, s["dy"].to(d)
        g = w * dy
        dx = rstd * (g - (g.sum(1, keepdim=True) + xh * torch.einsum("th,th->t", g, xh)[:, None]) / H)
        if s["dsum"] is not None:
            dx += s["dsum"].to(d)
        return {"dx": dx, "dweight": torch.einsum("th,th->h", dy, xh), "dbias": dy.sum(0)}
    x, w = s["x"].to(d), s["w"].to(d)
    z = torch.einsum("th,vh->tv", x, w)
    lse = torch.logsumexp(z, 1)
    rows = torch.nonzero(s["labels"] >= 0)[:, 0]
    cols = s["labels"][rows].long()
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, cols]
    out = {"loss": loss, "lse": lse}
    if case["direction"] == "train":
        scale = torch.zeros_like(lse)
        scale[rows] = s["dloss"].to(d)[rows]
        p = torch.softmax(z, 1)
        del z
        p[rows, cols] -= 1.0
        p *= scale[:, None]
        out["dx"], out["dw"] = p @ w, p.mT @ x
    return out
