"""Operators of a training step of a transformer of expert layers, as measured cases.

Causal attention over packed prompts, rotary positions, the router's balance
loss, and the gradient norm with clipping: each case is one pass through one of
them, in plain torch (``own = False``) or through the library's entry points
(``own = True``).
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the first token of a conversation: all latency
        dict(name="attn_token", op="attn", direction="fwd", lengths="1", tail=0, Hq=32, Hkv=8, D=128, fused=True),
        # prefill of one long prompt with grouped heads
        dict(name="attn_prompt", op="attn", direction="fwd", lengths="8192", tail=0, Hq=32, Hkv=8, D=128, fused=True),
        # a very long document on one key-value head of half the width, its own tensors
        dict(name="attn_long", op="attn", direction="fwd", lengths="32768", tail=0, Hq=8, Hkv=1, D=64, fused=False),
        # a training batch: documents packed into 8192 rows, an empty one and one of a single token among them,
        # some rows of padding behind the last
        dict(name="attn_train", op="attn", direction="train", lengths="3907,1,0,2050,1311,517,300,70", tail=36, Hq=32,
             Hkv=8, D=128, fused=True),
        # a small ragged step, three heads to a key-value head, of an odd width
        dict(name="attn_train_odd", op="attn", direction="train", lengths="517,129,300,57", tail=0, Hq=6, Hkv=2, D=80,
             fused=True),
        # one decoding step's queries and keys, rotated out of the projection's output
        dict(name="rotary_token", op="rotary", T=1, heads=40, extra=8, D=128, R=128, interleaved=False, base=10000.0,
             factor=1.0, original=4096, first=4095, inverse=False),
        # a training batch's queries and keys (the values beside them stay where they are)
        dict(name="rotary_batch", op="rotary", T=16384, heads=40, extra=8, D=128, R=128, interleaved=False,
             base=10000.0, factor=1.0, original=4096, first=0, inverse=False),
        # gradient of a rotation of part of the head, in pairs, far into a context stretched 32 times
        dict(name="rotary_long", op="rotary", T=4099, heads=16, extra=0, D=192, R=64, interleaved=True, base=500000.0,
             factor=32.0, original=4096, first=120000, inverse=True),
        # the router of a tiny layer
        dict(name="balance_small", op="balance", T=256, E=8, k=2, score="softmax", padding=0.0),
        # the router of a training batch over many experts, some of the rows padding
        dict(name="balance_batch", op="balance", T=16384, E=256, k=8, score="sigmoid", padding=0.05),
        # gradients of a small model on the way to its optimiser, below the limit
        dict(name="clip_small", op="clip", H=128, E=4, F=256, V=2003, layers=2, limit=1e6),
        # gradients of some hundred million weights, clipped
        dict(name="clip_model", op="clip", H=2048, E=16, F=1024, V=50001, layers=4, limit=1.0),
    ]


# ---------------------------------------------------------------- drawn cases
def _log_int(rng, lo, hi, multiple=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of `multiple`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / multiple)) * multiple
    return min(max(v, lo), hi)


_MOST = 14 * 128 * 32 * 8000 * 1200         # multiply-adds of the largest attention drawn


def draw(rng):
    op = rng.choice(["attn", "attn", "rotary", "balance", "clip"])
    if op == "attn":
        direction = rng.choice(["fwd", "train"])
        D = rng.choice([8, 32, 64, 80, 96, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        rows = _log_int(rng, 1, 8192)
        lengths = []
        for _ in range(rng.choice([1, 1, 2, 5, 17])):
            lengths.append(min(_log_int(rng, 1, 8192), rows - sum(lengths)))
            if rng.random() < 0.1:
                lengths.append(0)
        while sum(lengths) > 1 and _pairs(lengths) * Hq * D * (4 if direction == "fwd" else 14) > _MOST:
            lengths = [n // 2 for n in lengths]
        return dict(op="attn", direction=direction, lengths=",".join(str(n) for n in lengths),
                    tail=rng.choice([0, 0, 1, 77]), Hq=Hq, Hkv=Hkv, D=D, fused=rng.random() < 0.7)
    if op == "rotary":
        D = _log_int(rng, 16, 256, 8)
        R = rng.randint(1, D // 16) * 16
        heads = _log_int(rng, 1, 48)
        return dict(op="rotary", T=_log_int(rng, 1, 16384 * 40 * 128 // max(heads * D, 40 * 128)), heads=heads,
                    extra=rng.choice([0, 1, 8]), D=D, R=R, interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 8.0, 32.0]), original=4096,
                    first=rng.choice([0, 5, 4095, 120000, 1000003]), inverse=rng.random() < 0.5)
    if op == "balance":
        E = _log_int(rng, 4, 256)               # (k = E: every expert as often, and no gradient)
        return dict(op="balance", T=_log_int(rng, 16, 16384), E=E, k=rng.randint(1, min(E // 2, 8)),
                    score=rng.choice(["softmax", "sigmoid"]), padding=rng.choice([0.0, 0.05, 0.5]))
    return dict(op="clip", H=_log_int(rng, 8, 1024), E=_log_int(rng, 1, 8), F=_log_int(rng, 8, 1024),
                V=_log_int(rng, 10, 50001), layers=rng.randint(1, 6), limit=rng.choice([0.1, 1.0, 1e6]))


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    t = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)
    return t.to(torch.bfloat16)


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def _pairs(lengths):
    return sum(n * (n + 1) // 2 for n in lengths)


def _heads(make, case, T):
    """Tensors of the queries', keys' and values' shapes, as parts of one buffer or each its own."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["fused"]:
        t = make(T, Hq + 2 * Hkv, D)
        return t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:]
    return make(T, Hq, D), make(T, Hkv, D), make(T, Hkv, D)


def _zeros(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device=DEV)


def _frequencies(case):
    """Angle per position of each rotated pair (float64), and the factor on the rotated values.

    Stretched contexts: pairs that turn fewer than `slow` times within the
    original length are slowed by the factor, those that turn more than `fast`
    times are left, the ones between are blended.
    """
    R, base, factor = case["R"], case["base"], case["factor"]
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if factor == 1.0:
        return f.to(DEV), 1.0
    fast, slow = 32.0, 1.0

    def pair(turns):
        return R * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
    ramp = ((torch.arange(R // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return (f * (1.0 - ramp) + f / factor * ramp).to(DEV), 0.1 * math.log(factor) + 1.0


def _gradient_shapes(case):
    """Shapes and types of the gradients of a model of expert layers."""
    H, E, F, V = case["H"], case["E"], case["F"], case["V"]
    f32, bf16 = torch.float32, torch.bfloat16
    shapes = [((V, H), f32), ((V, H), bf16), ((H,), f32)]
    for _ in range(case["layers"]):
        shapes += [((H,), f32), ((H,), f32), ((E, H), f32), ((E, 2 * F, H), f32), ((E, H, F), f32), ((2 * H, H), bf16)]
    return shapes


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "attn":
        n = _lengths(case)
        T = sum(n) + case["tail"]
        s["ends"] = [sum(n[:i]) for i in range(len(n) + 1)]
        s["cu"] = torch.tensor(s["ends"], dtype=torch.int32, device=DEV)
        s["q"], s["k"], s["v"] = _heads(lambda *d: _normal(g, *d), case, T)
        s["out"] = _zeros(T, case["Hq"], case["D"])
        s["lse"] = torch.zeros(case["Hq"], T, device=DEV)
        if case["direction"] == "train":
            s["dout"] = _normal(g, T, case["Hq"], case["D"])
            s["dq"], s["dk"], s["dv"] = _heads(_zeros, case, T)
    elif case["op"] == "rotary":
        T, heads, D = case["T"], case["heads"], case["D"]
        s["x"] = _normal(g, T, heads + case["extra"], D)[:, :heads]
        s["out"] = _zeros(T, heads, D)
        start = case["first"] + int(torch.randint(0, 64, (1,), generator=g, device=DEV))
        s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device=DEV)
        s["freq"], s["scale"] = _frequencies(case)
    elif case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        lean = torch.empty(E, device=DEV).normal_(0.0, 1.0, generator=g)            # some experts are liked by all
        s["logits"] = torch.empty(T, E, device=DEV).normal_(0.0, 1.5, generator=g) + lean
        s["topk"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        s["tokens"] = torch.randint(0, 32000, (T,), generator=g, device=DEV, dtype=torch.int32)
        s["tokens"][torch.rand(T, device=DEV, generator=g) < case["padding"]] = -1
        s["dloss"] = torch.full((1,), 0.01, device=DEV) * (1.0 + torch.rand(1, device=DEV, generator=g))
        s["loss"], s["counts"] = torch.zeros(1, device=DEV), torch.zeros(E, dtype=torch.int32, device=DEV)
        s["slope"], s["dlogits"] = torch.zeros(E, device=DEV), torch.zeros(T, E, device=DEV)
    else:
        s["grads"], s["outs"] = [], []
        for i, (shape, dtype) in enumerate(_gradient_shapes(case)):
            t = torch.empty(shape, device=DEV).normal_(0.0, 10.0 ** -(2 + i % 4), generator=g).to(dtype)
            s["grads"].append(t)
            s["outs"].append(torch.empty_like(t))
        s["norm"] = torch.zeros(1, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attn(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G, T, scale = Hq // Hkv, s["q"].shape[0], s["D"] ** -0.5
    f32 = dict(dtype=torch.float32, device=DEV)
    out, lse = torch.zeros(T, Hq, D, **f32), torch.zeros(Hq, T, **f32)
    train = s["direction"] == "train"
    if train:
        dq, dk, dv = (torch.zeros(T, h, D, **f32) for h in (Hq, Hkv, Hkv))
    for a, b in zip(s["ends"], s["ends"][1:]):
        n = b - a
        if n == 0:
            continue
        later = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
        step = max(1, (1 << 28) // (n * n))                     # query heads at a time: scores of a gigabyte
        for kv in range(Hkv):
            k, v = s["k"][a:b, kv].float(), s["v"][a:b, kv].float()
            for h in range(kv * G, kv * G + G, step):
                heads = slice(h, min(h + step, kv * G + G))
                q = s["q"][a:b, heads].float().transpose(0, 1)
                p = (q @ k.T * scale).masked_fill_(later, float("-inf"))
                m = p.amax(2, keepdim=True)
                p = p.sub_(m).exp_()
                total = p.sum(2, keepdim=True)
                p.div_(total)
                o = p @ v
                out[a:b, heads] = o.transpose(0, 1)
                lse[heads, a:b] = (m + total.log())[:, :, 0]
                if train:
                    do = s["dout"][a:b, heads].float().transpose(0, 1)
                    dv[a:b, kv] += (p.transpose(1, 2) @ do).sum(0)
                    ds = (do @ v.T).sub_((do * o).sum(2, keepdim=True)).mul_(p).mul_(scale)
                    dq[a:b, heads] = (ds @ k).transpose(0, 1)
                    dk[a:b, kv] += (ds.transpose(1, 2) @ q).sum(0)
    res = {"out": out.to(torch.bfloat16), "lse": lse}
    if train:
        res.update(dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16), dv=dv.to(torch.bfloat16))
    return res


def _plain_rotary(s):
    R = s["R"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    c, d = (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()
    if s["inverse"]:
        d = -d
    x = s["x"].float()
    out = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        out[..., 0:R:2], out[..., 1:R:2] = a * c - b * d, b * c + a * d
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        out[..., :R // 2], out[..., R // 2:R] = a * c - b * d, b * c + a * d
    return out.to(torch.bfloat16)


def _plain_balance(s):
    E, k = s["E"], s["k"]
    valid = s["tokens"] >= 0
    N = valid.sum().clamp(min=1).double()
    x = s["logits"]
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, s["topk"].clamp(min=0).reshape(-1).long(),
                      valid[:, None].expand(-1, k).reshape(-1).to(torch.int32))
    if s["score"] == "softmax":
        e = (x - x.amax(1, keepdim=True)).exp()
        p = e / e.sum(1, keepdim=True)
    else:
        g = 1.0 / (1.0 + torch.exp(-x))
        p = g / g.sum(1, keepdim=True)
    p = p * valid[:, None]
    slope = (E * counts.double() / (k * N * N)).float()
    loss = (slope.double() * p.sum(0, dtype=torch.float64)).sum().float().reshape(1)
    d = p * (slope - (p * slope).sum(1, keepdim=True)) * s["dloss"]
    if s["score"] == "sigmoid":
        d = d * (1.0 - g)
    return {"loss": loss, "counts": counts, "slope": slope, "dlogits": d}


def _plain_clip(s):
    total = sum((t.float() * t.float()).sum(dtype=torch.float64) for t in s["grads"])
    norm = total.sqrt().float().reshape(1)
    c = (s["limit"] / (norm + 1e-6)).clamp(max=1.0)
    return [norm] + [(t.float() * c).to(t.dtype) for t in s["grads"]]


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
    if s["op"] == "attn":
        T = s["q"].shape[0]
        ws = _ws(api, api.moe_attention_workspace_bytes(T, s["Hq"], s["Hkv"], s["D"]))
        api.moe_attention_forward(s["q"], s["k"], s["v"], s["cu"], s["out"], s["lse"], ws)
        res = {"out": s["out"], "lse": s["lse"]}
        if s["direction"] == "train":
            api.moe_attention_backward(s["q"], s["k"], s["v"], s["cu"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"],
                                       s["dv"], ws)
            res.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
        return res
    if s["op"] == "rotary":
        api.moe_rotary(s["x"], s["positions"], s["freq"], s["out"], interleaved=s["interleaved"], scale=s["scale"],
                       inverse=s["inverse"])
        return s["out"]
    if s["op"] == "balance":
        ws = _ws(api, api.moe_balance_loss_workspace_bytes(s["T"], s["E"]))
        api.moe_balance_loss_forward(s["logits"], s["topk"], s["loss"], s["counts"], s["slope"], ws, tokens=s["tokens"],
                                     score=s["score"])
        api.moe_balance_loss_backward(s["logits"], s["slope"], s["dloss"], s["dlogits"], tokens=s["tokens"],
                                      score=s["score"])
        return {"loss": s["loss"], "counts": s["counts"], "slope": s["slope"], "dlogits": s["dlogits"]}
    ws = _ws(api, api.moe_grad_norm_workspace_bytes(len(s["grads"])))
    api.moe_grad_norm(s["grads"], s["norm"], ws)
    api.moe_grad_clip(s["grads"], s["norm"], s["limit"], outs=s["outs"])
    return [s["norm"]] + s["outs"]


_PLAIN = {"attn": _plain_attn, "rotary": _plain_rotary, "balance": _plain_balance, "clip": _plain_clip}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "attn":
        n, Hq, Hkv, D = _lengths(case), case["Hq"], case["Hkv"], case["D"]
        T, pairs = sum(n), _pairs(n)
        # q, k, v -> out, lse; with the gradients: dout -> dq, dk, dv
        bytes_ = T * D * 2 * (2 * Hq + 2 * Hkv) + 4 * T * Hq
        if case["direction"] == "fwd":
            return {"bytes": bytes_, "flops": 4 * D * Hq * pairs}
        return {"bytes": bytes_ + T * D * 2 * (2 * Hq + 2 * Hkv), "flops": 14 * D * Hq * pairs}
    if case["op"] == "rotary":
        n = case["T"] * case["heads"] * case["D"]
        return {"bytes": 4 * n + 4 * case["T"] + 4 * case["R"], "flops": 3 * case["T"] * case["heads"] * case["R"]}
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 8 * T * E + 4 * T * (k + 1) + 12 * E + 8, "flops": 12 * T * E}
    n = b = 0
    for shape, dtype in _gradient_shapes(case):
        size = math.prod(shape)
        n, b = n + size, b + size * (4 if dtype is torch.float32 else 2)
    return {"bytes": 2 * b + 4, "flops": 3 * n}


# ---------------------------------------------------------------- 64 bits
def _exact_attn(case, s):
    Hq, Hkv = case["Hq"], case["Hkv"]
    G, train = Hq // Hkv, case["direction"] == "train"
    d = torch.float64
    out, lse = torch.zeros_like(s["out"], dtype=d), torch.zeros_like(s["lse"], dtype=d)
    grads = [torch.zeros(s[n].shape, dtype=d, device=DEV) for n in ("q", "k", "v")]
    for a, b in zip(s["ends"], s["ends"][1:]):
        if a == b:
            continue
        seen = torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).tril()
        for h in range(Hq):                                      # gradients by differentiation of the forward
            q, k, v = (t[a:b, i].to(d).requires_grad_(train)
                       for t, i in ((s["q"], h), (s["k"], h // G), (s["v"], h // G)))
            z = torch.where(seen, torch.einsum("id,jd->ij", q, k) / math.sqrt(case["D"]), -math.inf)
            o = torch.softmax(z, 1) @ v
            out[a:b, h], lse[h, a:b] = o.detach(), torch.logsumexp(z.detach(), 1)
            if train:
                parts = torch.autograd.grad(o, (q, k, v), s["dout"][a:b, h].to(d))
                for t, i, part in zip(grads, (h, h // G, h // G), parts):
                    t[a:b, i] += part
    res = {"out": out, "lse": lse}
    if train:
        res.update(zip(("dq", "dk", "dv"), grads))
    return res


def exact(case, seed):
    """What run() returns, from the definitions, in float64."""
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "attn":
        return _exact_attn(case, s)
    if case["op"] == "rotary":
        R = case["R"]
        turn = torch.polar(torch.full_like(s["freq"], s["scale"]), s["freq"])       # rotation as complex products
        turn = torch.polar(turn.abs()[None].expand(case["T"], -1), torch.outer(s["positions"].to(d), s["freq"]))
        turn = (turn.conj() if case["inverse"] else turn)[:, None]
        x = s["x"].to(d)
        part = x[..., :R]
        pair = part.reshape(*part.shape[:2], R // 2, 2) if case["interleaved"] else \
            part.reshape(*part.shape[:2], 2, R // 2).transpose(2, 3)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        y = y if case["interleaved"] else y.transpose(2, 3)
        return torch.cat([y.reshape(part.shape), x[..., R:]], 2)
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        rows = torch.nonzero(s["tokens"] >= 0)[:, 0]
        N = len(rows)
        counts = torch.bincount(s["topk"][rows].reshape(-1).long(), minlength=E)
        z = s["logits"][rows].to(d).requires_grad_()
        share = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z) / torch.sigmoid(z).sum(1, True)
        slope = counts.to(d) * E / (k * max(N, 1) ** 2)
        loss = (share * slope).sum()
        dlogits = torch.zeros(case["T"], E, dtype=d, device=DEV)
        dlogits[rows] = torch.autograd.grad(loss, z, s["dloss"].to(d)[0])[0]
        return {"loss": loss.detach().reshape(1), "counts": counts.to(torch.int32), "slope": slope, "dlogits": dlogits}
    norm = torch.sqrt(torch.stack([torch.linalg.vector_norm(t.reshape(-1), dtype=d) ** 2 for t in s["grads"]]).sum())
    c = min(1.0, case["limit"] / (float(norm) + 1e-6))
    return [norm.reshape(1)] + [t.to(d) * c for t in s["grads"]]
