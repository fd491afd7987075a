"""The token model with attention, rotary positions, balance losses and clipping: loss and every gradient against an
fp64 autograd form of the same formulas, packed and padded batches, and the training script."""
import math

import numpy as np
import pytest
import torch

from moe_expert_layer_05_gb300 import api, lm
from test_gpu_lm import _experts, _norm

pytestmark = pytest.mark.gpu


def _rotate(x, pos):
    n = x.shape[2] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    a = pos[:, None, None] * f
    c, s = torch.cos(a), torch.sin(a)
    return torch.cat([x[..., :n] * c - x[..., n:] * s, x[..., n:] * c + x[..., :n] * s], 2)


def _attention(x, p, i, m, cu):
    T, (Hq, Hkv, D) = len(x), (m.heads, m.kv_heads, m.head_dim)
    qkv = (x @ p[f"layer{i}.wqkv"].T).view(T, Hq + 2 * Hkv, D)
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    rows = []
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        t = qkv[a:b]
        qk = _rotate(t[:, :Hq + Hkv], torch.arange(b - a, dtype=torch.float64))
        k, v = (y.repeat_interleave(Hq // Hkv, 1) for y in (qk[:, Hq:], t[:, Hq + Hkv:]))
        z = torch.einsum("ihd,jhd->hij", qk[:, :Hq], k) / math.sqrt(D)
        z = z.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), -math.inf)
        rows.append(torch.einsum("hij,jhd->ihd", torch.softmax(z, 2), v))
    got = torch.cat(rows) if rows else out[:0]
    out = torch.cat([out[:cu[0]], got, out[cu[-1]:]])
    return out.reshape(T, -1) @ p[f"layer{i}.wo"].T


def _balance(x, p, i, idx, tokens):
    E, k = p[f"layer{i}.w_router"].shape[0], idx.shape[1]
    on = tokens >= 0
    share = torch.softmax(x[on] @ p[f"layer{i}.w_router"].T, 1)
    c = torch.bincount(idx[on].reshape(-1), minlength=E).double()
    return E / (k * int(on.sum()) ** 2) * (c * share.sum(0)).sum()


def _reference(m, tokens, labels, idx, cu):
    p = {n: t.detach().double().cpu().requires_grad_() for n, t in m.params.items()}
    s = p["table"][tokens.clamp(min=0)] * (tokens >= 0)[:, None] * m.embed_scale
    extra = 0.0
    for j, (kind, i) in enumerate(m.sublayers):
        n = _norm(s, p[f"norm{j}.weight"], p[f"norm{j}.bias"], m.eps)
        if kind == "attention":
            s = s + _attention(n, p, i, m, cu)
        else:
            s = s + _experts(n, p, i, idx[i])
            if m.balance:
                extra = extra + m.balance * _balance(n, p, i, idx[i], tokens)
    j = len(m.sublayers)
    n = _norm(s, p[f"norm{j}.weight"], p[f"norm{j}.bias"], m.eps)
    z = n @ (p["table"] if m.tied else p["head"]).T
    loss = torch.nn.functional.cross_entropy(z, labels, ignore_index=-1) + extra
    loss.backward()
    return float(loss.detach()), {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("heads,kv,D,layers,balance", [(4, 2, 32, 1, 0.0), (4, 1, 32, 2, 0.05), (3, 3, 48, 1, 0.2)])
@pytest.mark.parametrize("cu", [[0, 260], [0, 100, 100, 101, 200, 260], [0, 130, 237]])
def test_model_against_fp64_autograd(lib, heads, kv, D, layers, balance, cu):
    """bf16 activations pass about five roundings of relative 1.7e-3 (standard deviation) a sublayer each way, the
    attention's four more (p, ds, q and k turned): 4e-2 in rel-L2 leaves a gradient a factor of two; a wrong or missing
    path is off by its own size.  Tokens behind the last sequence are padding, without a label."""
    T, V = 260, 301
    m = lm.MoEModel(T, 128, 4, 2, 256, V, layers=layers, heads=heads, kv_heads=kv, head_dim=D, balance=balance, seed=layers)
    gen = torch.Generator().manual_seed(T)
    tokens, labels = (torch.randint(0, V, (T,), generator=gen) for _ in range(2))
    tokens[cu[-1]:] = -1
    labels[cu[-1]:] = -1
    labels[::7] = -1
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    m.step(tokens.int().cuda().roll(5).clamp(min=0), labels.int().cuda())       # another batch first: nothing of it stays
    loss = float(m.step(tokens.int().cuda(), labels.int().cuda(), cud))
    assert m.status() == 0
    idx = [b.fields()["topk_idx"].long().cpu() for b in m.blocks]
    want, grads = _reference(m, tokens, labels, idx, cu)
    assert abs(loss - want) <= 5e-3 * abs(want)
    for n, ref in grads.items():
        got = m.grads[n].double().cpu()
        rel = float(torch.linalg.norm(got - ref) / torch.linalg.norm(ref))
        assert rel <= 4e-2, f"{n}: rel-L2 {rel:.3e}"
    if balance:
        on = tokens >= 0
        for i in range(layers):
            np.testing.assert_array_equal(m.counts[i].cpu().numpy(), np.bincount(idx[i][on].reshape(-1), minlength=4))


def test_step_twice_gives_the_same_bits(lib):
    m = lm.MoEModel(300, 128, 8, 2, 128, 777, layers=2, heads=4, kv_heads=2, balance=0.01)
    gen = torch.Generator(device="cuda").manual_seed(5)
    tokens, labels = (torch.randint(0, 777, (300,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(2))
    cu = torch.tensor([0, 77, 300], dtype=torch.int32, device="cuda")
    a = float(m.step(tokens, labels, cu))
    first = {n: g.clone() for n, g in m.grads.items()}
    assert float(m.step(tokens, labels, cu)) == a
    assert all(torch.equal(first[n], g) for n, g in m.grads.items())


def test_a_step_of_one_sequence_is_captured(lib):
    """Without boundaries (one sequence of all tokens) a step copies nothing from the host: it can be captured, and the
    graph replayed on other tokens."""
    m = lm.MoEModel(300, 128, 8, 2, 128, 777, layers=1, heads=4, kv_heads=2, balance=0.01)
    gen = torch.Generator(device="cuda").manual_seed(8)
    tokens, labels = (torch.randint(0, 777, (300,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(2))
    others = [torch.randint(0, 777, (300,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(2)]
    m.step(tokens, labels, torch.tensor([0, 50, 300], dtype=torch.int32, device="cuda"))
    want = float(m.step(*others))
    grads = {n: g.clone() for n, g in m.grads.items()}
    m.step(tokens, labels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = m.step(tokens, labels)
    tokens.copy_(others[0])
    labels.copy_(others[1])
    graph.replay()
    assert float(loss) == want and m.status() == 0
    assert all(torch.equal(grads[n], g) for n, g in m.grads.items())


def test_clip_scales_every_gradient(lib):
    m = lm.MoEModel(130, 128, 4, 2, 128, 301, layers=1, heads=2, balance=0.01)
    gen = torch.Generator(device="cuda").manual_seed(6)
    tokens, labels = (torch.randint(0, 301, (130,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(2))
    m.step(tokens, labels)
    before = {n: g.double() for n, g in m.grads.items()}
    norm = math.sqrt(sum(float((g ** 2).sum()) for g in before.values()))
    assert abs(float(m.clip(norm / 3)) - norm) <= 1e-5 * norm
    for n, g in m.grads.items():
        half = 2.0 ** -8 if g.dtype is torch.bfloat16 else 2.0 ** -20
        assert bool(((g.double() - before[n] / 3).abs() <= 1.01 * half * before[n].abs() / 3 + 1e-40).all()), n
    assert abs(float(m.clip(norm)) - norm / 3) <= 1e-3 * norm                  # (bf16 gradients were rounded)


def test_training_script_runs_with_everything(lib):
    losses = lm.main(["--steps", "12", "--vocab", "203", "--tokens", "384", "--hidden", "128", "--heads", "2",
                      "--kv-heads", "1", "--length", "50", "--balance", "0.01", "--clip", "1.0"])
    assert len(losses) == 12 and all(math.isfinite(x) for x in losses)
