"""The token model that joins the embedding, the norms, the expert layers and the
vocabulary loss: loss and every gradient against an fp64 autograd form of the
same formulas, and a short training run."""
import math

import numpy as np
import pytest
import torch

from moe_expert_layer_05_gb300 import lm

pytestmark = pytest.mark.gpu


def _norm(s, w, b, eps):
    mean = s.mean(1, keepdim=True)
    var = ((s - mean) ** 2).mean(1, keepdim=True)
    return (s - mean) / torch.sqrt(var + eps) * w + b


def _experts(x, p, i, idx):
    """The expert layer with the routing decision (idx [T, k]) given; its gates are differentiated."""
    logits = x @ p[f"layer{i}.w_router"].T
    gate = torch.softmax(logits.gather(1, idx), 1)
    y = torch.zeros_like(x)
    F = p[f"layer{i}.w2"].shape[2]
    for e in range(logits.shape[1]):
        t, slot = torch.nonzero(idx == e, as_tuple=True)
        z = x[t] @ p[f"layer{i}.w1"][e].T
        h = gate[t, slot][:, None] * torch.nn.functional.silu(z[:, :F]) * z[:, F:]
        y = y.index_add(0, t, h @ p[f"layer{i}.w2"][e].T)
    return y


def _reference(m, tokens, labels, idx):
    p = {n: t.detach().double().cpu().requires_grad_() for n, t in m.params.items()}
    s = p["table"][tokens.clamp(min=0)] * (tokens >= 0)[:, None] * m.embed_scale
    for i in range(m.layers):
        s = s + _experts(_norm(s, p[f"norm{i}.weight"], p[f"norm{i}.bias"], m.eps), p, i, idx[i])
    n = _norm(s, p[f"norm{m.layers}.weight"], p[f"norm{m.layers}.bias"], m.eps)
    z = n @ (p["table"] if m.tied else p["head"]).T
    loss = torch.nn.functional.cross_entropy(z, labels, ignore_index=-1)
    loss.backward()
    return float(loss.detach()), {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("layers,T,V", [(1, 130, 301), (2, 515, 1003)])
def test_model_against_fp64_autograd(lib, tied, layers, T, V):
    """bf16 activations pass about five roundings of relative 1.7e-3 (standard deviation) a layer each way, so
    3e-2 in rel-L2 leaves a gradient a factor of two or more; a wrong or missing path is off by its own size."""
    m = lm.MoEModel(T, 128, 4, 2, 256, V, layers=layers, tied=tied, seed=layers)
    gen = torch.Generator().manual_seed(T)
    tokens, labels = (torch.randint(0, V, (T,), generator=gen) for _ in range(2))
    tokens[3] = -1
    labels[::7] = -1
    loss = float(m.step(tokens.int().cuda(), labels.int().cuda()))
    assert m.status() == 0
    idx = [b.fields()["topk_idx"].long().cpu() for b in m.blocks]
    want, grads = _reference(m, tokens, labels, idx)
    assert abs(loss - want) <= 5e-3 * want
    for n, ref in grads.items():
        got = m.grads[n].double().cpu()
        rel = float(torch.linalg.norm(got - ref) / torch.linalg.norm(ref))
        assert rel <= 3e-2, f"{n}: rel-L2 {rel:.3e}"


def test_step_twice_gives_the_same_bits(lib):
    m = lm.MoEModel(300, 128, 8, 2, 128, 777, layers=2)
    gen = torch.Generator(device="cuda").manual_seed(5)
    tokens, labels = (torch.randint(0, 777, (300,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(2))
    a = float(m.step(tokens, labels))
    first = {n: g.clone() for n, g in m.grads.items()}
    assert float(m.step(tokens, labels)) == a
    assert all(torch.equal(first[n], g) for n, g in m.grads.items())


def test_training_learns_the_rule(lib):
    losses = lm.main(["--steps", "40", "--vocab", "503", "--tokens", "512", "--hidden", "128"])
    # (the head is tied: at the start the stream's own token has the largest logit, so the loss begins above log V)
    assert losses[0] > math.log(503)
    assert np.mean(losses[-5:]) < 0.5 * losses[0]
