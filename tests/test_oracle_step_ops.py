"""The fp64 forms of attention, rotary positions, the balance loss and clipping: gradients against central
differences and torch's autograd, and pinned properties (CPU only)."""
import math

import numpy as np
import pytest
import torch

from oracle import model_oracle as M


def _difference(f, a, direction, h=1e-5):
    return (f(a + h * direction) - f(a - h * direction)) / (2 * h)


@pytest.mark.parametrize("cu,Hq,Hkv", [([0, 7], 2, 1), ([1, 4, 4, 9], 3, 3), ([0, 1, 2, 8], 4, 2)])
def test_attention_gradients(cu, Hq, Hkv):
    r = np.random.default_rng(sum(cu))
    T, D, scale = 10, 6, 0.7
    q, k, v, c = (r.standard_normal((T, h, D)) for h in (Hq, Hkv, Hkv, Hq))
    g = M.attention_grad(q, k, v, cu, scale, c)
    for name, arg, fun in (("dq", q, lambda a: (M.attention(a, k, v, cu, scale)["out"] * c).sum()),
                           ("dk", k, lambda a: (M.attention(q, a, v, cu, scale)["out"] * c).sum()),
                           ("dv", v, lambda a: (M.attention(q, k, a, cu, scale)["out"] * c).sum())):
        d = r.standard_normal(arg.shape)
        assert abs(_difference(fun, arg, d) - (g[name] * d).sum()) < 1e-7, name
    rows = np.zeros(T, bool)
    rows[cu[0]:cu[-1]] = True
    assert not g["dq"][~rows].any() and not g["dv"][~rows].any() and not g["out"][~rows].any()


def test_attention_is_torch_s():
    r = np.random.default_rng(1)
    q, k, v = (r.standard_normal((9, h, 8)) for h in (4, 2, 2))
    f = M.attention(q, k, v, [0, 9], 8 ** -0.5)
    t = [torch.from_numpy(a.transpose(1, 0, 2).copy()) for a in (q, k, v)]
    z = t[0] @ t[1].repeat_interleave(2, 0).transpose(1, 2) / math.sqrt(8)
    z = z.masked_fill(torch.ones(9, 9, dtype=torch.bool).triu(1), -math.inf)
    want = torch.softmax(z, 2) @ t[2].repeat_interleave(2, 0)
    np.testing.assert_allclose(f["out"], want.numpy().transpose(1, 0, 2), atol=1e-12)
    np.testing.assert_allclose(f["lse"], torch.logsumexp(z, 2).numpy(), atol=1e-12)
    np.testing.assert_allclose(f["out"][0], np.repeat(v[0], 2, 0), atol=1e-12)        # a row that sees itself alone


def test_rotary_turns_and_turns_back():
    r = np.random.default_rng(2)
    x, pos, freq = r.standard_normal((5, 3, 20)), np.array([0, 1, 7, 100, -3]), np.array([1.0, 0.3, 0.01, 0.0])
    for interleaved in (False, True):
        y = M.rotary(x, pos, freq, interleaved)
        np.testing.assert_allclose(M.rotary(y, pos, freq, interleaved, inverse=True), x, atol=1e-12)
        np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
        np.testing.assert_allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2), atol=1e-12)
        np.testing.assert_allclose(y[0], x[0], atol=1e-12)                            # position 0
    # a quarter turn takes (a, b) to (-b, a)
    y = M.rotary(np.array([[[1.0, 2.0]]]), np.array([1]), np.array([math.pi / 2]))
    np.testing.assert_allclose(y[0, 0], [-2.0, 1.0], atol=1e-12)
    # scores of turned queries and keys depend on the distance alone
    q, k = r.standard_normal((2, 1, 1, 8))
    dots = [float((M.rotary(q, np.array([p + 5]), freq) * M.rotary(k, np.array([p]), freq)).sum()) for p in (0, 3, 90)]
    np.testing.assert_allclose(dots, dots[0], atol=1e-10)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_gradient(sigmoid):
    r = np.random.default_rng(3)
    x, tokens = r.standard_normal((12, 6)), np.array([0, 1, -1, 3, 4, 5, 6, -1, 8, 9, 10, 11])
    topk = np.argsort(-x, 1)[:, :2]
    g = M.balance_loss(x, topk, 2, tokens, sigmoid)
    d = r.standard_normal(x.shape)
    num = _difference(lambda a: M.balance_loss(a, topk, 2, tokens, sigmoid)["loss"], x, d)
    assert abs(num - (g["grad"] * d).sum()) < 1e-8
    assert not g["grad"][[2, 7]].any() and g["counts"].sum() == 20
    np.testing.assert_allclose(g["grad"].sum(1) if not sigmoid else 0.0, 0.0, atol=1e-14)
    # by torch, the choices held fixed
    t = torch.from_numpy(x[tokens >= 0]).requires_grad_()
    p = torch.sigmoid(t) / torch.sigmoid(t).sum(1, keepdim=True) if sigmoid else torch.softmax(t, 1)
    c = torch.bincount(torch.from_numpy(topk[tokens >= 0].reshape(-1)), minlength=6).double()
    loss = 6 / (2 * 10 * 10) * (c * p.sum(0)).sum()
    loss.backward()
    assert abs(float(loss.detach()) - g["loss"]) < 1e-12
    np.testing.assert_allclose(t.grad.numpy(), g["grad"][tokens >= 0], atol=1e-14)


def test_balance_of_even_and_of_one_sided_routers():
    topk = np.array([[t % 4] for t in range(8)])
    assert abs(M.balance_loss(np.zeros((8, 4)), topk, 1)["loss"] - 1.0) < 1e-14
    sure = np.where(np.arange(4) == 2, 50.0, 0.0)[None].repeat(8, 0)
    assert abs(M.balance_loss(sure, np.full((8, 1), 2), 1)["loss"] - 4.0) < 1e-12
    dead = np.zeros((8, 4))
    dead[:, 3] = -np.inf
    dead[5] = -np.inf
    g = M.balance_loss(dead, np.zeros((8, 1), int), 1)
    assert np.isfinite(g["grad"]).all() and not g["grad"][:, 3].any() and not g["grad"][5].any()


def test_clip_is_torch_s():
    r = np.random.default_rng(4)
    g = [r.standard_normal((3, 4)), r.standard_normal(5) * 10, np.zeros(0)]
    for limit in (0.5, 100.0):
        p = [torch.nn.Parameter(torch.zeros(a.shape, dtype=torch.float64)) for a in g]
        for q, a in zip(p, g):
            q.grad = torch.from_numpy(a.copy())
        n = torch.nn.utils.clip_grad_norm_(p, limit)
        norm, out = M.clip(g, limit)
        assert abs(float(n) - norm) < 1e-12
        for q, o in zip(p, out):
            np.testing.assert_allclose(q.grad.numpy(), o, atol=1e-12)
