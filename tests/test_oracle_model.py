"""The fp64 forms of the embedding, layer norm and cross entropy: gradients
against central differences, and pinned properties (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import model_oracle as M


def _difference(f, a, direction, h=1e-5):
    return (f(a + h * direction) - f(a - h * direction)) / (2 * h)


def test_bf16_rounding_is_torch_s():
    v = np.random.default_rng(0).standard_normal(4096).astype(np.float32) * 100
    v[:4] = [1.00390625, 1.01171875, 0.0, -0.0]        # ties go to even
    want = torch.from_numpy(v).to(torch.bfloat16).float().numpy()
    np.testing.assert_array_equal(M.round_bf16(v).astype(np.float32), want)


def test_embedding_grad_against_differences():
    r = np.random.default_rng(1)
    table, tok = r.standard_normal((13, 8)), np.array([3, 0, 3, -1, 12, 3, 5])
    c = r.standard_normal((7, 8))
    g, _, count = M.embedding_grad(tok, c, 13, scale=1.5)
    d = r.standard_normal(table.shape)
    num = _difference(lambda t: (M.embedding(tok, t, 1.5) * c).sum(), table, d)
    assert abs(num - (g * d).sum()) < 1e-8
    assert count[3] == 3 and count.sum() == 6 and not g[1].any()


@pytest.mark.parametrize("T,H", [(1, 8), (5, 24), (3, 200)])
def test_layer_norm_grad_against_differences(T, H):
    r = np.random.default_rng(H)
    s, w, b, c = r.standard_normal((T, H)) + 0.5, r.standard_normal(H), r.standard_normal(H), r.standard_normal((T, H))
    f = M.layer_norm(s, w, b)
    g = M.layer_norm_grad(c, s, w, f["mean"], f["rstd"])
    for name, arg, fun in (("dx", s, lambda a: (M.layer_norm(a, w, b)["y"] * c).sum()),
                           ("dweight", w, lambda a: (M.layer_norm(s, a, b)["y"] * c).sum()),
                           ("dbias", b, lambda a: (M.layer_norm(s, w, a)["y"] * c).sum())):
        d = r.standard_normal(arg.shape)
        assert abs(_difference(fun, arg, d) - (g[name] * d).sum()) < 1e-6, name


def test_cross_entropy_grad_against_differences():
    r = np.random.default_rng(7)
    x, w, lab = r.standard_normal((6, 16)), r.standard_normal((11, 16)), np.array([0, 10, -1, 4, 4, 7])
    dl = r.standard_normal(6)
    g = M.cross_entropy_grad(x, w, lab, dl)
    for name, arg, fun in (("dx", x, lambda a: (M.cross_entropy(a, w, lab)["loss"] * dl).sum()),
                           ("dw", w, lambda a: (M.cross_entropy(x, a, lab)["loss"] * dl).sum())):
        d = r.standard_normal(arg.shape)
        assert abs(_difference(fun, arg, d) - (g[name] * d).sum()) < 1e-7, name
    assert not g["dx"][2].any()
    np.testing.assert_allclose(g["d"].sum(1), 0.0, atol=1e-12)       # softmax minus one-hot sums to zero


def test_cross_entropy_is_torch_s():
    r = np.random.default_rng(8)
    x, w, lab = r.standard_normal((6, 16)), r.standard_normal((11, 16)), np.array([0, 10, -1, 4, 4, 7])
    t = torch.nn.functional.cross_entropy(torch.from_numpy(x @ w.T), torch.from_numpy(lab), ignore_index=-1,
                                          reduction="none")
    np.testing.assert_allclose(M.cross_entropy(x, w, lab)["loss"], t.numpy(), atol=1e-12)
