"""The embedding, the layer norm and the vocabulary cross entropy where their
kernels take another course than at small sizes: several rows for each group of
warps, several groups of tiles, a dominant logit in a large vocabulary, values
at the ends of the number range, and what is not finite.  Against the fp64
oracle, as in test_gpu_model.py, whose error bounds are used where none is
derived here."""
import numpy as np
import pytest
import torch

from gpu_helpers import f64
from moe_expert_layer_05_gb300 import api
from oracle import model_oracle as M
from test_gpu_model import BF, DEV, U, _bf, _dz, _labels, _nan, _within, _ws

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _dev(a, dtype=None):
    return torch.from_numpy(np.asarray(a, dtype)).to(DEV)


def _loss(x, w, lab):
    """loss, lse and the workspace of one forward call (inputs on the device)."""
    T, (V, H) = len(x), w.shape
    loss, lse = _nan(T, dtype=F32), _nan(T, dtype=F32)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V))
    api.moe_cross_entropy_forward(x, w, lab, loss, lse, ws)
    return loss, lse, ws


# -------------------------------------------------------------- cross entropy
@pytest.mark.parametrize("T,H", [(1, 64), (2, 64), (40, 64), (140, 64), (5, 4160), (140, 4160)])
@pytest.mark.parametrize("top", [20.25, 90.0])
def test_cross_entropy_dominant_label_in_a_large_vocabulary(lib, T, H, top):
    """Rows that are sure of their label: the sum of exponentials is one and a little, so the loss is what the sum's
    errors leave.  The label's logit is the same fp32 value in both terms of the loss.  A pair of sums is joined
    with one rounding of the larger (fewer than V / 2048 + 96 in a row) and an exponential of zero, which is exact;
    what is smaller by e^20 does not count; then lse is rounded once, and the logarithm's argument twice more."""
    V, label = 131072 if H < 4096 else 32768, 3
    rng = np.random.default_rng(T + H)
    x, w = _bf(rng, T, H, std=0.1), _bf(rng, V, H, std=0.1)
    x[:, 0], w[:, 0], w[label, 0] = top, 0.0, 1.0
    ref = M.cross_entropy(f64(x), f64(w), np.full(T, label))
    loss, lse, _ = _loss(x.to(DEV), w.to(DEV), torch.full((T,), label, dtype=torch.int32, device=DEV))
    ulp = np.spacing(ref["lse"].astype(np.float32)).astype(np.float64)
    _within(f64(loss), ref["loss"], (V / 2048 + 96) * U + 1.5 * ulp, "loss")
    assert (f64(loss) >= -ulp).all()


def test_cross_entropy_backward_reports_bad_labels(lib):
    H, V = 64, 300
    for T in (6, 200):                                    # (d in two parts, and in one)
        rng = np.random.default_rng(T)
        x, w = _bf(rng, T, H).to(DEV), _bf(rng, V, H, std=0.1).to(DEV)
        good = rng.integers(0, V, T).astype(np.int32)
        good[::3] = -1
        for bad in (V, -2, 511, 2 ** 31 - 1, -(2 ** 31), None):
            lab = good.copy()
            if bad is not None:
                lab[T - 1] = bad
            _, lse, ws = _loss(x, w, _dev(lab))
            api.moe_workspace_init(ws[:256])
            api.moe_cross_entropy_backward(x, w, _dev(lab), lse, torch.ones(T, device=DEV), _nan(T, H), _nan(V, H), ws)
            assert api.moe_read_device_status(ws) == (0 if bad is None else -5), (T, bad)


def _sure_rows(T, H, top):
    """Each row sure of a label of its own (p within e^-top V of 1): what is left of exp(z - lse) - 1 there is the
    gradient, and the error of z - lse its error.  z is the same fp32 value in the forward's lse and here, so that
    error is lse's rounding (half an ulp), the product's with log2 e (less than one ulp of lse) and the relative
    error of lse's sum (2 (V / 2048 + 96) u, with the two exponentials' 2^-21); an error of z itself counts only in
    proportion to d.  The rest as for other rows."""
    V = 8192
    rng = np.random.default_rng(T + H)
    x, lab = _bf(rng, T, H), rng.permutation(V)[:T].astype(np.int32)
    w = _bf(rng, V, H, std=1 / np.sqrt(H)).float()
    xf = x.float()
    w[torch.from_numpy(lab).long()] += top * xf / (xf * xf).sum(1, keepdim=True)
    w = w.to(BF)
    xd, wd, ld = x.to(DEV), w.to(DEV), _dev(lab)
    _, lse, ws = _loss(xd, wd, ld)
    dl = (rng.uniform(0.5, 1.5, T) / T).astype(np.float32)
    dx, dw = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(xd, wd, ld, lse, _dev(dl), dx, dw, ws)
    ref = M.cross_entropy(f64(x), f64(w), lab)
    g = M.cross_entropy_grad(f64(x), f64(w), lab, dl.astype(np.float64))
    dz = 2 * _dz(ref, H).max()
    ulp = np.spacing(ref["lse"].astype(np.float32)).astype(np.float64)
    d_err = dl * (1.5 * ulp + 2 * (V / 2048 + 96) * U + 2.0 ** -21)
    label_err = {"dx": d_err[:, None] * np.abs(f64(w)[lab]), "dw": np.zeros(w.shape)}
    label_err["dw"][lab] = d_err[:, None] * np.abs(f64(x))
    for got, name in ((dx, "dx"), (dw, "dw")):
        _within(f64(got), g[name], 2.0 ** -8 * np.abs(g[name]) + 2.0 ** -7 * g[name + "_sq"]
                + (2 * dz + 2.0 ** -15) * g[name + "_mag"] + 1.01 * label_err[name] + 1e-30, name)
    assert api.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T,H", [(5, 1024), (140, 4096), (3, 7168), (70, 4104), (140, 7168), (33, 16384)])
@pytest.mark.parametrize("top", [20.0, 60.0])
def test_cross_entropy_gradient_of_sure_rows(lib, T, H, top):
    _sure_rows(T, H, top)


@pytest.mark.parametrize("T,H", [(1, 64), (1, 1024), (2, 1024), (1, 7168), (2, 4096)])
@pytest.mark.parametrize("top", [20.0, 60.0])
def test_cross_entropy_gradient_of_one_or_two_sure_rows(lib, T, H, top):
    _sure_rows(T, H, top)


# ----------------------------------------------------------------- layer norm
def _norm_grad_case(rng, T, H, spread=1.0):
    s = _bf(rng, T, H, std=spread, mean=0.3 * spread)
    return s, _bf(rng, H, std=0.2, mean=1.0), _bf(rng, T, H)


@pytest.mark.parametrize("H", [512, 4096, 10248])
@pytest.mark.parametrize("size", [1e-20, 3e18])
def test_layer_norm_backward_at_the_ends_of_the_range(lib, H, size):
    """Rows so small (eps = 0) or large that the square of their rstd leaves fp32: rstd and dx do not."""
    T = 40
    rng = np.random.default_rng(H)
    s, w, dy = _norm_grad_case(rng, T, H, spread=size)
    f = M.layer_norm(f64(s), f64(w), eps=0.0)
    mean, rstd = _dev(f["mean"], np.float32), _dev(f["rstd"], np.float32)
    dx, dw, db = _nan(T, H), _nan(H, dtype=F32), _nan(H, dtype=F32)
    ws = _ws(api.moe_layer_norm_workspace_bytes(T, H))
    api.moe_layer_norm_backward(dy.to(DEV), s.to(DEV), w.to(DEV), mean, rstd, dx, dw, db, ws)
    ref = M.layer_norm_grad(f64(dy), f64(s), f64(w), f64(mean), f64(rstd))
    chain = H / 8 + 64
    _within(f64(dx), ref["dx"], 2.0 ** -8 * np.abs(ref["dx"]) + (chain + 16) * U * ref["dx_mag"], "dx")
    _within(f64(dw), ref["dweight"], 88 * U * ref["dweight_mag"] + 1e-30, "dweight")


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("H", [64, 2056])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -3.0])
def test_embedding_padding_is_zero_whatever_the_scale(lib, H, scale):
    V = 20
    table = _bf(np.random.default_rng(H), V, H).to(DEV)
    tok = torch.tensor([3, -1, 19, -1, 0], dtype=torch.int32, device=DEV)
    out, ws = _nan(5, H), _ws(256)
    api.moe_embedding_forward(tok, table, out, ws, scale=scale)
    pad = tok < 0
    assert not out[pad].view(torch.int16).any()              # (+0, to the bit)
    want = (table[tok[~pad].long()].float() * scale).to(BF)
    assert torch.equal(out[~pad].nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
