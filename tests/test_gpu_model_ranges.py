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


@pytest.mark.parametrize("T,H", [(1, 1024), (2, 4096), (5, 1024), (140, 4096), (140, 7168)])
def test_cross_entropy_gradient_vanishes_where_the_label_is_certain(lib, T, H):
    """Probabilities of other entries below e^-80 V: lse is the label's logit to the bit (its sum of exponentials is
    1 within 2^-22, the logit's place 2^-18 or more), so that entry's gradient is zero and the others' below e^-75."""
    V = 3000
    rng = np.random.default_rng(T + H)
    x, lab = _bf(rng, T, H), rng.permutation(V)[:T].astype(np.int32)
    w = _bf(rng, V, H, std=1 / np.sqrt(H)).float()
    xf = x.float()
    w[torch.from_numpy(lab).long()] += rng.uniform(85, 110) * xf / (xf * xf).sum(1, keepdim=True)
    xd, wd, ld = x.to(DEV), w.to(BF).to(DEV), _dev(lab)
    loss, lse, ws = _loss(xd, wd, ld)
    dx, dw = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(xd, wd, ld, lse, torch.ones(T, device=DEV), dx, dw, ws)
    assert not loss.any()
    assert dx.abs().max() <= 1e-25 and dw.abs().max() <= 1e-25


@pytest.mark.parametrize("T,H,V", [(4400, 64, 700), (9000, 72, 513), (1300, 16384, 300)])
def test_cross_entropy_several_groups_of_tiles(lib, T, H, V):
    """More row blocks than one group of the tile order holds, the last group shorter than the others."""
    rng = np.random.default_rng(T)
    x, w, lab = _bf(rng, T, H), _bf(rng, V, H, std=1.5 / np.sqrt(H)), _labels(rng, T, V, True)
    xd, wd, ld = x.to(DEV), w.to(DEV), _dev(lab)
    loss, lse, ws = _loss(xd, wd, ld)
    ref = M.cross_entropy(f64(x), f64(w), lab)
    tol = _dz(ref) + (V / 16 + 64) * U
    _within(f64(lse), ref["lse"], tol, "lse")
    _within(f64(loss), ref["loss"], np.where(lab >= 0, 2 * tol, 0.0), "loss")
    dl = (rng.standard_normal(T) / T).astype(np.float32)
    lse32 = ref["lse"].astype(np.float32)
    g = M.cross_entropy_grad(f64(x), f64(w), lab, dl.astype(np.float64), lse32.astype(np.float64))
    dx, dw = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(xd, wd, ld, _dev(lse32), _dev(dl), dx, dw, ws)
    dz = _dz(ref, H).max()
    for got, name in ((dx, "dx"), (dw, "dw")):
        _within(f64(got), g[name], 2.0 ** -8 * np.abs(g[name]) + 2.0 ** -7 * g[name + "_sq"]
                + (2 * dz + 2.0 ** -15) * g[name + "_mag"] + 1e-30, name)
    assert api.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T,H", [(1, 64), (2, 64), (50, 200), (300, 200), (5, 4160), (140, 4160)])
def test_cross_entropy_entries_masked_by_the_lowest_value(lib, T, H):
    """Rows of w at the lowest value of the type, against positive x: logits of -infinity (or nearly), which count
    for nothing; whole tiles and the first columns of others."""
    V = 1500
    rng = np.random.default_rng(T)
    x, w = _bf(rng, T, H).abs(), _bf(rng, V, H, std=0.5 / np.sqrt(H))
    masked = np.zeros(V, bool)
    masked[:300], masked[512:1024], masked[1100:1110] = True, True, True
    keep = np.nonzero(~masked)[0]
    wm = w.clone()
    wm[torch.from_numpy(masked)] = torch.finfo(BF).min
    lab = rng.integers(0, len(keep), T)
    ref = M.cross_entropy(f64(x), f64(w)[keep], lab)
    xd, wd, ld = x.to(DEV), wm.to(DEV), _dev(keep[lab], np.int32)
    loss, lse, ws = _loss(xd, wd, ld)
    tol = _dz(ref, H) + (V / 16 + 64) * U
    _within(f64(lse), ref["lse"], tol, "lse")
    _within(f64(loss), ref["loss"], 2 * tol, "loss")
    dx, dw = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(xd, wd, ld, lse, torch.ones(T, device=DEV), dx, dw, ws)
    g = M.cross_entropy_grad(f64(x), f64(w)[keep], lab, np.ones(T))
    scale = 2 * (_dz(ref, H).max() + tol.max()) + 2.0 ** -15
    for got, name in ((f64(dx), "dx"), (f64(dw)[keep], "dw")):
        _within(got, g[name], 2.0 ** -8 * np.abs(g[name]) + 2.0 ** -7 * g[name + "_sq"] + scale * g[name + "_mag"]
                + 1e-30, name)
    assert not f64(dw)[masked].any()


@pytest.mark.parametrize("T", [2, 50, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_cross_entropy_not_finite_rows_stay_alone(lib, T, value):
    """A scored row that is not finite has a loss and a dx of NaN and leaves the other rows' as they are."""
    H, V = 64, 700
    rng = np.random.default_rng(T)
    x, w, lab = _bf(rng, T, H), _bf(rng, V, H, std=0.2), _labels(rng, T, V, False)
    wd, ld = w.to(DEV), _dev(lab)
    out = []
    for bad in (False, True):
        xd = x.to(DEV)
        if bad:
            xd[1] = value
        loss, lse, ws = _loss(xd, wd, ld)
        dx, dw = _nan(T, H), _nan(V, H)
        api.moe_cross_entropy_backward(xd, wd, ld, lse, torch.ones(T, device=DEV), dx, dw, ws)
        out.append((loss, lse, dx, dw))
    others = torch.arange(T, device=DEV) != 1
    for a, b in zip(out[0][:3], out[1][:3]):
        assert torch.equal(a[others], b[others]) and torch.isfinite(a).all() and b[1].isnan().all()
    assert out[1][3].isnan().all()


# ----------------------------------------------------------------- layer norm
def _norm_grad_case(rng, T, H, spread=1.0):
    s = _bf(rng, T, H, std=spread, mean=0.3 * spread)
    return s, _bf(rng, H, std=0.2, mean=1.0), _bf(rng, T, H)


@pytest.mark.parametrize("T,H", [(30000, 64), (9000, 1000), (5000, 2056), (1500, 7168), (1400, 8192), (1000, 10248),
                                 (1000, 16384)])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_layer_norm_backward_many_rows_a_group(lib, T, H, with_dsum):
    """More rows for each group of warps than its ring holds: buffers used again, sums over rows."""
    rng = np.random.default_rng(T + H)
    s, w, dy = _norm_grad_case(rng, T, H)
    dsum = _bf(rng, T, H) if with_dsum else None
    f = M.layer_norm(f64(s), f64(w))
    mean, rstd = _dev(f["mean"], np.float32), _dev(f["rstd"], np.float32)
    dev = [t.to(DEV) for t in (dy, s, w)]
    dsum_d = None if dsum is None else dsum.to(DEV)
    ws = _ws(api.moe_layer_norm_workspace_bytes(T, H))
    got = []
    for _ in range(2):
        dx, dw, db = _nan(T, H), _nan(H, dtype=F32), _nan(H, dtype=F32)
        api.moe_layer_norm_backward(*dev, mean, rstd, dx, dw, db, ws, dsum=dsum_d)
        got.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ref = M.layer_norm_grad(f64(dy), f64(s), f64(w), f64(mean), f64(rstd), None if dsum is None else f64(dsum))
    chain, rows = H / 8 + 64, T / 100 + 80
    _within(f64(dx), ref["dx"], 2.0 ** -8 * np.abs(ref["dx"]) + (chain + 16) * U * ref["dx_mag"] + 1e-30, "dx")
    _within(f64(dw), ref["dweight"], (rows + 8) * U * ref["dweight_mag"] + 1e-30, "dweight")
    _within(f64(db), ref["dbias"], rows * U * ref["dbias_mag"] + 1e-30, "dbias")
    assert api.moe_read_device_status(ws) == 0


def test_layer_norm_backward_random_rows_past_32_bit_offsets(lib):
    """2.2e9 random elements; dx compared at both ends and across 2^31 elements, the sums over all rows."""
    T, H, step = 530_000, 4096, 10_000
    g = torch.Generator(device=DEV).manual_seed(21)
    s, dy, dx = (torch.empty(T, H, dtype=BF, device=DEV) for _ in range(3))
    for i in range(0, T, step):
        for t in (s, dy):
            t[i:i + step] = torch.randn(step, H, device=DEV, generator=g).to(BF)
    w = (1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(BF)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    dw_ref, db_ref, dw_mag, db_mag = torch.zeros(4, H, dtype=torch.float64, device=DEV)
    for i in range(0, T, step):
        rows = slice(i, i + step)
        c, d = s[rows].double(), dy[rows].double()
        mean[rows], rstd[rows] = c.mean(1).float(), torch.rsqrt(c.var(1, unbiased=False) + 1e-5).float()
        xh = (c - mean[rows, None].double()) * rstd[rows, None].double()
        dw_ref += (d * xh).sum(0)
        dw_mag += (d * xh).abs().sum(0)
        db_ref += d.sum(0)
        db_mag += d.abs().sum(0)
    dx.fill_(float("nan"))
    dw, db = _nan(H, dtype=F32), _nan(H, dtype=F32)
    ws = _ws(api.moe_layer_norm_workspace_bytes(T, H))
    api.moe_layer_norm_backward(dy, s, w, mean, rstd, dx, dw, db, ws)
    assert all(torch.isfinite(dx[i:i + step]).all() for i in range(0, T, step))
    at = (1 << 31) // H
    for rows in (slice(0, 300), slice(at - 150, at + 150), slice(T - 300, T)):
        ref = M.layer_norm_grad(f64(dy[rows]), f64(s[rows]), f64(w), f64(mean[rows]), f64(rstd[rows]))
        _within(f64(dx[rows]), ref["dx"], 2.0 ** -8 * np.abs(ref["dx"]) + (H / 8 + 80) * U * ref["dx_mag"], "dx")
    rows = T / 100 + 80
    _within(f64(dw), dw_ref.cpu().numpy(), (rows + 8) * U * dw_mag.cpu().numpy(), "dweight")
    _within(f64(db), db_ref.cpu().numpy(), rows * U * db_mag.cpu().numpy(), "dbias")
    assert api.moe_read_device_status(ws) == 0


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


@pytest.mark.parametrize("T,H", [(7, 64), (9, 1000), (700, 4096), (6, 16384)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_layer_norm_not_finite_rows_stay_alone(lib, T, H, value):
    rng = np.random.default_rng(T)
    x, w, dy = (t.to(DEV) for t in _norm_grad_case(rng, T, H))
    r = _bf(rng, T, H).to(DEV)
    out = []
    for bad in (False, True):
        xb = x.clone()
        if bad:
            xb[1, H // 2] = value
        y, s, dx, mean, rstd = _nan(T, H), _nan(T, H), _nan(T, H), _nan(T, dtype=F32), _nan(T, dtype=F32)
        api.moe_layer_norm_forward(xb, w, None, y, mean, rstd, residual=r, sum_out=s)
        api.moe_layer_norm_backward(dy, s, w, mean, rstd, dx, _nan(H, dtype=F32), None,
                                    _ws(api.moe_layer_norm_workspace_bytes(T, H)))
        out.append((y, mean, rstd, dx))
    others = torch.arange(T, device=DEV) != 1
    for a, b in zip(*out):
        assert torch.equal(a[others], b[others]) and torch.isfinite(a).all()
    assert out[1][0][1].isnan().all() and out[1][3][1].isnan().all()


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
