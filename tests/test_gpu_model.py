"""GPU parity of the token embedding, the layer norm and the vocabulary cross
entropy, through the C ABI, against the fp64 oracle on the same seeded inputs.

Tolerances (derived, u = 2^-24 the unit rounding of fp32):
  * a value rounded once to bf16: 2^-8 |ref|;
  * an fp32 sum of m terms in any order: (m + c) u times the sum of the terms'
    magnitudes, c for the roundings of a term itself;
  * logits: K exact bf16 products added in fp32 on the tensor cores, which
    align and truncate: K/16 steps of at most 2^-23 of the partial sum, which
    is below sum |x w|; 2^-15 of it covers K up to 4096 (the forward adds longer
    ones in segments of 2048, the gradient's logits take K/16 2^-23 of it);
  * gradients of the cross entropy: their operand d is rounded to bf16, an
    independent error of at most 2^-9 per term, of standard deviation below
    2^-9.8: six of them, and the terms in quadrature, give 2^-7 sqrt(sum of
    squared terms); d's own relative error from the logits is 2 dz.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import f64, i64, rel_l2
from moe_expert_layer_05_gb300 import api
from oracle import model_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF = torch.bfloat16


def _bf(rng, *shape, std=1.0, mean=0.0):
    return torch.from_numpy((rng.standard_normal(shape, dtype=np.float32) * np.float32(std) + np.float32(mean))).to(BF)


def _ws(nbytes):
    """A workspace whose scratch holds garbage (only the status region is initialised)."""
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
    api.moe_workspace_init(ws[:256])
    return ws


def _nan(*shape, dtype=BF):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def _within(got, ref, bound, what):
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{what}: worst excess {over.max():.3e}, {int((over > 0).sum())} values"


# ------------------------------------------------------------------ embedding
def _tokens(rng, n, V, kind):
    if kind == "same":
        t = np.full(n, V - 1)
    elif kind == "zipf":
        t = np.minimum(rng.zipf(1.3, n) - 1, V - 1)
    elif kind == "none":
        t = np.full(n, -1)
    else:
        t = rng.integers(0, V, n)
    t = t.astype(np.int32)
    if kind in ("zipf", "random") and n > 3:
        t[rng.random(n) < 0.1] = -1
    return t


@pytest.mark.parametrize("n,V,H,scale", [(1, 5, 8, 1.0), (7, 1000, 64, 8.0), (1003, 257, 1000, 0.3),
                                         (300, 5003, 4096, 64.0), (5, 3, 16384, 1.0)])
def test_embedding_forward_exact(lib, n, V, H, scale):
    rng = np.random.default_rng(n + H)
    table, tok = _bf(rng, V, H, std=0.02), _tokens(rng, n, V, "random")
    out, ws = _nan(n, H), _ws(256)
    api.moe_embedding_forward(torch.from_numpy(tok).to(DEV), table.to(DEV), out, ws, scale=scale)
    rows = table.float()[torch.from_numpy(np.maximum(tok, 0)).long()] * np.float32(scale)
    want = (rows * torch.from_numpy(tok >= 0)[:, None]).to(BF)
    assert torch.equal(out.cpu().float(), want.float())
    assert api.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("n,V,H", [(0, 7, 64), (1, 1, 8), (1, 1000, 128), (63, 10, 64), (64, 10, 64), (65, 3, 1000), (128, 90, 1032), (129, 90, 1032),
                                   (2048, 256, 64), (2049, 255, 72), (4097, 600, 64), (5000, 70000, 64), (16384, 700, 256),
                                   (20011, 50001, 128), (70000, 65536, 16), (16385, 300_000, 8), (65536, 40_000, 8), (65537, 40_001, 8),
                                   (70001, 300_000, 8)])
@pytest.mark.parametrize("kind", ["random", "zipf", "same", "none"])
@pytest.mark.parametrize("tied", [False, True])
def test_embedding_backward(lib, n, V, H, kind, tied):
    rng = np.random.default_rng(n + V)
    tok, dy = _tokens(rng, n, V, kind), _bf(rng, n, H)
    base = _bf(rng, V, H, std=0.1) if tied else None
    scale = 1.0 if n % 2 else 5.5
    dt, ws = _nan(V, H, dtype=torch.float32), _ws(api.moe_embedding_workspace_bytes(n, V, H))
    args = (torch.from_numpy(tok).to(DEV), dy.to(DEV))
    base_d = base.to(DEV) if tied else None
    api.moe_embedding_backward(*args, dt, ws, scale=scale, base=base_d)
    ref, mag, count = M.embedding_grad(tok.astype(np.int64), f64(dy), V, scale, f64(base) if tied else None)
    _within(f64(dt), ref, (count[:, None] + 4) * U * mag, "dtable")
    again = _nan(V, H, dtype=torch.float32)
    api.moe_embedding_backward(*args, again, ws, scale=scale, base=base_d)
    assert torch.equal(dt, again)                       # the same bits on a used workspace
    assert api.moe_read_device_status(ws) == 0


def test_embedding_backward_at_16_byte_alignment(lib):
    """Buffers that start 16 bytes into an allocation: the least the calls ask for."""
    n, V, H = 300, 40, 72
    rng = np.random.default_rng(8)
    tok, dy, base = _tokens(rng, n, V, "zipf"), _bf(rng, n, H), _bf(rng, V, H)
    flat = lambda *shape, dtype, off: torch.full((int(np.prod(shape)) + off,), float("nan"), dtype=dtype,   # noqa: E731
                                                 device=DEV)[off:].view(*shape)
    dt, dyd, based = flat(V, H, dtype=torch.float32, off=4), flat(n, H, dtype=BF, off=8), flat(V, H, dtype=BF, off=8)
    dyd.copy_(dy), based.copy_(base)
    tokd = torch.zeros(n + 4, dtype=torch.int32, device=DEV)[4:]
    tokd.copy_(torch.from_numpy(tok))
    need = api.moe_embedding_workspace_bytes(n, V, H)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device=DEV)[16:]
    api.moe_workspace_init(ws[:256])
    api.moe_embedding_backward(tokd, dyd, dt, ws, base=based)
    ref, mag, count = M.embedding_grad(tok.astype(np.int64), f64(dy), V, 1.0, f64(base))
    _within(f64(dt), ref, (count[:, None] + 4) * U * mag, "dtable")


def test_embedding_bad_ids_are_reported_and_left_out(lib):
    V, H = 50, 64
    rng = np.random.default_rng(5)
    tok = np.array([0, 49, 50, -2, 2 ** 31 - 1, -(2 ** 31), -1, 7], np.int32)
    table, dy = _bf(rng, V, H).to(DEV), _bf(rng, 8, H).to(DEV)
    t = torch.from_numpy(tok).to(DEV)
    ws, out = _ws(api.moe_embedding_workspace_bytes(8, V, H)), _nan(8, H)
    api.moe_embedding_forward(t, table, out, ws)
    assert api.moe_read_device_status(ws) == -5
    good = torch.tensor([0, 1, 7], device=DEV)
    assert torch.equal(out[good], table[t[good].long()]) and not out[2:7].any()
    api.moe_workspace_init(ws[:256])
    dt = _nan(V, H, dtype=torch.float32)
    api.moe_embedding_backward(t, dy, dt, ws)
    assert api.moe_read_device_status(ws) == -5
    want = torch.zeros(V, H, device=DEV)
    want[t[good].long()] = dy[good].float()
    assert torch.equal(dt, want)


def test_embedding_past_32_bit_offsets(lib):
    V, H, n = 600_000, 4096, 257           # 2.4e9 elements
    g = torch.Generator(device=DEV).manual_seed(3)
    table = torch.empty(V, H, dtype=BF, device=DEV)
    tok = torch.randint(V - 5000, V, (n,), device=DEV, generator=g, dtype=torch.int32)
    tok[0], tok[1] = V - 1, 0
    table[tok.long()] = torch.randn(n, H, device=DEV, generator=g).to(BF)
    ws, out = _ws(api.moe_embedding_workspace_bytes(n, V, H)), _nan(n, H)
    api.moe_embedding_forward(tok, table, out, ws)
    assert torch.equal(out, table[tok.long()])
    del table
    dt = _nan(V, H, dtype=torch.float32)
    api.moe_embedding_backward(tok, out, dt, ws)
    used = torch.zeros(V, dtype=torch.bool, device=DEV)
    used[tok.long()] = True
    assert not dt[~used].any()
    want = torch.zeros(V, 8, dtype=torch.float64, device=DEV).index_add_(0, tok.long(), out[:, -8:].double())
    assert (dt[:, -8:].double() - want).abs().max() < 1e-4


# ----------------------------------------------------------------- layer norm
LN_SHAPES = [(1, 8), (1, 4096), (3, 64), (37, 1000), (300, 1024), (305, 1032), (64, 2048), (33, 4104), (130, 7168),
             (1003, 1000), (9, 8192), (5, 16384)]


def _ln_row(rng, T, H):
    """Rows of unlike mean and size, among them a constant one (variance zero) and one with a large mean."""
    x = rng.standard_normal((T, H), dtype=np.float32) * np.exp(rng.standard_normal((1, H), dtype=np.float32) * 0.5)
    if T > 2:
        x[1] = 0.75
        x[2] = x[2] * 0.5 + 100.0
    return torch.from_numpy(x).to(BF)


@pytest.mark.parametrize("T,H", LN_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_layer_norm_forward(lib, T, H, residual, with_bias):
    rng = np.random.default_rng(T * H)
    x, w = _ln_row(rng, T, H), _bf(rng, H, std=0.2, mean=1.0)
    b = _bf(rng, H, std=0.2) if with_bias else None
    r = _bf(rng, T, H, std=2.0) if residual else None
    dev = lambda t: None if t is None else t.to(DEV)                    # noqa: E731
    y, mean, rstd = _nan(T, H), _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
    s_out = _nan(T, H) if residual else None
    api.moe_layer_norm_forward(dev(x), dev(w), dev(b), y, mean, rstd, residual=dev(r), sum_out=s_out, eps=1e-5)
    s = f64(x) if not residual else M.round_bf16((x.float() + r.float()).numpy())
    if residual:
        np.testing.assert_array_equal(f64(s_out), s)
    ref = M.layer_norm(s, f64(w), None if b is None else f64(b))
    m = H / 8 + 64                            # roundings along the longest chain of a row's sum
    mean_err = (m * U) * np.abs(s).mean(1)
    _within(f64(mean), ref["mean"], mean_err + 1e-30, "mean")
    # variance: each term relative, plus the mean's error twice through (s - mu)
    var = ((s - ref["mean"][:, None]) ** 2).mean(1)
    var_err = (m + 8) * U * var + 2 * mean_err * np.sqrt(var) + mean_err ** 2
    rstd_rel = 0.5 * var_err / (var + 1e-5) + 8 * U
    _within(f64(rstd), ref["rstd"], rstd_rel * ref["rstd"], "rstd")
    xh = (s - ref["mean"][:, None]) * ref["rstd"][:, None]
    slack = np.abs(f64(w)) * (np.abs(xh) * (rstd_rel[:, None] + 4 * U) + (mean_err * ref["rstd"])[:, None]
                              + 4 * U * np.abs(s) * ref["rstd"][:, None])
    _within(f64(y), ref["y"], 2.0 ** -8 * np.abs(ref["y"]) + 1.01 * slack + 1e-30, "y")


@pytest.mark.parametrize("T,H", LN_SHAPES)
@pytest.mark.parametrize("with_dsum", [False, True])
def test_layer_norm_backward(lib, T, H, with_dsum):
    rng = np.random.default_rng(T * H + 1)
    s, w, dy = _ln_row(rng, T, H), _bf(rng, H, std=0.2, mean=1.0), _bf(rng, T, H)
    dsum = _bf(rng, T, H) if with_dsum else None
    f = M.layer_norm(f64(s), f64(w))
    mean, rstd = (torch.from_numpy(f[k].astype(np.float32)).to(DEV) for k in ("mean", "rstd"))
    dx, dw, db = _nan(T, H), _nan(H, dtype=torch.float32), _nan(H, dtype=torch.float32)
    ws = _ws(api.moe_layer_norm_workspace_bytes(T, H))
    run = lambda dx, dw, db: api.moe_layer_norm_backward(                # noqa: E731
        dy.to(DEV), s.to(DEV), w.to(DEV), mean, rstd, dx, dw, db, ws, dsum=None if dsum is None else dsum.to(DEV))
    run(dx, dw, db)
    ref = M.layer_norm_grad(f64(dy), f64(s), f64(w), f64(mean), f64(rstd), None if dsum is None else f64(dsum))
    # (s - mu) rounds once: relative to |s - mu|, so xh keeps a relative error of 2 u
    chain = H / 8 + 64
    _within(f64(dx), ref["dx"], 2.0 ** -8 * np.abs(ref["dx"]) + (chain + 16) * U * ref["dx_mag"] + 1e-30, "dx")
    rows = T / 100 + 80                       # rows a block adds, then the blocks' sums
    _within(f64(dw), ref["dweight"], (rows + 8) * U * ref["dweight_mag"] + 1e-30, "dweight")
    _within(f64(db), ref["dbias"], rows * U * ref["dbias_mag"] + 1e-30, "dbias")
    dx2, dw2 = _nan(T, H), _nan(H, dtype=torch.float32)
    run(dx2, dw2, None)                       # without a bias; the same bits
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_layer_norm_backward_against_differences(lib):
    """The kernels' own forward, differenced: <c, y(s + h d) - y(s - h d)> / 2h against <dx, d>.  s on a grid of
    2^-6 with steps of 2^-6, so the stepped inputs are exact in bf16; y's rounding (2^-9 of values near 1, in
    quadrature over T H terms, over 2h) leaves about 2^-9 * sqrt(2 T H) / (2 h sqrt(12))."""
    T, H, h = 16, 512, 2.0 ** -6
    rng = np.random.default_rng(11)
    s = np.round(rng.uniform(-1.9, 1.9, (T, H)) * 64) / 64
    d = rng.choice([-1.0, 1.0], (T, H))
    c, w = _bf(rng, T, H), _bf(rng, H, std=0.2, mean=1.0)
    out = {}
    for sign in (1.0, -1.0, 0.0):
        y, mean, rstd = _nan(T, H), _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
        api.moe_layer_norm_forward(torch.from_numpy(s + sign * h * d).to(BF).to(DEV), w.to(DEV), None, y, mean, rstd)
        out[sign] = f64(y), mean, rstd
    num = ((out[1.0][0] - out[-1.0][0]) * f64(c)).sum() / (2 * h)
    dx, dw, db = _nan(T, H), _nan(H, dtype=torch.float32), _nan(H, dtype=torch.float32)
    api.moe_layer_norm_backward(c.to(DEV), torch.from_numpy(s).to(BF).to(DEV), w.to(DEV), out[0.0][1], out[0.0][2], dx,
                                dw, db, _ws(api.moe_layer_norm_workspace_bytes(T, H)))
    noise = 2.0 ** -9 * np.sqrt(2 * T * H) / (2 * h * np.sqrt(12))
    assert abs(num - (f64(dx) * d).sum()) <= 6 * noise + 1e-2 * np.sqrt(T * H)


def test_layer_norm_no_rows(lib):
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    v = torch.empty(0, dtype=torch.float32, device=DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    api.moe_layer_norm_forward(e, w, None, e, v, v)
    dw, db = _nan(64, dtype=torch.float32), _nan(64, dtype=torch.float32)
    api.moe_layer_norm_backward(e, e, w, v, v, e, dw, db, _ws(256))
    assert not dw.any() and not db.any()


def test_layer_norm_past_32_bit_offsets(lib):
    T, H = 530_000, 4096                     # 2.2e9 elements
    x = torch.empty(T, H, dtype=BF, device=DEV)
    x[-3:] = torch.randn(3, H, device=DEV).to(BF)
    x[:-3] = 0.0
    w = torch.ones(H, dtype=BF, device=DEV)
    y, mean, rstd = torch.empty_like(x), _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
    api.moe_layer_norm_forward(x, w, None, y, mean, rstd)
    ref = M.layer_norm(f64(x[-3:]), np.ones(H))
    assert np.abs(f64(y[-3:]) - ref["y"]).max() < 0.02 and not y[:-3].any()
    dx, dw, db = torch.empty_like(x), _nan(H, dtype=torch.float32), _nan(H, dtype=torch.float32)
    api.moe_layer_norm_backward(y, x, w, mean, rstd, dx, dw, db, _ws(api.moe_layer_norm_workspace_bytes(T, H)))
    g = M.layer_norm_grad(f64(y[-3:]), f64(x[-3:]), np.ones(H), f64(mean[-3:]), f64(rstd[-3:]))
    assert np.abs(f64(dx[-3:]) - g["dx"]).max() < 0.02
    np.testing.assert_allclose(f64(dw), g["dweight"], rtol=1e-4, atol=1e-4)


# -------------------------------------------------------------- cross entropy
def _labels(rng, T, V, ignored):
    t = rng.integers(0, V, T).astype(np.int32)
    t[0], t[-1] = V - 1, 0 if T > 1 else V - 1
    if ignored:
        t[rng.random(T) < 0.3] = -1
    return t


def _dz(ref, K=4096):
    return max(2.0 ** -15, K / 16 * 2.0 ** -23) * ref["z_mag"] + 2.0 ** -22 * (np.abs(ref["lse"]) + 1)


CE_SHAPES = [(1, 8, 1), (1, 64, 1000), (2, 8, 255), (5, 72, 256), (64, 200, 257), (127, 1000, 511), (128, 128, 5003),
             (129, 1000, 5003), (256, 64, 1000), (300, 264, 769), (1003, 1000, 2049), (513, 4096, 3001),
             (3000, 64, 300), (2500, 512, 1025),
             (3, 7168, 513), (70, 8192, 511), (131, 4104, 300), (300, 16384, 257)]


@pytest.mark.parametrize("T,H,V", CE_SHAPES)
def test_cross_entropy_forward(lib, T, H, V):
    rng = np.random.default_rng(T + H + V)
    x, w, lab = _bf(rng, T, H), _bf(rng, V, H, std=1.5 / np.sqrt(H)), _labels(rng, T, V, T > 4)
    loss, lse = _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V))
    api.moe_cross_entropy_forward(x.to(DEV), w.to(DEV), torch.from_numpy(lab).to(DEV), loss, lse, ws)
    ref = M.cross_entropy(f64(x), f64(w), lab)
    tol = _dz(ref) + (V / 16 + 64) * U                        # log of a sum of positive terms: its relative error
    _within(f64(lse), ref["lse"], tol, "lse")
    _within(f64(loss), ref["loss"], np.where(lab >= 0, 2 * tol, 0.0), "loss")
    assert api.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T,H,V", CE_SHAPES)
@pytest.mark.parametrize("piece", [0, 256, 700])
def test_cross_entropy_backward(lib, T, H, V, piece):
    rng = np.random.default_rng(T + H + V + 1)
    x, w, lab = _bf(rng, T, H), _bf(rng, V, H, std=1.5 / np.sqrt(H)), _labels(rng, T, V, T > 4)
    fwd = M.cross_entropy(f64(x), f64(w), lab)
    lse32 = fwd["lse"].astype(np.float32)
    dl = (rng.standard_normal(T) / T).astype(np.float32)
    x2 = x.clone()
    dl2, lse2 = dl.copy(), lse32.copy()
    for i, t in enumerate(np.nonzero(lab < 0)[0]):            # what an unscored row holds must not matter
        x2[t] = [float("nan"), float("inf"), 3e38][i % 3]
        dl2[t], lse2[t] = [(np.nan, np.nan), (np.inf, -np.inf), (1.0, np.inf)][i % 3]
    dx, dw = _nan(T, H), _nan(V, H)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V, piece))
    args = [t.to(DEV) for t in (x2, w, torch.from_numpy(lab), torch.from_numpy(lse2), torch.from_numpy(dl2))]
    api.moe_cross_entropy_backward(*args, dx, dw, ws, piece=piece)
    ref = M.cross_entropy_grad(f64(x), f64(w), lab, dl.astype(np.float64), lse32.astype(np.float64))
    dz = _dz(fwd, H).max()
    for got, name in ((dx, "dx"), (dw, "dw")):
        bound = (2.0 ** -8 * np.abs(ref[name]) + 2.0 ** -7 * ref[name + "_sq"]
                 + (2 * dz + 2.0 ** -15) * ref[name + "_mag"] + 1e-30)
        _within(f64(got), ref[name], bound, name)
    assert not f64(dx)[lab < 0].any()
    dx2, dw2 = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(*args, dx2, dw2, ws, piece=piece)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)      # the same bits on a used workspace
    assert api.moe_read_device_status(ws) == 0


def test_cross_entropy_training_sizes(lib):
    """Rel-L2 of the gradients at a larger size: two roundings of 2^-9 (the operand's and the output's), each of
    relative standard deviation 1.7e-3, stay below 4e-3 together."""
    T, H, V = 700, 2048, 20011
    rng = np.random.default_rng(3)
    x, w, lab = _bf(rng, T, H), _bf(rng, V, H, std=0.02), _labels(rng, T, V, True)
    xd, wd, ld = x.to(DEV), w.to(DEV), torch.from_numpy(lab).to(DEV)
    loss, lse = _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V))
    api.moe_cross_entropy_forward(xd, wd, ld, loss, lse, ws)
    dl = torch.full((T,), 1.0 / T, device=DEV)
    dx, dw = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(xd, wd, ld, lse, dl, dx, dw, ws)
    ref = M.cross_entropy_grad(f64(x), f64(w), lab, np.full(T, 1.0 / T))
    assert rel_l2(f64(dx), ref["dx"]) <= 4e-3 and rel_l2(f64(dw), ref["dw"]) <= 4e-3
    assert abs(f64(loss).sum() - M.cross_entropy(f64(x), f64(w), lab)["loss"].sum()) <= 2e-5 * T * np.log(V)


@pytest.mark.parametrize("T,skip,equal", [(1, 0, True), (2, 0, False), (33, 1, True), (64, 0, False), (65, 0, True),
                                          (600, 300, True), (2000, 1500, True)])
@pytest.mark.parametrize("piece", [0, 1024])
def test_cross_entropy_few_rows_or_equal_weights(lib, T, skip, equal, piece):
    """Where the roundings of d do not average out over rows: few of them, or all of one weight, half a place above a
    power of two, where its own rounding costs most (3.9e-3).  What is left is the rounding of the exact gradients to
    bf16 (about 1.7e-3 in rel-L2), and for equal weights the label's probability, below the last place of -1 + p: its
    root mean square is e^(1/2) / V = 3.3e-4 for logits of deviation one.  Independent errors add up in squares."""
    H, V = 512, 5000
    rng = np.random.default_rng(T)
    x, w, lab = _bf(rng, T, H), _bf(rng, V, H, std=1.0 / np.sqrt(H)), _labels(rng, T, V, False)
    lab[:skip] = -1
    dl = np.full(T, (1 + 0.99 * 2.0 ** -8) * 2.0 ** -9, np.float32)
    if not equal:
        dl *= rng.uniform(1.0, 1.003, T).astype(np.float32)
    fwd = M.cross_entropy(f64(x), f64(w), lab)
    ref = M.cross_entropy_grad(f64(x), f64(w), lab, np.where(lab >= 0, dl, 0.0).astype(np.float64))
    dl[:skip] = np.nan
    dx, dw = _nan(T, H), _nan(V, H)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V, piece))
    api.moe_cross_entropy_backward(x.to(DEV), w.to(DEV), torch.from_numpy(lab).to(DEV),
                                   torch.from_numpy(fwd["lse"].astype(np.float32)).to(DEV),
                                   torch.from_numpy(dl).to(DEV), dx, dw, ws, piece=piece)
    for got, name in ((dx, "dx"), (dw, "dw")):
        rounded = rel_l2(f64(torch.from_numpy(ref[name]).to(torch.bfloat16)), ref[name])
        assert rel_l2(f64(got), ref[name]) <= np.hypot(rounded, 2 * 3.3e-4)
    assert not f64(dx)[:skip].any()
    assert api.moe_read_device_status(ws) == 0


def test_cross_entropy_extreme_logits(lib):
    """Logits of several hundred in both signs: the running maximum keeps every exponential finite, and
    probabilities that underflow are zero."""
    T, H, V = 140, 64, 3000
    rng = np.random.default_rng(4)
    x, w, lab = _bf(rng, T, H, std=8.0), _bf(rng, V, H, std=4.0), _labels(rng, T, V, False)
    for rows in (T, 3):
        loss, lse = _nan(rows, dtype=torch.float32), _nan(rows, dtype=torch.float32)
        xd, wd, ld = x[:rows].to(DEV), w.to(DEV), torch.from_numpy(lab[:rows]).to(DEV)
        ws = _ws(api.moe_cross_entropy_workspace_bytes(rows, H, V))
        api.moe_cross_entropy_forward(xd, wd, ld, loss, lse, ws)
        ref = M.cross_entropy(f64(x[:rows]), f64(w), lab[:rows])
        tol = _dz(ref) + (V / 16 + 64) * U
        assert np.abs(ref["z"]).max() > 300
        _within(f64(lse), ref["lse"], tol, "lse")
        _within(f64(loss), ref["loss"], 2 * tol, "loss")
        dx, dw = _nan(rows, H), _nan(V, H)
        api.moe_cross_entropy_backward(xd, wd, ld, lse, torch.ones(rows, device=DEV), dx, dw, ws)
        g = M.cross_entropy_grad(f64(x[:rows]), f64(w), lab[:rows], np.ones(rows))
        scale = 2 * tol.max() + 2.0 ** -15
        _within(f64(dx), g["dx"], 2.0 ** -8 * np.abs(g["dx"]) + 2.0 ** -7 * g["dx_sq"] + scale * (g["dx_mag"] + np.abs(f64(w)).max()), "dx")


def test_cross_entropy_bad_labels_are_reported_and_left_out(lib):
    T, H, V = 6, 64, 300
    rng = np.random.default_rng(6)
    x, w = _bf(rng, T, H).to(DEV), _bf(rng, V, H, std=0.1).to(DEV)
    lab = torch.tensor([0, 299, 300, -2, 511, -1], dtype=torch.int32, device=DEV)
    none = torch.tensor([0, 299, -1, -1, -1, -1], dtype=torch.int32, device=DEV)
    got = []
    for l, code in ((lab, -5), (none, 0)):
        ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V))
        loss, lse = _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
        api.moe_cross_entropy_forward(x, w, l, loss, lse, ws)
        assert api.moe_read_device_status(ws) == code
        dx, dw = _nan(T, H), _nan(V, H)
        api.moe_cross_entropy_backward(x, w, l, lse, torch.ones(T, device=DEV), dx, dw, ws)
        got.append((loss, lse, dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not got[0][0][2:].any() and not got[0][2][2:].any()


def test_cross_entropy_no_tokens(lib):
    e, v = torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, dtype=torch.float32, device=DEV)
    lab, w = torch.empty(0, dtype=torch.int32, device=DEV), torch.ones(300, 64, dtype=BF, device=DEV)
    ws, dw = _ws(api.moe_cross_entropy_workspace_bytes(0, 64, 300)), _nan(300, 64)
    api.moe_cross_entropy_forward(e, w, lab, v, v, ws)
    api.moe_cross_entropy_backward(e, w, lab, v, v, e, dw, ws)
    assert not dw.any()


def test_cross_entropy_past_32_bit_offsets(lib):
    T, H, V = 3, 4096, 600_000               # a head of 2.4e9 elements
    g = torch.Generator(device=DEV).manual_seed(9)
    w = torch.empty(V, H, dtype=BF, device=DEV)
    for i in range(0, V, 60_000):
        w[i:i + 60_000] = (torch.randn(60_000, H, device=DEV, generator=g) * 0.02).to(BF)
    x = torch.randn(T, H, device=DEV, generator=g).to(BF)
    lab = torch.tensor([V - 1, 0, 555_555], dtype=torch.int32, device=DEV)
    z = torch.cat([x.double() @ w[i:i + 60_000].double().T for i in range(0, V, 60_000)], 1)
    ref = torch.logsumexp(z, 1)
    loss, lse = _nan(T, dtype=torch.float32), _nan(T, dtype=torch.float32)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V))
    api.moe_cross_entropy_forward(x, w, lab, loss, lse, ws)
    want = ref - z[torch.arange(T, device=DEV), lab.long()]
    assert (lse.double() - ref).abs().max() < 1e-3 and (loss.double() - want).abs().max() < 2e-3
    dx, dw = _nan(T, H), _nan(V, H)
    api.moe_cross_entropy_backward(x, w, lab, lse, torch.ones(T, device=DEV), dx, dw, ws)
    d = torch.exp(z - ref[:, None])
    d[torch.arange(T, device=DEV), lab.long()] -= 1.0
    rows = torch.tensor([0, 1, 299_999, 555_555, V - 257, V - 1], device=DEV)
    wd = d[:, rows].T @ x.double()
    assert torch.linalg.norm(dw[rows].double() - wd) <= 4e-3 * torch.linalg.norm(wd)
    wx = sum(d[:, i:i + 60_000] @ w[i:i + 60_000].double() for i in range(0, V, 60_000))
    assert torch.linalg.norm(dx.double() - wx) <= 4e-3 * torch.linalg.norm(wx)
    assert api.moe_read_device_status(ws) == 0


# ------------------------------------------------------------------- together
def test_calls_run_on_the_given_stream_and_in_a_graph(lib):
    """A side stream that first waits for its inputs, then the same calls captured once and replayed on new
    inputs: equal to the calls made one by one."""
    T, H, V = 200, 256, 1003
    rng = np.random.default_rng(12)
    side = torch.cuda.Stream()
    ws = _ws(max(api.moe_embedding_workspace_bytes(T, V, H), api.moe_layer_norm_workspace_bytes(T, H),
                 api.moe_cross_entropy_workspace_bytes(T, H, V)))
    w, b = torch.ones(H, dtype=BF, device=DEV), torch.zeros(H, dtype=BF, device=DEV)
    buf = {k: torch.zeros(T, H, dtype=BF, device=DEV) for k in ("e", "y", "dy", "de")}
    vec = {k: torch.zeros(T, dtype=torch.float32, device=DEV) for k in ("mean", "rstd", "loss", "lse")}
    dw, dn, dt = (torch.zeros(V, H, dtype=BF, device=DEV), torch.zeros(2, H, device=DEV), torch.zeros(V, H, device=DEV))
    table, tok = torch.zeros(V, H, dtype=BF, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    dl = torch.full((T,), 1.0 / T, device=DEV)

    def step(stream=None):
        api.moe_embedding_forward(tok, table, buf["e"], ws, scale=4.0, stream=stream)
        api.moe_layer_norm_forward(buf["e"], w, b, buf["y"], vec["mean"], vec["rstd"], stream=stream)
        api.moe_cross_entropy_forward(buf["y"], table, tok, vec["loss"], vec["lse"], ws, stream=stream)
        api.moe_cross_entropy_backward(buf["y"], table, tok, vec["lse"], dl, buf["dy"], dw, ws, piece=256, stream=stream)
        api.moe_layer_norm_backward(buf["dy"], buf["e"], w, vec["mean"], vec["rstd"], buf["de"], dn[0], dn[1], ws,
                                    stream=stream)
        api.moe_embedding_backward(tok, buf["de"], dt, ws, scale=4.0, base=dw, stream=stream)

    def outputs():
        return [t.clone() for t in (*buf.values(), *vec.values(), dw, dn, dt)]

    def fill(seed):
        r = np.random.default_rng(seed)
        table.copy_(_bf(r, V, H, std=0.3).to(DEV))
        tok.copy_(torch.from_numpy(r.integers(0, V, T).astype(np.int32)).to(DEV))

    wanted = {}
    for seed in (1, 2):
        fill(seed)
        step()
        torch.cuda.synchronize()
        wanted[seed] = outputs()
    fill(1)
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outputs(), wanted[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 1):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outputs(), wanted[seed]))
    assert api.moe_read_device_status(ws) == 0
