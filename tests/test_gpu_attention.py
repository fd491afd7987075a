"""Causal attention over packed sequences and its gradient against the fp64 form.

Bounds, from the roundings that the kernels make (U = 2^-24 in fp32, B = 2^-8 in
bf16): a score is off by the additions of its D products, (D + 8) U of the sum of
their magnitudes, and by two units of the exponential and its argument; p by that,
relatively, and lse absolutely.  out: p rounded to bf16 and its own rounding.  Gradients:
p and ds rounded to bf16, delta from an out that was rounded, their own rounding.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import f64
from moe_expert_layer_05_gb300 import api
from oracle import model_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, B = 2.0 ** -24, 2.0 ** -8
FILL = 7.0                       # what outputs hold before the call


def _bf(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)


def _ws(T, Hq, Hkv, D):
    ws = torch.empty(api.moe_attention_workspace_bytes(T, Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    ws.fill_(255)                # scratch of any content
    api.moe_workspace_init(ws[:256])
    return ws


def _case(lengths, Hq, Hkv, D, seed=0, first=0, tail=0, std=1.0, layout="fused"):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32) + first
    T = int(cu[-1]) + tail
    q, k, v, do = (_bf(rng, T, h, D, std=std) for h in (Hq, Hkv, Hkv, Hq))
    return cu, T, q, k, v, do


def _place(parts, layout):
    """The tensors on the GPU: parts of one buffer, each [heads, T, D] turned round, or dense."""
    if layout == "fused":
        whole = torch.cat(parts, 1).to(DEV)
        out, at = [], 0
        for t in parts:
            out.append(whole[:, at:at + t.shape[1]])
            at += t.shape[1]
        return out
    if layout == "heads_first":
        return [t.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for t in parts]
    return [t.to(DEV) for t in parts]


def _run(cu, T, q, k, v, do, scale=None, layout="fused"):
    Hq, Hkv, D = q.shape[1], k.shape[1], q.shape[2]
    qd, kd, vd = _place([q, k, v], layout)
    cud = torch.from_numpy(cu).to(DEV)
    out, dod = _place([torch.full(q.shape, FILL, dtype=torch.bfloat16), do], layout)
    lse = torch.full((Hq, T), FILL, device=DEV)
    ws = _ws(T, Hq, Hkv, D)
    api.moe_attention_forward(qd, kd, vd, cud, out, lse, ws, scale=scale)
    dq, dk, dv = _place([torch.full(t.shape, FILL, dtype=torch.bfloat16) for t in (q, k, v)], layout)
    api.moe_attention_backward(qd, kd, vd, cud, out, lse, dod, dq, dk, dv, ws, scale=scale)
    assert api.moe_read_device_status(ws) == 0
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def _check(got, cu, T, q, k, v, do, scale=None):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    f = M.attention_grad(f64(q), f64(k), f64(v), cu, scale, f64(do))
    rows = np.zeros(T, bool)
    for a, b in zip(cu, cu[1:]):
        rows[a:b] = True
    # a score's error; the argument's roundings count by the size of the scores, 3 of them
    eps = (D + 12) * U * f["s_mag"] + (np.diff(cu).max(initial=0) + 32) * U              # [Hq, T]
    e_row = eps.T[:, :, None]
    e_all = float(eps.max(initial=0.0))
    x = {m: f64(t) for m, t in got.items()}
    def within(a, ref, tol, what):
        bad = ~(np.abs(a - ref) <= tol)
        if bad.any():
            pytest.fail(f"{what}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(a - ref) / tol)} of the bound")
    within(x["lse"][:, rows], f["lse"][:, rows], (eps + 8 * U * np.abs(f["lse"]) + 4 * U)[:, rows], "lse")
    within(x["out"][rows], f["out"][rows], (B * np.abs(f["out"]) + 1.01 * (B + 2 * e_row) * f["out_mag"] + 1e-30)[rows], "out")
    for g in ("dq", "dk", "dv"):
        tol = B * np.abs(f[g]) + 1.02 * (B + 3 * e_all + (D + 8) * U) * f[g + "_mag"] + 1e-30
        if g != "dv":
            tol += 1.02 * (2 * B + 3 * e_all) * f[g + "_delta"]
        within(x[g][rows], f[g][rows], tol[rows], g)
        # And as a whole, roundings of random sign: the result's and the terms', 1.2 B together.  delta: each of the
        # products dout out in it is off by out's rounding, at most B / sqrt(3) (root of the mean square),
        # independently; a row's delta moves dq by scale sum_j p k and dk by scale p q.  Where a row's softmax is
        # sharp, dp - delta is a small difference and this is the larger part.
        norm = np.linalg.norm(f[g][rows])
        if norm > 0 and rows.sum() > 64:
            moved = B / 3 ** 0.5 * np.sqrt(f[g + "_delta_sq"][rows].sum()) if g != "dv" else 0.0
            off = np.linalg.norm(x[g][rows] - f[g][rows])
            if not off <= 1.2 * (B * norm + moved):
                pytest.fail(f"{g}: {off / norm} off as a whole (delta's part {moved / norm})")
    for m in ("out", "dq", "dk", "dv"):
        assert (x[m][~rows] == FILL).all(), m
    assert (x["lse"][:, ~rows] == FILL).all()


@pytest.mark.parametrize("D", [8, 40, 64, 80, 128])
@pytest.mark.parametrize("lengths", [[1], [2], [127], [128], [129], [300], [517]])
def test_one_sequence(lib, lengths, D):
    c = _case(lengths, 4, 2, D, seed=D + lengths[0])
    _check(_run(*c), *c)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 4), (6, 2), (8, 1), (10, 2)])
@pytest.mark.parametrize("lengths,first,tail", [([5, 0, 130, 1, 1, 64, 300], 0, 3), ([40] * 9, 0, 0), ([1] * 140, 2, 9),
                                                ([255, 1, 0, 0, 200], 131, 260), ([384], 0, 1)])
def test_packed(lib, lengths, first, tail, Hq, Hkv):
    c = _case(lengths, Hq, Hkv, 64, seed=Hq, first=first, tail=tail)
    _check(_run(*c), *c)


@pytest.mark.parametrize("layout", ["fused", "heads_first", "dense"])
@pytest.mark.parametrize("D", [64, 128])
def test_layouts(lib, layout, D):
    c = _case([200, 77], 4, 2, D, seed=3, tail=5)
    _check(_run(*c, layout=layout), *c)


@pytest.mark.parametrize("std,scale", [(4.0, None), (0.01, None), (1.0, 1.0), (1.0, 1e-3)])
def test_sharp_and_flat_scores(lib, std, scale):
    """Scores of some hundreds (a softmax of one key) and of nothing."""
    c = _case([150, 260], 4, 2, 64, seed=5, std=std)
    _check(_run(*c, scale=scale), *c, scale=scale)


def test_maximum_that_keeps_growing(lib):
    """Keys whose scores rise away from the diagonal, so that the reference moves at every tile."""
    cu, T, q, k, v, do = _case([640], 2, 1, 64, seed=9)
    q[:] = q.abs()
    k[:] = (k.abs().float() * torch.linspace(8, 0.1, T)[:, None, None]).to(torch.bfloat16)
    _check(_run(cu, T, q, k, v, do), cu, T, q, k, v, do)


def test_longer_rows_and_repeated_calls(lib):
    c = _case([1500, 3, 700], 4, 2, 128, seed=11, tail=7)
    a = _run(*c)
    _check(a, *c)
    b = _run(*c)
    for n in a:
        assert torch.equal(a[n], b[n]), n


# ---------------------------------------------------------------- values that are not finite
def _plain_where_finite(c, bad_rows, tensors):
    """Outputs with `bad_rows` of the named inputs NaN or infinite, and the same inputs with zeros there."""
    cu, T, q, k, v, do = c
    parts = dict(q=q, k=k, v=v, do=do)
    dirty, clean = {n: t.clone() for n, t in parts.items()}, {n: t.clone() for n, t in parts.items()}
    for i, r in enumerate(bad_rows):
        for n in tensors:
            dirty[n][r, :, i % 3::3] = (float("nan"), float("inf"), -float("inf"))[i % 3]
            clean[n][r, :, i % 3::3] = 0
    return _run(cu, T, *dirty.values()), _run(cu, T, *clean.values())


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
def test_rows_of_no_sequence_may_hold_anything(lib, Hq, Hkv):
    c = _case([100, 61], Hq, Hkv, 64, seed=21, first=40, tail=70)
    a, b = _plain_where_finite(c, [0, 39, 201, 202, 260], ["q", "k", "v", "do"])
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("tensors", [["q"], ["k"], ["v"], ["do"]])
def test_not_finite_rows_reach_what_sees_them_and_no_other(lib, tensors, Hq, Hkv):
    """Sequences [0, 150), [150, 290), [290, 700); row 200 of the second and 433 of the third are not finite."""
    cu, T, *_ = c = _case([150, 140, 410], Hq, Hkv, 64, seed=23)
    bad = [200, 433]
    a, b = _plain_where_finite(c, bad, tensors)
    seq = np.searchsorted(cu, np.arange(T), side="right") - 1
    i, j = np.arange(T)[:, None], np.arange(T)[None]
    sees = (seq[i] == seq[j]) & (j <= i)
    spoilt = np.zeros(T, bool)
    spoilt[bad] = True
    on_rows = spoilt if tensors in (["q"], ["do"]) else (sees & spoilt[None]).any(1)     # rows whose own sums meet it
    forward = on_rows if tensors != ["do"] else np.zeros(T, bool)
    for n in ("out", "dq"):
        hit = forward if n == "out" else on_rows
        x, y = a[n].float().cpu().numpy(), b[n].float().cpu().numpy()
        assert (x[~hit] == y[~hit]).all(), (n, "clean rows")
        assert (~np.isfinite(x[hit])).any((1, 2)).all(), (n, "rows that see it")
    # keys seen by a spoilt row get it back in their gradients (every column of the group's sum)
    keys = (sees & on_rows[:, None]).any(0)
    for n in ("dk", "dv"):
        x, y = a[n].float().cpu().numpy(), b[n].float().cpu().numpy()
        assert (x[~keys] == y[~keys]).all(), (n, "clean keys")
        assert (~np.isfinite(x[keys])).any((1, 2)).all(), (n, "keys seen by it")


def test_out_has_the_column_that_is_not_finite(lib):
    cu, T, q, k, v, do = _case([300], 2, 1, 64, seed=25)
    v[170, 0, 5] = float("inf")
    v[171, 0, 9] = float("nan")
    x = _run(cu, T, q, k, v, do)["out"].float().cpu().numpy()
    bad = np.zeros(x.shape, bool)
    bad[170:, :, 5] = True
    bad[171:, :, 9] = True
    assert (np.isfinite(x) == ~bad).all()
    assert (x[170:200, :, 5] == np.inf).all()


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 64), (2, 2, 80), (300, 100, 64)])
def test_every_column_that_is_not_finite_is_given_back(lib, Hq, Hkv, D):
    """Infinities of both signs and NaN in the values, each in columns of its own, in masked tiles and others."""
    cu, T, q, k, v, do = _case([3, 497], Hq, Hkv, D, seed=27, std=0.5)
    want = np.zeros((T, D), np.float32)
    for row, col, y in ((0, 1, np.inf), (2, 2, -np.inf), (5, 3, np.inf), (5, 63, np.nan), (130, 9, -np.inf), (300, 9, np.inf),
                        (300, 8, -np.inf), (301, 10, np.nan), (400, 10, np.inf), (450, 16, np.nan), (499, D - 1, np.inf)):
        v[row, :, col] = y
        with np.errstate(invalid="ignore"):
            want[row:3 if row < 3 else T, col] += y
    x = _run(cu, T, q, k, v, do)["out"].float().cpu().numpy()
    for h in range(Hq):
        y = np.where(np.isfinite(x[:, h]), 0.0, x[:, h])
        assert np.array_equal(y, want, equal_nan=True), h


def test_values_of_nan_through_a_long_sequence(lib):
    """Every value NaN, in a sequence of 2^19 rows that begins inside a tile: each row gives up looking at the first key
    that it sees, and no wait of the launch runs into its limit."""
    T = 2 ** 19
    gen = torch.Generator(DEV).manual_seed(2)
    q, k = (torch.randn(T, 1, 64, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(2))
    v = torch.full_like(k, float("nan"))
    out, lse, ws = torch.zeros_like(q), torch.zeros(1, T, device=DEV), _ws(T, 1, 1, 64)
    cu = torch.tensor([5, T - 100], dtype=torch.int32, device=DEV)
    api.moe_attention_forward(q, k, v, cu, out, lse, ws)
    assert api.moe_read_device_status(ws) == 0
    assert torch.isnan(out[5:-100]).all() and not out[:5].any() and not out[-100:].any()
    assert torch.isfinite(lse[:, 5:-100]).all()


# ---------------------------------------------------------------- boundaries
@pytest.mark.parametrize("cu", [[0, 90, 60, 200], [-5, 100, 200], [0, 100, 900], [0, 2 ** 31 - 1, 200]])
def test_bad_boundaries_are_reported(lib, cu):
    """(every index made from them is kept inside [0, T]: row_map)"""
    T = 200
    rng = np.random.default_rng(1)
    q, k, v = (_bf(rng, T, h, 64).to(DEV) for h in (2, 1, 1))
    out, lse, ws = torch.zeros_like(q), torch.zeros(2, T, device=DEV), _ws(T, 2, 1, 64)
    api.moe_attention_forward(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), out, lse, ws)
    assert api.moe_read_device_status(ws) == -5


def test_no_rows_and_no_sequences(lib):
    ws = _ws(0, 2, 1, 64)
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(2, 0, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    api.moe_attention_forward(e, k, k, cu, e, lse, ws)
    api.moe_attention_backward(e, k, k, cu, e, lse, e, e, k, k, ws)
    q = torch.full((9, 2, 64), FILL, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, 9), FILL, device=DEV)
    ws = _ws(9, 2, 1, 64)
    for c in (cu[:1], cu):                       # no sequence, and two empty ones
        api.moe_attention_forward(q, q[:, :1], q[:, :1], c, q, lse, ws)
    assert (q == FILL).all() and (lse == FILL).all() and api.moe_read_device_status(ws) == 0


# ---------------------------------------------------------------- streams, graphs, bounded waits
def test_side_stream_and_graph_replay(lib):
    c = _case([130, 400, 1], 4, 2, 64, seed=31)
    want = _run(*c)
    cu, T, q, k, v, do = c
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    cud = torch.from_numpy(cu).to(DEV)
    got = {n: torch.zeros(t.shape, dtype=t.dtype, device=DEV) for n, t in want.items()}
    ws = _ws(T, 4, 2, 64)

    def both():
        api.moe_attention_forward(qd, kd, vd, cud, got["out"], got["lse"], ws)
        api.moe_attention_backward(qd, kd, vd, cud, got["out"], got["lse"], dod, got["dq"], got["dk"], got["dv"], ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in got.values():
        t.zero_()
    for _ in range(3):
        graph.replay()
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_wait_limit_gives_timeout_status_and_the_context_recovers(lib):
    """A limit of 1 ns that no wait can meet: the calls return, and the same context then computes correctly."""
    c = _case([900], 2, 1, 128, seed=33)
    cu, T, q, k, v, do = c
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    cud = torch.from_numpy(cu).to(DEV)
    out, lse, ws = torch.zeros_like(qd), torch.zeros(2, T, device=DEV), _ws(T, 2, 1, 128)
    dq, dk, dv = torch.zeros_like(qd), torch.zeros_like(kd), torch.zeros_like(vd)
    for backward in (False, True):
        api.moe_debug_set_wait_limit_ns(1)
        try:
            if backward:
                api.moe_attention_backward(qd, kd, vd, cud, out, lse, dod, dq, dk, dv, ws)
            else:
                api.moe_attention_forward(qd, kd, vd, cud, out, lse, ws)
            torch.cuda.synchronize()
        finally:
            api.moe_debug_set_wait_limit_ns(0)
        assert api.moe_read_device_status(ws) == -6
        api.moe_workspace_init(ws[:256])
    _check(_run(*c), *c)
