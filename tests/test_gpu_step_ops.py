"""Rotary positions, the router's balance loss, the gradient norm and clipping, against the fp64 forms.

Bounds: U = 2^-24 is half a step of fp32, B = 2^-8 of bf16, both relative to the value.
"""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import f64
from moe_expert_layer_05_gb300 import api
from oracle import model_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, B = 2.0 ** -24, 2.0 ** -8


def _within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        pytest.fail(f"{what}: {bad.sum()} of {bad.size}, worst {np.max((np.abs(got - ref) / (tol + 1e-300)))} of the bound")


def _ws(nbytes):
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV).fill_(255)
    api.moe_workspace_init(ws[:256])
    return ws


# --------------------------------------------------------------------- rotary
def _rotary_check(x, pos, freq, got, interleaved, scale, inverse):
    """A turned value: two products and their sum (3 U), sine and cosine from an angle of 2^-24 turns (2 pi 2^-24
    + 2^-25 for its fp32 form and 2 U of their own, say 12 U), all relative to |a| + |b| at most; then bf16."""
    ref = M.rotary(f64(x), pos, freq, interleaved, scale, inverse)
    n = len(freq)
    mag = np.abs(f64(x))
    a, b = (mag[..., 0:2 * n:2], mag[..., 1:2 * n:2]) if interleaved else (mag[..., :n], mag[..., n:2 * n])
    tol = np.zeros(ref.shape)
    s = 16 * U * scale * (a + b)
    if interleaved:
        tol[..., 0:2 * n:2], tol[..., 1:2 * n:2] = s, s
    else:
        tol[..., :n], tol[..., n:2 * n] = s, s
    tol[..., :2 * n] += B * np.abs(ref[..., :2 * n])
    _within(f64(got), ref, tol, "rotary")


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,width,R", [(1, 1, 16, 16), (1, 40, 128, 128), (5, 3, 40, 32), (131, 5, 72, 48),
                                             (64, 2, 512, 512), (9, 33, 24, 16)])
def test_rotary(lib, T, heads, width, R, interleaved, inverse):
    rng = np.random.default_rng(T + width)
    x = torch.from_numpy(rng.standard_normal((T, heads, width)).astype(np.float32)).to(torch.bfloat16)
    pos = rng.integers(-50, 200000, T).astype(np.int32)
    freq, scale = api.moe_rotary_frequencies(R)
    out = torch.zeros(T, heads, width, dtype=torch.bfloat16, device=DEV)
    xd, pd = x.to(DEV), torch.from_numpy(pos).to(DEV)
    api.moe_rotary(xd, pd, freq, out, interleaved=interleaved, scale=1.25, inverse=inverse)
    _rotary_check(x, pos, freq.cpu().numpy(), out, interleaved, 1.25, inverse)
    api.moe_rotary(xd, pd, freq, xd, interleaved=interleaved, scale=1.25, inverse=inverse)     # in place
    assert torch.equal(xd, out)


def test_rotary_of_parts_of_one_buffer(lib):
    """Queries and keys turned where they lie; the values between and behind them stay as they are."""
    rng = np.random.default_rng(3)
    whole = torch.from_numpy(rng.standard_normal((77, 9, 64)).astype(np.float32)).to(torch.bfloat16)
    pos = rng.permutation(77).astype(np.int32)
    freq, _ = api.moe_rotary_frequencies(32, base=500.0)
    d = whole.to(DEV)
    pd = torch.from_numpy(pos).to(DEV)
    api.moe_rotary(d[:, 2:7], pd, freq, d[:, 2:7])
    assert torch.equal(d[:, :2].cpu(), whole[:, :2]) and torch.equal(d[:, 7:].cpu(), whole[:, 7:])
    _rotary_check(whole[:, 2:7], pos, freq.cpu().numpy(), d[:, 2:7], False, 1.0, False)
    out = torch.zeros(5, 77, 64, dtype=torch.bfloat16, device=DEV).transpose(0, 1)              # heads first
    api.moe_rotary(whole.to(DEV)[:, 2:7], pd, freq, out)
    assert torch.equal(out, d[:, 2:7])


def test_rotary_far_positions_and_fast_pairs(lib):
    pos = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 1000003, 16777217], np.int32)
    freq = np.array([1.0, 1e-9, 3.0, 7.5, 100.25, -0.3, 2 * math.pi, 0.0])
    x = torch.ones(8, 1, 16, dtype=torch.bfloat16)
    out = torch.zeros(8, 1, 16, dtype=torch.bfloat16, device=DEV)
    api.moe_rotary(x.to(DEV), torch.from_numpy(pos).to(DEV), torch.from_numpy(freq).to(DEV), out)
    # exact angles: position times the fp64 frequency, in whole numbers
    from fractions import Fraction
    ref = np.zeros((8, 1, 16))
    two_pi = Fraction(31415926535897932384626433832795028841971, 5 * 10 ** 39)
    for t in range(8):
        for i in range(8):
            turn = Fraction(int(pos[t])) * Fraction(float(freq[i])) / two_pi
            a = float((turn - math.floor(turn)) * two_pi)
            ref[t, 0, i], ref[t, 0, i + 8] = math.cos(a) - math.sin(a), math.cos(a) + math.sin(a)
    # the frequency in turns is rounded to fp64 (2^-53 of it): 2^31 * 100 / 2 pi * 2^-53 turns at the fastest pair
    _within(f64(out), ref, B * np.abs(ref) + 2 * (16 * U + 2 ** 31 * np.abs(np.tile(freq, 2)) * 2.0 ** -52), "far")


def test_rotary_gradient_is_the_transpose(lib):
    """<rotate(x), y> = <x, rotate back(y)>, and differences of the fp64 form along a direction."""
    rng = np.random.default_rng(7)
    x, y = (torch.from_numpy(rng.standard_normal((50, 4, 32)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    pos = rng.integers(0, 9000, 50).astype(np.int32)
    freq, _ = api.moe_rotary_frequencies(32)
    pd, out = torch.from_numpy(pos).to(DEV), torch.zeros(50, 4, 32, dtype=torch.bfloat16, device=DEV)
    api.moe_rotary(y.to(DEV), pd, freq, out, inverse=True, scale=1.1)
    fn = freq.cpu().numpy()
    d = rng.standard_normal(x.shape)
    num = ((M.rotary(f64(x) + d, pos, fn, scale=1.1) - M.rotary(f64(x) - d, pos, fn, scale=1.1)) / 2 * f64(y)).sum()
    assert abs((f64(out) * d).sum() - num) <= B * np.abs(f64(out) * d).sum()


def test_rotary_frequencies(lib):
    for R in (16, 64, 128):
        f, s = api.moe_rotary_frequencies(R, base=10000.0)
        _within(f.cpu(), 10000.0 ** (-np.arange(0, R, 2) / R), 1e-14 * f.cpu().numpy(), "plain")
        g, _ = api.moe_rotary_frequencies(R, scaling="linear", factor=4.0)
        _within(g.cpu(), f.cpu().numpy() / 4, 1e-15, "linear")
    f, s = api.moe_rotary_frequencies(64, base=500000.0, scaling="by_parts", factor=32.0, original_length=4096)
    plain = 500000.0 ** (-np.arange(0, 64, 2) / 64)
    turns = 4096 * plain / (2 * math.pi)
    f = f.cpu().numpy()
    assert abs(s - (0.1 * math.log(32) + 1)) < 1e-6
    np.testing.assert_allclose(f[turns > 40], plain[turns > 40], rtol=1e-12)
    np.testing.assert_allclose(f[turns < 0.7], plain[turns < 0.7] / 32, rtol=1e-12)
    between = (turns < 20) & (turns > 2)
    assert ((f < plain) & (f > plain / 32))[between].all() and (np.diff(f) < 0).all()


# --------------------------------------------------------------- balance loss
def _balance_run(logits, topk, tokens, sigmoid, dloss=0.37):
    T, E = logits.shape
    score = "sigmoid" if sigmoid else "softmax"
    ld, td = torch.from_numpy(logits).to(DEV), torch.from_numpy(topk).to(DEV)
    tok = None if tokens is None else torch.from_numpy(tokens).to(DEV)
    loss, slope = torch.full((1,), 9.0, device=DEV), torch.full((E,), 9.0, device=DEV)
    counts = torch.full((E,), 9, dtype=torch.int32, device=DEV)
    d = torch.full((T, E), 9.0, device=DEV)
    ws = _ws(api.moe_balance_loss_workspace_bytes(T, E))
    api.moe_balance_loss_forward(ld, td, loss, counts, slope, ws, tokens=tok, score=score)
    api.moe_balance_loss_backward(ld, slope, torch.full((1,), dloss, device=DEV), d, tokens=tok, score=score)
    return loss, counts, slope, d, ws


def _balance_check(logits, topk, tokens, sigmoid, dloss=0.37):
    loss, counts, slope, d, ws = _balance_run(logits, topk, tokens, sigmoid, dloss)
    ref = M.balance_loss(logits.astype(np.float64), topk, topk.shape[1], tokens, sigmoid)
    assert api.moe_read_device_status(ws) == 0
    np.testing.assert_array_equal(counts.cpu().numpy(), ref["counts"])
    _within(slope.cpu(), ref["slope"], 2 * U * ref["slope"], "slope")
    # a probability: the exponent's difference is exact or rounded by U of the logits' spread, exp 2 U, the sum of E
    # terms in a tree and over lanes, a quotient; then sums over the rows (all of one sign)
    T, E = logits.shape
    fin = np.where(np.isfinite(logits), logits, 0.0)
    spread = np.abs(fin).max(initial=0.0) * 2
    rel = (spread + E / 8 + 24) * U
    _within(loss.cpu(), [ref["loss"]], (rel + (T / 100 + 64) * U) * ref["loss"], "loss")
    g = np.float32(dloss).astype(np.float64)
    _within(d.cpu(), g * ref["grad"], g * (3 * rel + 8 * U) * ref["grad_mag"] + 1e-37, "dlogits")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (257, 16, 2), (100, 17, 3), (1003, 64, 6),
                                   (515, 100, 8), (2000, 129, 32), (4099, 256, 8)])
def test_balance_loss(lib, T, E, k, sigmoid):
    rng = np.random.default_rng(T + E)
    logits = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32)
    topk = np.argsort(-logits, 1)[:, :k].astype(np.int32).copy()
    _balance_check(logits, topk, None, sigmoid)
    tokens = rng.integers(-1, 4, T).astype(np.int32)
    _balance_check(logits, topk, tokens, sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_rows_that_do_not_count_may_hold_anything(lib, sigmoid):
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((40, 24)).astype(np.float32)
    topk = np.argsort(-logits, 1)[:, :4].astype(np.int32).copy()
    tokens = np.zeros(40, np.int32)
    tokens[[0, 7, 39]] = -1
    logits[0], logits[7], logits[39] = np.nan, np.inf, -np.inf
    topk[[0, 7]] = 2 ** 30
    _balance_check(logits, topk, tokens, sigmoid)
    tokens[:] = -1                                    # none counts
    loss, counts, slope, d, ws = _balance_run(logits, topk, tokens, sigmoid)
    for t in (loss, counts, slope, d):
        assert not t.any()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_masked_experts_and_extreme_logits(lib, sigmoid):
    rng = np.random.default_rng(6)
    logits = rng.standard_normal((64, 40)).astype(np.float32)
    logits[:, 30:] = -np.inf                          # experts that are out of use
    logits[3] = -np.inf                               # a row that may choose nothing
    logits[4] -= 200.0                                # sigmoids with no fp32 value
    logits[5] += 300.0
    logits[6, :20] -= 500.0
    topk = np.argsort(-logits, 1, kind="stable")[:, :2].astype(np.int32).copy()
    _balance_check(logits, topk, None, sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [5, 8, 24, 64, 100, 129, 160, 256])
def test_balance_rows_of_nan_are_seen_in_the_loss(lib, E, sigmoid):
    """A token whose activations are NaN has a row of nothing else, or of NaN beside experts that are out of use."""
    rng = np.random.default_rng(E)
    logits = rng.standard_normal((70, E)).astype(np.float32)
    topk = np.argsort(-logits, 1)[:, :2].astype(np.int32).copy()
    for row, lost in ((3, slice(None)), (40, slice(0, E // 2)), (69, slice(E - 1, E))):
        x = logits.copy()
        x[row] = -np.inf
        x[row, lost] = np.nan
        loss, counts, slope, d, ws = _balance_run(x, topk, None, sigmoid, dloss=1.0)
        with np.errstate(invalid="ignore"):
            ref = M.balance_loss(x.astype(np.float64), topk, 2, None, sigmoid)
        assert math.isnan(ref["loss"]) and math.isnan(float(loss)) and api.moe_read_device_status(ws) == 0
        np.testing.assert_array_equal(counts.cpu().numpy(), ref["counts"])
        d, others = f64(d), np.arange(70) != row
        assert np.isnan(d[row]).all()
        rel = (2 * np.abs(logits).max() + E / 8 + 24) * U
        _within(d[others], ref["grad"][others], ((3 * rel + 8 * U) * ref["grad_mag"] + 1e-37)[others], "dlogits")


def test_balance_of_an_even_router_is_one(lib):
    E, k = 16, 4
    logits = np.zeros((32, E), np.float32)
    topk = np.array([[(t * k + i) % E for i in range(k)] for t in range(32)], np.int32)
    loss, counts, slope, d, _ = _balance_run(logits, topk, None, False)
    assert float(loss) == 1.0 and (counts == 8).all() and float(d.abs().max()) <= 1e-9


def test_balance_bad_choice_is_reported_and_not_counted(lib):
    rng = np.random.default_rng(8)
    logits = rng.standard_normal((30, 12)).astype(np.float32)
    topk = np.argsort(-logits, 1)[:, :3].astype(np.int32).copy()
    topk[4, 1], topk[9, 2] = 12, -1
    _, counts, _, _, ws = _balance_run(logits, topk, None, False)
    assert api.moe_read_device_status(ws) == -5
    np.testing.assert_array_equal(counts.cpu().numpy(), M.balance_loss(logits.astype(np.float64), topk, 3)["counts"])


def test_balance_gradient_against_differences(lib):
    rng = np.random.default_rng(9)
    for sigmoid in (False, True):
        logits = rng.standard_normal((20, 10)).astype(np.float32)
        topk = np.argsort(-logits, 1)[:, :2].astype(np.int32).copy()
        _, _, _, d, _ = _balance_run(logits, topk, None, sigmoid, dloss=1.0)
        x, v, h = logits.astype(np.float64), rng.standard_normal((20, 10)), 1e-5
        num = (M.balance_loss(x + h * v, topk, 2, None, sigmoid)["loss"]
               - M.balance_loss(x - h * v, topk, 2, None, sigmoid)["loss"]) / (2 * h)
        assert abs(num - (f64(d) * v).sum()) <= 1e-6


def test_balance_same_bits_on_every_run_and_with_the_router(lib):
    """The router's own logits and choices; the calls again, on another stream."""
    T, H, E, k = 700, 128, 32, 4
    cfg = api.make_config(T, H, E, k, 128)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, wr = (torch.randn(n, H, device=DEV, generator=gen).to(torch.bfloat16) for n in (T, E))
    logits, idx = torch.zeros(T, E, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    gate, ws = torch.zeros(T, k, device=DEV), _ws(api.moe_workspace_bytes(cfg))
    api.moe_router_topk(cfg, x, wr, None, logits, idx, gate, ws)
    l, t = logits.cpu().numpy(), idx.cpu().numpy()
    _balance_check(l, t, None, False)
    a = _balance_run(l, t, None, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _balance_run(l, t, None, False)
    torch.cuda.synchronize()
    for p, q in zip(a[:4], b[:4]):
        assert torch.equal(p, q)


# -------------------------------------------------------------- gradient norm
def _grads(rng, sizes, scale=1.0):
    out = []
    for i, n in enumerate(sizes):
        t = torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32))
        out.append(t.to(torch.bfloat16) if i % 2 else t)
    return out


def _clip_check(grads, limit, in_place=False):
    d = [g.to(DEV) for g in grads]
    norm, ws = torch.full((1,), 9.0, device=DEV), _ws(api.moe_grad_norm_workspace_bytes(len(d)))
    api.moe_grad_norm(d, norm, ws)
    outs = None if in_place else [torch.full_like(g, 9.0) for g in d]
    api.moe_grad_clip(d, norm, limit, outs=outs)
    got = d if in_place else outs
    want, ref = M.clip([f64(g) for g in grads], limit)
    # squares and their sums in fp32 over 32 or 64 values, fp64 from there, one rounding of the root
    if want > (2 - 2.0 ** -24) * 2.0 ** 127:
        # 5000 values of 1e37 have a norm of 7e38: the nearest fp32 value is infinity, and the factor 0
        assert math.isinf(float(norm)) and not any(t.any() for t in got)
        return got
    assert abs(float(norm) - want) <= 24 * U * want
    for g, r, src in zip(got, ref, grads):
        half = B if src.dtype is torch.bfloat16 else U
        _within(f64(g), r, (half + 30 * U) * np.abs(r) + 2.0 ** -149 * (2.0 ** 16 if half == B else 1), "clipped")
    assert api.moe_read_device_status(ws) == 0
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sizes", [[1], [3, 0, 5, 7], [8191, 8192, 8193, 16385], [70001] * 5, [9] * 64, [9] * 65,
                                   [33] * 1100, [3_000_001, 2_000_003]])
def test_clip(lib, sizes, in_place):
    rng = np.random.default_rng(len(sizes))
    grads = _grads(rng, sizes)
    _clip_check(grads, 0.5, in_place)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(_clip_check(grads, 1e9, in_place), grads))   # below the limit


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-15, 1e15, 1e25, 1e37])
def test_norm_of_values_whose_squares_have_no_fp32(lib, scale):
    rng = np.random.default_rng(1)
    _clip_check(_grads(rng, [5001, 64, 9]), 1.0 if scale > 1 else 1e-30)
    mixed = _grads(rng, [5001, 64, 9], scale) + _grads(rng, [777], 1.0)
    _clip_check(mixed, 0.1)
    _clip_check(_grads(rng, [5001, 64, 9], scale), 3.0)


def test_no_gradients_zeros_and_not_finite(lib):
    norm, ws = torch.full((1,), 9.0, device=DEV), _ws(api.moe_grad_norm_workspace_bytes(0))
    api.moe_grad_norm([], norm, ws)
    api.moe_grad_clip([], norm, 1.0)
    assert float(norm) == 0.0
    z = [torch.zeros(1000, device=DEV), torch.zeros(0, device=DEV), torch.zeros(17, device=DEV, dtype=torch.bfloat16)]
    api.moe_grad_norm(z, norm, ws := _ws(api.moe_grad_norm_workspace_bytes(3)))
    api.moe_grad_clip(z, norm, 0.0)
    assert float(norm) == 0.0 and not any(t.any() for t in z)
    for bad, what in ((float("inf"), torch.isinf), (float("nan"), torch.isnan)):
        g = [torch.ones(100, device=DEV), torch.ones(50, device=DEV, dtype=torch.bfloat16)]
        g[1][7] = bad
        api.moe_grad_norm(g, norm, ws)
        assert bool(what(norm).all())
        api.moe_grad_clip(g, norm, 1.0)
        assert torch.isnan(g[1][7]) and bool(((g[0] == 0) if math.isinf(bad) else torch.isnan(g[0])).all())


@pytest.mark.parametrize("in_place", [False, True])
def test_no_limit_leaves_every_gradient(lib, in_place):
    """An infinite limit: the factor is 1 with a finite norm, with one past fp32's range and with an infinite value."""
    rng = np.random.default_rng(14)
    norm = torch.zeros(1, device=DEV)
    for scale, bad in ((1.0, None), (3e37, None), (1.0, math.inf), (1.0, math.nan)):
        grads = _grads(rng, [5001, 64, 9], scale)
        if bad is not None:
            grads[1][5] = bad
        d = [g.to(DEV) for g in grads]
        api.moe_grad_norm(d, norm, _ws(api.moe_grad_norm_workspace_bytes(3)))
        assert math.isfinite(float(norm)) == (scale == 1.0 and bad is None)
        outs = d if in_place else [torch.full_like(g, 9.0) for g in d]
        api.moe_grad_clip(d, norm, math.inf, outs=None if in_place else outs)
        for got, g in zip(outs, grads):
            assert torch.isnan(got).all() if bad is math.nan else torch.equal(got.cpu(), g)


def test_clip_in_a_graph_that_is_replayed(lib):
    rng = np.random.default_rng(4)
    g = [t.to(DEV) for t in _grads(rng, [5000, 333, 70000])]
    norm, ws = torch.zeros(1, device=DEV), _ws(api.moe_grad_norm_workspace_bytes(3))
    outs = [torch.zeros_like(t) for t in g]

    def step():
        api.moe_grad_norm(g, norm, ws)
        api.moe_grad_clip(g, norm, 1.0, outs=outs)

    step()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in g:
        t.mul_(4.0)
    graph.replay()
    graph.replay()
    for a, b in zip(outs, want):                      # four times the gradients, the same direction and length
        _within(f64(a), f64(b), (2 * B if a.dtype is torch.bfloat16 else 1e-5) * np.abs(f64(b)), "replayed")
