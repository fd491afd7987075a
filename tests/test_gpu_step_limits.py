"""The step operators at the edges of what they take: groups of every size, offsets past 32 bits, calls at once on
two streams, a captured step whose inputs change, the same expert twice in a row of choices."""
import math

import numpy as np
import pytest
import torch

from moe_expert_layer_05_gb300 import api
from test_gpu_attention import DEV, FILL, U, _case, _check, _run, _ws
from test_gpu_step_ops import _balance_check, _within
from test_gpu_step_ops import _ws as _scratch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(5, 1), (6, 1), (7, 1), (8, 1), (16, 1), (14, 2)])
def test_group_sizes(lib, Hq, Hkv, D):
    """Few keys, so that a group's heads are shared out among as many CTAs as its size allows."""
    c = _case([70, 1, 90], Hq, Hkv, D, seed=Hq, tail=3)
    _check(_run(*c), *c)


def test_scales_at_the_ends(lib):
    """2^-64: every key counts the same."""
    c = _case([150, 30], 4, 2, 64, seed=2)
    _check(_run(*c, scale=2.0 ** -64), *c, scale=2.0 ** -64)


def test_attention_offsets_past_32_bits(lib):
    """260 rows 2^23 + 8 elements apart: 2.18e9 elements from the first to the last."""
    c = _case([130, 126], 4, 2, 64, seed=8, tail=4)
    cu, T, q, k, v, do = c
    want = _run(*c)
    pitch = 2 ** 23 + 8
    buf = torch.empty(T * pitch, dtype=torch.bfloat16, device=DEV)
    at = 0

    def part(src):
        nonlocal at
        t = torch.as_strided(buf, src.shape, (pitch, src.shape[2], 1), at)
        at += src.shape[1] * src.shape[2]
        return t.copy_(src)

    qd, kd, vd, dod = (part(t) for t in (q, k, v, do))
    out, dq, dk, dv = (part(torch.full(t.shape, FILL, dtype=torch.bfloat16)) for t in (q, q, k, v))
    assert (T - 1) * pitch > 2 ** 31 and dv.data_ptr() - qd.data_ptr() > 0
    lse = torch.full((4, T), FILL, device=DEV)
    ws, cud = _ws(T, 4, 2, 64), torch.from_numpy(cu).to(DEV)
    api.moe_attention_forward(qd, kd, vd, cud, out, lse, ws)
    api.moe_attention_backward(qd, kd, vd, cud, out, lse, dod, dq, dk, dv, ws)
    got = dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    # heads that far apart, too
    far = torch.as_strided(buf, (T, 4, 64), (64, 2 ** 29 + 8, 1), 0).copy_(q)
    assert 3 * 2 ** 29 + T * 64 < buf.numel()
    out2 = torch.full(q.shape, FILL, dtype=torch.bfloat16, device=DEV)
    api.moe_attention_forward(far, k.to(DEV), v.to(DEV), cud, out2, lse, ws)
    assert torch.equal(out2, want["out"]) and api.moe_read_device_status(ws) == 0


def test_rotary_offsets_past_32_bits(lib):
    T, heads, width, pitch = 270, 3, 64, 2 ** 23 + 8
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((T, heads, width)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    pos = torch.from_numpy(rng.integers(0, 100000, T).astype(np.int32)).to(DEV)
    freq, _ = api.moe_rotary_frequencies(32)
    want = torch.empty_like(x)
    api.moe_rotary(x, pos, freq, want)
    buf = torch.empty(T * pitch, dtype=torch.bfloat16, device=DEV)
    src = torch.as_strided(buf, x.shape, (pitch, width, 1), 0).copy_(x)
    dst = torch.as_strided(buf, x.shape, (pitch, width, 1), heads * width)
    api.moe_rotary(src, pos, freq, dst)
    assert torch.equal(dst, want)
    api.moe_rotary(src, pos, freq, src)
    assert torch.equal(src, want)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_of_the_most_tokens(lib, sigmoid):
    """2^24 tokens of 160 experts, 2.7e9 logits: zeros but for the last 100 rows.

    Sums of 2^24 / (152 blocks * 32 rows) terms of one sign a lane and some forty more, each addition off by U."""
    T, E, last, rng = 1 << 24, 160, 100, np.random.default_rng(6)
    score = "sigmoid" if sigmoid else "softmax"
    tail = rng.standard_normal((last, E)).astype(np.float32)
    logits = torch.zeros(T, E, device=DEV)
    logits[-last:] = torch.from_numpy(tail).to(DEV)
    topk = torch.randint(0, E, (T, 1), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    topk[: T // 3] = 7
    loss, slope = torch.zeros(1, device=DEV), torch.zeros(E, device=DEV)
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    ws = _scratch(api.moe_balance_loss_workspace_bytes(T, E))
    api.moe_balance_loss_forward(logits, topk, loss, counts, slope, ws, score=score)
    want = torch.bincount(topk.view(-1), minlength=E).cpu().numpy()
    np.testing.assert_array_equal(counts.cpu().numpy(), want)
    w = E * want.astype(np.float64) / float(T) ** 2
    x = tail.astype(np.float64)
    p = 1 / (1 + np.exp(-x)) if sigmoid else np.exp(x)
    rest = 1 - p if sigmoid else 1.0
    p /= p.sum(1, keepdims=True)
    ref = (w * ((T - last) / E + p.sum(0))).sum()
    _within(loss.cpu(), [ref], (T / (152 * 32) + 100) * U * ref, "loss")
    d = torch.full((T, E), 9.0, device=DEV)
    one = torch.full((1,), float(T), device=DEV)
    api.moe_balance_loss_backward(logits, slope, one, d, score=score)
    dot = (p * w).sum(1, keepdims=True)
    rel = (2 * np.abs(tail).max() + E / 8 + 24) * U
    _within(d[-last:].cpu(), T * p * (w - dot) * rest, (3 * rel + 8 * U) * T * p * (w + dot), "dlogits")
    even = T / E * (w - w.mean()) * (0.5 if sigmoid else 1.0)
    rel = (E / 8 + 24) * U
    for row in (0, T // 2, T - last - 1):
        _within(d[row].cpu(), even, (3 * rel + 8 * U) * T / E * (w + w.mean()), "dlogits of an even row")


def test_norm_and_clip_past_32_bits(lib):
    """A tensor of 2^31 + 777 bf16 values, the last 777 of them ones; one of fp32 beside it."""
    n = 2 ** 31 + 777
    big = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    big[-777:] = 1
    small = torch.full((223,), 1.0, device=DEV)
    norm, ws = torch.zeros(1, device=DEV), _scratch(api.moe_grad_norm_workspace_bytes(2))
    api.moe_grad_norm([big, small], norm, ws)
    assert abs(float(norm) - 1000 ** 0.5) <= 24 * U * 1000 ** 0.5
    api.moe_grad_clip([big, small], norm, 1000 ** 0.5 / 4)
    assert (big[-777:] == 0.25).all() and not big[:-777].any()
    _within(small.cpu(), np.full(223, 0.25), 31 * U * 0.25, "clipped")


def test_the_same_expert_twice_in_a_row(lib):
    rng = np.random.default_rng(12)
    topk = rng.integers(0, 9, (300, 4)).astype(np.int32)
    topk[:50] = 3
    _balance_check(rng.standard_normal((300, 9)).astype(np.float32), topk, None, False)


def _step(seed):
    """One step's operators over tensors of their own: rotary, attention and its gradients, the balance loss, clipping."""
    cu, T, q, k, v, do = _case([300, 77, 140], 4, 2, 64, seed=seed)
    rng = np.random.default_rng(seed)
    s = dict(q=q.to(DEV), k=k.to(DEV), v=v.to(DEV), do=do.to(DEV), cu=torch.from_numpy(cu).to(DEV),
             logits=torch.from_numpy(rng.standard_normal((T, 16)).astype(np.float32)).to(DEV),
             topk=torch.from_numpy(rng.integers(0, 16, (T, 2)).astype(np.int32)).to(DEV),
             pos=torch.arange(T, dtype=torch.int32, device=DEV), freq=api.moe_rotary_frequencies(64)[0])
    for n in ("q", "k", "v"):
        s["d" + n] = torch.zeros_like(s[n])
    s.update(rq=torch.zeros_like(s["q"]), rk=torch.zeros_like(s["k"]), out=torch.zeros_like(s["q"]),
             lse=torch.zeros(4, T, device=DEV), loss=torch.zeros(1, device=DEV), slope=torch.zeros(16, device=DEV),
             counts=torch.zeros(16, dtype=torch.int32, device=DEV), dl=torch.zeros(T, 16, device=DEV),
             norm=torch.zeros(1, device=DEV), one=torch.ones(1, device=DEV), aws=_ws(T, 4, 2, 64),
             bws=_scratch(api.moe_balance_loss_workspace_bytes(T, 16)), nws=_scratch(api.moe_grad_norm_workspace_bytes(4)))

    def run():
        api.moe_rotary(s["q"], s["pos"], s["freq"], s["rq"])
        api.moe_rotary(s["k"], s["pos"], s["freq"], s["rk"])
        api.moe_attention_forward(s["rq"], s["rk"], s["v"], s["cu"], s["out"], s["lse"], s["aws"])
        api.moe_attention_backward(s["rq"], s["rk"], s["v"], s["cu"], s["out"], s["lse"], s["do"], s["dq"], s["dk"],
                                   s["dv"], s["aws"])
        api.moe_rotary(s["dq"], s["pos"], s["freq"], s["dq"], inverse=True)
        api.moe_rotary(s["dk"], s["pos"], s["freq"], s["dk"], inverse=True)
        api.moe_balance_loss_forward(s["logits"], s["topk"], s["loss"], s["counts"], s["slope"], s["bws"])
        api.moe_balance_loss_backward(s["logits"], s["slope"], s["one"], s["dl"])
        grads = [s["dq"], s["dk"], s["dv"], s["dl"]]
        api.moe_grad_norm(grads, s["norm"], s["nws"])
        api.moe_grad_clip(grads, s["norm"], 0.5)

    return s, run


OUT = ("out", "lse", "dq", "dk", "dv", "loss", "slope", "counts", "dl", "norm")


def _values(s):
    return {n: s[n].clone() for n in OUT}


def test_two_steps_at_once(lib):
    steps = [_step(41), _step(42)]
    want = []
    for s, run in steps:
        run()
        torch.cuda.synchronize()
        want.append(_values(s))
    streams = [torch.cuda.Stream() for _ in steps]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for (s, run), st in zip(steps, streams):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for (s, _), w in zip(steps, want):
        for n in OUT:
            assert torch.equal(s[n], w[n]), n
        assert not math.isnan(float(s["norm"]))


def test_a_captured_step_whose_inputs_change(lib):
    """Other values, other sequences (of the same number) and other choices in the tensors of a captured step."""
    s, run = _step(51)
    other, run_other = _step(52)
    other["cu"].copy_(torch.tensor([2, 2, 500, 510], dtype=torch.int32, device=DEV))
    run_other()
    want = _values(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    for n in ("q", "k", "v", "do", "cu", "logits", "topk"):
        s[n].copy_(other[n])
    for n in ("out", "lse", "dq", "dk", "dv"):
        s[n].zero_()                     # (rows of no sequence stay as they were)
    graph.replay()
    torch.cuda.synchronize()
    for n in OUT:
        assert torch.equal(s[n], want[n]), n
