"""Attention of more tiles than SMs: CTAs that work through several of them, some without rows."""
import numpy as np
import pytest
import torch

from moe_expert_layer_05_gb300 import api
from test_gpu_attention import DEV, _case, _check, _run, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(400, 400), (480, 160)])
def test_many_heads_of_few_rows(lib, Hq, Hkv, D):
    """Groups of odd sizes take 256 rows at a time: the second 128 have none, in every item of every CTA."""
    c = _case([60, 1, 39], Hq, Hkv, D, seed=Hq + D)
    _check(_run(*c), *c)


@pytest.mark.parametrize("Hq,Hkv", [(96, 96), (128, 64)])
def test_sequences_between_rows_of_none(lib, Hq, Hkv):
    """Tiles without a row before the first sequence and behind the last one, between those with rows."""
    c = _case([200, 1, 0, 70], Hq, Hkv, 64, seed=Hq, first=300, tail=400)
    _check(_run(*c), *c)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(16384, 8, 1, 64), (8192, 6, 2, 64), (8192, 8, 2, 128), (4100, 15, 5, 128)])
def test_many_launches_end_and_agree(lib, T, Hq, Hkv, D):
    """Launch after launch on one workspace: every wait ends, the bits are the same."""
    cu, T, q, k, v, do = _case([T - 3000, 1, 2500, 499], Hq, Hkv, D, seed=T)
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    cud, ws = torch.from_numpy(cu).to(DEV), _ws(T, Hq, Hkv, D)
    outs = [torch.zeros_like(qd) for _ in range(2)]
    lse = torch.zeros(Hq, T, device=DEV)
    grads = [[torch.zeros_like(t) for t in (qd, kd, vd)] for _ in range(2)]
    for i in range(60):
        api.moe_attention_forward(qd, kd, vd, cud, outs[i > 0], lse, ws)
        if i % 10 == 0:
            api.moe_attention_backward(qd, kd, vd, cud, outs[i > 0], lse, dod, *grads[i > 0], ws)
    assert api.moe_read_device_status(ws) == 0
    assert torch.equal(outs[0], outs[1])
    for a, b in zip(*grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 64), (32, 8, 128), (15, 5, 80)])
def test_a_limit_that_no_wait_can_meet_ends_the_launch(lib, Hq, Hkv, D):
    """CTAs with items left return all the same, and the next call on the workspace has them all again."""
    c = _case([3000, 1, 1100], Hq, Hkv, D, seed=3)
    cu, T, q, k, v, do = c
    want = _run(*c)
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    cud, ws = torch.from_numpy(cu).to(DEV), _ws(T, Hq, Hkv, D)
    got = {n: torch.zeros(t.shape, dtype=t.dtype, device=DEV) for n, t in want.items()}

    def forward():
        api.moe_attention_forward(qd, kd, vd, cud, got["out"], got["lse"], ws)

    def backward():
        api.moe_attention_backward(qd, kd, vd, cud, got["out"], got["lse"], dod, got["dq"], got["dk"], got["dv"], ws)

    for call in (forward, backward):
        api.moe_debug_set_wait_limit_ns(1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            api.moe_debug_set_wait_limit_ns(0)
        assert api.moe_read_device_status(ws) == -6
        ws[:4].zero_()               # (the status word alone: the counters have to be back at zero)
    forward()
    backward()
    assert api.moe_read_device_status(ws) == 0
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("lengths", [[0] * 100 + [5] + [0] * 1500 + [130] + [0] * 70 + [1] * 90 + [0] * 33 + [300, 0, 0],
                                     [3] * 200 + [0] * 31 + [150], [1] * 32, [2] * 31 + [200], [0] * 5000 + [140]])
def test_many_sequences_most_of_them_empty(lib, lengths, Hq, Hkv):
    c = _case(lengths, Hq, Hkv, 64, seed=len(lengths), first=3, tail=2)
    _check(_run(*c), *c)


@pytest.mark.parametrize("seed", range(6))
def test_many_bad_boundaries_are_reported(lib, seed):
    """Boundaries in any order, below 0 and far past the rows: reported, nothing outside the tensors touched."""
    rng = np.random.default_rng(seed)
    cu, T, q, k, v, do = _case([700], 3 + seed % 2, 1, 64, seed=seed)
    bad = rng.integers(-300, 1000, 200 + 500 * (seed % 3)).astype(np.int32)
    bad[rng.integers(0, len(bad), 9)] = [-2 ** 31, 2 ** 31 - 1, 700, 0, 701, -1, 128, 127, 2 ** 30]
    Hq = q.shape[1]
    guard = 64
    def placed(t):
        whole = torch.full((T + 2 * guard, *t.shape[1:]), 5.0, dtype=torch.bfloat16, device=DEV)
        whole[guard:guard + T] = t.to(DEV)
        return whole, whole[guard:guard + T]
    whole, out = placed(torch.zeros_like(q))
    grads = [placed(torch.zeros_like(t)) for t in (q, k, v)]
    lse = torch.full((Hq + 2, T), 5.0, device=DEV)
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    cud = torch.from_numpy(bad).to(DEV)
    for call in range(2):
        ws = _ws(T, Hq, 1, 64)
        if call == 0:
            api.moe_attention_forward(qd, kd, vd, cud, out, lse[1:-1], ws)
        else:
            api.moe_attention_backward(qd, kd, vd, cud, out, lse[1:-1], dod, *(g for _, g in grads), ws)
        assert api.moe_read_device_status(ws) == -5
    for w in [whole] + [w for w, _ in grads]:
        assert (w[:guard] == 5).all() and (w[-guard:] == 5).all()
    assert (lse[0] == 5).all() and (lse[-1] == 5).all()


@pytest.mark.parametrize("D", [8, 64, 80, 128])
@pytest.mark.parametrize("Hq,Hkv", [(200, 100), (160, 20), (180, 60), (170, 34)])
@pytest.mark.parametrize("lengths,first,tail", [([1], 0, 0), ([129, 0, 130, 1], 2, 5), ([5, 120, 3, 128], 0, 40)])
def test_two_tiles_an_item(lib, lengths, first, tail, Hq, Hkv, D):
    """Heads enough that items have two tiles of rows: of two heads, or (groups of odd sizes) of 256 rows."""
    c = _case(lengths, Hq, Hkv, D, seed=Hq + D, first=first, tail=tail)
    _check(_run(*c), *c)


def test_values_that_are_not_finite_with_two_tiles_an_item(lib):
    """Row 200 of [150, 290) and 301 of [290, 400): only what sees them may differ from the call without them."""
    for Hq, Hkv in ((200, 100), (180, 60)):
        cu, T, q, k, v, do = c = _case([150, 140, 110], Hq, Hkv, 64, seed=Hq)
        clean = _run(*c)
        for t in (k, v):
            dirty = {"k": k.clone(), "v": v.clone()}
            name = "k" if t is k else "v"
            dirty[name][200, :, ::3], dirty[name][301, :, 1::3] = float("nan"), float("inf")
            got = _run(cu, T, q, dirty["k"], dirty["v"], do)
            keep = torch.ones(T, dtype=torch.bool)
            keep[200:290] = keep[301:400] = False
            assert torch.equal(got["out"][keep], clean["out"][keep]) and torch.isfinite(got["out"][keep]).all()
            assert not torch.isfinite(got["out"][250].float()).all() and not torch.isfinite(got["out"][350].float()).all()


@pytest.mark.parametrize("D", [64, 128])
def test_infinite_values_give_the_same_bits_on_every_run(lib, D):
    """256 rows of one head: a key tile that one half has to mask and the other does not, with an infinite value whose
    probability is 0 in fp32 for most of the rows that see it (0 * inf, unless it has been taken out and is added back)."""
    cu, T, q, k, v, do = _case([40, 300, 172], 180, 60, D, seed=D, std=6.0)
    for row in (41, 130, 200, 300, 341, 400):
        v[row, :, row % 7::7] = float("inf") if row % 2 else -float("inf")
    qd, kd, vd = (t.to(DEV) for t in (q, k, v))
    cud, ws = torch.from_numpy(cu).to(DEV), _ws(T, 180, 60, D)
    first = None
    for _ in range(60):
        out, lse = torch.zeros_like(qd), torch.zeros(180, T, device=DEV)
        api.moe_attention_forward(qd, kd, vd, cud, out, lse, ws)
        if first is None:
            first = out, lse
            assert not torch.isfinite(out.float()).all() and torch.isfinite(out[:40].float()).all()
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
    assert api.moe_read_device_status(ws) == 0
