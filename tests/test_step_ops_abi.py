"""Refusals of the attention, rotary, balance-loss and gradient-norm calls, before any launch (no GPU needed: the
device check comes after the argument checks, and every call here fails an argument check or names fake pointers
where no GPU could be reached), and the binding's own checks."""
import math
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

from moe_expert_layer_05_gb300 import api
from test_model_binding import PAST, FakeTensor

BIG = 1 << 40
NO_GPU = not torch.cuda.is_available()
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def heads(data=16, token=256, head=64):
    return struct.pack("qqq", data or 0, token, head)


def config(T=100, n=3, Hq=4, Hkv=2, D=64, scale=0.125):
    return struct.pack("5if", T, n, Hq, Hkv, D, scale)


def fwd(lib, cfg=None, q=None, k=None, v=None, cu=16, out=None, lse=16, ws=16, nbytes=BIG):
    h = heads()
    return lib.moe_attention_forward(config() if cfg is None else cfg, q or h, k or h, v or h, cu, out or h, lse, ws, nbytes,
                                     None)


def bwd(lib, cfg=None, at=None, value=None, cu=16, lse=16, ws=16, nbytes=BIG):
    """Every tensor in order q, k, v, out, dout, dq, dk, dv; number `at` replaced."""
    t = [heads()] * 8
    if at is not None:
        t[at] = value
    return lib.moe_attention_backward(config() if cfg is None else cfg, t[0], t[1], t[2], cu, t[3], lse, t[4], t[5], t[6],
                                      t[7], ws, nbytes, None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=(1 << 24) + 1), dict(n=-1), dict(n=(1 << 24) + 1), dict(Hq=0), dict(Hkv=0),
                                 dict(Hq=-4), dict(Hq=5), dict(Hq=1028, Hkv=4), dict(D=0), dict(D=4), dict(D=100),
                                 dict(D=136), dict(D=-64), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
                                 dict(scale=math.nan)])
def test_bad_attention_configs_refused(bad):
    lib = api.load()
    c = config(**bad)
    assert lib.moe_attention_workspace_bytes(c) == 0
    assert fwd(lib, c) == -1 and bwd(lib, c) == -1


def test_bad_attention_tensors_refused():
    lib = api.load()
    bad = [heads(data=0), heads(data=24), heads(token=0), heads(token=-256), heads(token=100), heads(head=0), heads(head=4),
           heads(token=1 << 38), heads(head=1 << 40)]
    for b in bad:
        for name in ("q", "k", "v", "out"):
            assert fwd(lib, **{name: b}) == -1, (name, b)
        for i in range(8):
            assert bwd(lib, at=i, value=b) == -1, (i, b)
    # outputs whose elements are not all different places: rows that overlap, heads that overlap
    for b in (heads(token=192), heads(head=32), heads(token=8, head=8), heads(token=64, head=99 * 64)):
        assert fwd(lib, out=b) == -1, b
        assert bwd(lib, at=5, value=b) == -1, b
    for name, v in (("cu", None), ("cu", 24), ("lse", None), ("lse", 24), ("ws", None), ("ws", 24)):
        assert fwd(lib, **{name: v}) == -1, name
        assert bwd(lib, **{name: v}) == -1, name
    assert lib.moe_attention_forward(config(), None, heads(), heads(), 16, heads(), 16, 16, BIG, None) == -1
    assert lib.moe_attention_forward(None, heads(), heads(), heads(), 16, heads(), 16, 16, BIG, None) == -1


def test_small_attention_workspaces_refused():
    lib = api.load()
    for T, Hq, Hkv, D in ((1, 1, 1, 8), (1000, 6, 2, 80), (8192, 32, 8, 128)):
        need = api.moe_attention_workspace_bytes(T, Hq, Hkv, D)
        assert need >= 256 + 8 * T * Hq
        c = config(T, 1, Hq, Hkv, D)
        dense = heads(token=Hq * D, head=D)
        assert lib.moe_attention_backward(c, dense, dense, dense, 16, dense, 16, dense, dense, dense, dense, 16, need - 1,
                                          None) == -4
        assert lib.moe_attention_forward(c, dense, dense, dense, 16, dense, 16, 16, 255, None) == -4
    assert api.moe_attention_workspace_bytes(2 ** 32 + 8, 1, 1, 64) == 0


def test_rotary_frequencies_checked():
    from ctypes import byref, c_double, c_float
    lib = api.load()
    f, s = (c_double * 256)(), c_float()

    def call(R=64, base=1e4, kind=0, factor=1.0, length=0, fast=32.0, slow=1.0, freq=f, scale=byref(s)):
        return lib.moe_rotary_frequencies(R, base, kind, factor, length, fast, slow, freq, scale)

    assert call() == 0
    for bad in (dict(R=0), dict(R=-16), dict(R=8), dict(R=24), dict(R=528), dict(base=1.0), dict(base=math.nan),
                dict(base=math.inf), dict(kind=3), dict(kind=-1), dict(freq=None), dict(scale=None),
                dict(kind=1, factor=0.5), dict(kind=1, factor=math.nan), dict(kind=2, factor=2.0),
                dict(kind=2, factor=2.0, length=4096, slow=0.0), dict(kind=2, factor=2.0, length=4096, fast=0.5)):
        assert call(**bad) == -1, bad
    assert call(kind=2, factor=2.0, length=4096) == 0
    plain, one = api.moe_rotary_frequencies(32, device="cpu")
    np.testing.assert_allclose(plain.numpy(), 1e4 ** (-np.arange(0, 32, 2) / 32), rtol=1e-14)
    assert one == 1.0


def test_rotary_arguments_checked():
    lib = api.load()

    def call(x=None, pos=16, freq=16, T=10, n=4, width=64, R=32, out=None):
        return lib.moe_rotary(x or heads(), pos, freq, T, n, width, R, 0, 1.0, 0, out or heads(data=1 << 20), None)

    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(n=0), dict(n=1025), dict(width=0), dict(width=60), dict(width=520),
                dict(R=0), dict(R=8), dict(R=80), dict(pos=None), dict(pos=24), dict(freq=None), dict(freq=24),
                dict(x=heads(data=0)), dict(x=heads(data=24)), dict(x=heads(token=100)), dict(x=heads(head=0)),
                dict(out=heads(data=0)), dict(out=heads(data=1 << 20, token=192)), dict(out=heads(data=1 << 20, head=32)),
                dict(out=heads(token=512))):                          # in place, with other strides than x's
        assert call(**bad) == -1, bad
    assert lib.moe_rotary(None, 16, 16, 10, 4, 64, 32, 0, 1.0, 0, heads(), None) == -1


def test_balance_arguments_checked():
    lib = api.load()

    def forward(logits=16, topk=16, tokens=None, T=8, E=16, k=2, score=0, loss=16, counts=16, slope=16, ws=16, n=BIG):
        return lib.moe_balance_loss_forward(logits, topk, tokens, T, E, k, score, loss, counts, slope, ws, n, None)

    def backward(logits=16, slope=16, tokens=None, T=8, E=16, score=0, dloss=16, dlogits=16):
        return lib.moe_balance_loss_backward(logits, slope, tokens, T, E, score, dloss, dlogits, None)

    both = [dict(logits=None), dict(logits=24), dict(tokens=24), dict(T=-1), dict(T=(1 << 24) + 1), dict(E=0), dict(E=257),
            dict(score=2), dict(score=-1), dict(slope=None), dict(slope=18)]
    for bad in both + [dict(topk=None), dict(topk=24), dict(k=0), dict(k=33, E=64), dict(k=17), dict(loss=None), dict(loss=17),
                       dict(counts=None), dict(counts=18), dict(ws=None), dict(ws=24)]:
        assert forward(**bad) == -1, bad
    for bad in both + [dict(dloss=None), dict(dloss=18), dict(dlogits=None), dict(dlogits=24)]:
        assert backward(**bad) == -1, bad
    for T, E in ((0, 1), (1, 8), (100000, 256)):
        need = api.moe_balance_loss_workspace_bytes(T, E)
        assert need >= 256 and forward(T=T, E=E, k=1, n=need - 1) == -4
    for T, E in ((-1, 8), (8, 0), (8, 257), (2 ** 32 + 8, 8)):
        assert api.moe_balance_loss_workspace_bytes(T, E) == 0


def tensors(*t):
    return b"".join(struct.pack("qqq", *x) for x in t)


def test_gradient_list_arguments_checked():
    lib = api.load()
    good = tensors((16, 100, 0), (0, 0, 1))
    assert api.moe_grad_norm_workspace_bytes(-1) == 0 and api.moe_grad_norm_workspace_bytes((1 << 20) + 1) == 0
    need = api.moe_grad_norm_workspace_bytes(2)
    assert need > 256
    for bad in (tensors((24, 100, 0)), tensors((0, 100, 0)), tensors((16, -1, 0)), tensors((16, 1 << 41, 0)),
                tensors((16, 5, 2)), tensors((16, 5, -1))):
        assert lib.moe_grad_norm(bad, 1, 16, 16, BIG, None) == -1
        assert lib.moe_grad_clip(bad, None, 1, 16, 1.0, None) == -1
        assert lib.moe_grad_clip(tensors((16, 5, 0)), bad, 1, 16, 1.0, None) == -1
    assert lib.moe_grad_norm(good, 2, 16, 16, need - 1, None) == -4
    for args in ((good, -1, 16, 16, BIG), (None, 2, 16, 16, BIG), (good, 2, None, 16, BIG), (good, 2, 18, 16, BIG),
                 (good, 2, 16, None, BIG), (good, 2, 16, 24, BIG), (good, (1 << 20) + 1, 16, 16, BIG)):
        assert lib.moe_grad_norm(*args, None) == -1
    for limit in (-1.0, math.nan):
        assert lib.moe_grad_clip(good, None, 2, 16, limit, None) == -1
    assert lib.moe_grad_clip(good, None, 2, None, 1.0, None) == -1
    for outs in (tensors((32, 99, 0), (0, 0, 1)), tensors((32, 100, 1), (0, 0, 1))):      # another size, another type
        assert lib.moe_grad_clip(good, outs, 2, 16, 1.0, None) == -1


@pytest.mark.skipif(not NO_GPU, reason="fake pointers")
def test_good_arguments_reach_the_device_check():
    lib = api.load()
    assert fwd(lib) == -2 and bwd(lib) == -2
    empty = config(T=0)
    assert fwd(lib, empty, cu=None, lse=None) == -2 and fwd(lib, config(n=0), cu=None) == -2
    # one head, one row: their strides are not looked at
    one = heads(token=-3, head=5)
    assert lib.moe_attention_forward(config(T=1, n=1, Hq=1, Hkv=1), one, one, one, 16, one, 16, 16, BIG, None) == -2
    # heads before rows
    turned = heads(token=64, head=6400)
    assert fwd(lib, q=turned, out=turned) == -2
    assert lib.moe_rotary(heads(), 16, 16, 10, 4, 64, 32, 1, 1.0, 1, heads(), None) == -2
    assert lib.moe_balance_loss_forward(16, 16, 16, 8, 16, 2, 1, 20, 20, 20, 16, BIG, None) == -2
    assert lib.moe_balance_loss_backward(16, 20, None, 8, 16, 0, 20, 16, None) == -2
    assert lib.moe_grad_norm(None, 0, 20, 16, BIG, None) == -2
    assert lib.moe_grad_clip(tensors((16, 5, 0)), tensors((32, 5, 0)), 1, 20, math.inf, None) == -2


C_SRC = r"""
#include <stddef.h>
#include <stdio.h>
#include "moe_gb300.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu %zu\n", sizeof(moe_heads), offsetof(moe_heads, token_stride),
         offsetof(moe_heads, head_stride), sizeof(moe_attention_config), offsetof(moe_attention_config, scale),
         sizeof(moe_tensor), offsetof(moe_tensor, n), offsetof(moe_tensor, type));
  return 0;
}
"""


def test_packed_words_are_the_header_s_structures():
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    out_dir = os.path.dirname(api.library_path())
    api.load()
    src, exe = os.path.join(out_dir, "c_abi_words.c"), os.path.join(out_dir, "c_abi_words")
    with open(src, "w") as fh:
        fh.write(C_SRC)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"), src,
                    "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [24, 8, 16, 24, 20, 24, 8, 16]


# ---------------------------------------------------------------- the binding
class Strided(FakeTensor):
    def __init__(self, *shape, strides=None, **kw):
        super().__init__(*shape, **kw)
        dense = [1]
        for n in reversed(shape[1:]):
            dense.insert(0, dense[0] * n)
        self.strides = tuple(dense) if strides is None else strides

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(api, "load", lambda: Library())
    monkeypatch.setattr(api, "stream_ptr", lambda *a: None)
    monkeypatch.setattr(api, "_device", lambda: 0, raising=False)
    return made


def _bf(*shape, **kw):
    return Strided(*shape, **kw)


def _f32(*shape):
    return FakeTensor(*shape, dtype=api._F32)


def _i32(*shape):
    return FakeTensor(*shape, dtype=api._I32)


def _calls():
    """Each call with tensors that are accepted."""
    q, k, v, out, do, dq, dk, dv = (_bf(10, h, 64) for h in (4, 2, 2, 4, 4, 4, 2, 2))
    ws, lse, cu = FakeTensor(1 << 20), _f32(4, 10), _i32(3)
    freq = FakeTensor(16, dtype=torch.float64)
    return {api.moe_attention_forward: [q, k, v, cu, out, lse, ws],
            api.moe_attention_backward: [q, k, v, cu, out, lse, do, dq, dk, dv, ws],
            api.moe_rotary: [_bf(10, 4, 64), _i32(10), freq, _bf(10, 4, 64)],
            api.moe_balance_loss_forward: [_f32(10, 8), _i32(10, 2), _f32(1), _i32(8), _f32(8), ws],
            api.moe_balance_loss_backward: [_f32(10, 8), _f32(8), _f32(1), _f32(10, 8)]}


def test_tensors_of_another_gpu_type_or_shape_are_refused(calls):
    for call, args in _calls().items():
        named = {"tokens": _i32(10)} if "balance" in call.__name__ else {}
        call(*args, **named)
        assert calls.pop() == call.__name__
        for t in [*args, *named.values()]:
            t.index = 1
            with pytest.raises(ValueError):
                call(*args, **named)
            t.index = 0
            if t.numel() == 1 << 20:
                continue                                # (the workspace is of any type)
            kept, t.dtype = t.dtype, torch.float16
            with pytest.raises(ValueError):
                call(*args, **named)
            t.dtype = kept
        assert calls == []
    args = _calls()[api.moe_attention_forward]
    for i, other in ((1, _bf(11, 2, 64)), (1, _bf(10, 2, 32)), (2, _bf(10, 1, 64)), (4, _bf(10, 2, 64)), (5, _f32(4, 11)),
                     (0, _bf(10, 4, 64, strides=(256, 64, 2))), (0, _bf(10, 256)), (3, _i32(0))):
        with pytest.raises(ValueError):
            api.moe_attention_forward(*[other if j == i else a for j, a in enumerate(args)])
    with pytest.raises(ValueError):
        api.moe_rotary(_bf(10, 64), _i32(10), FakeTensor(16, dtype=torch.float64), _bf(10, 64))
    assert calls == []


def test_sizes_past_32_bits_are_refused(calls):
    ws = FakeTensor(1 << 20)
    big = [lambda: api.moe_attention_forward(_bf(PAST, 4, 64), _bf(PAST, 2, 64), _bf(PAST, 2, 64), _i32(3), _bf(PAST, 4, 64),
                                             _f32(4, PAST), ws),
           lambda: api.moe_attention_forward(_bf(10, PAST, 64), _bf(10, 2, 64), _bf(10, 2, 64), _i32(3), _bf(10, PAST, 64),
                                             _f32(PAST, 10), ws),
           lambda: api.moe_attention_forward(_bf(10, 4, 64), _bf(10, 2, 64), _bf(10, 2, 64), _i32(PAST), _bf(10, 4, 64),
                                             _f32(4, 10), ws),
           lambda: api.moe_rotary(_bf(PAST, 4, 64), _i32(PAST), FakeTensor(16, dtype=torch.float64), _bf(PAST, 4, 64)),
           lambda: api.moe_rotary(_bf(10, 4, 64), _i32(10), FakeTensor(PAST, dtype=torch.float64), _bf(10, 4, 64)),
           lambda: api.moe_balance_loss_forward(_f32(PAST, 8), _i32(PAST, 2), _f32(1), _i32(8), _f32(8), ws),
           lambda: api.moe_balance_loss_backward(_f32(10, PAST), _f32(PAST), _f32(1), _f32(10, PAST))]
    for call in big:
        with pytest.raises(api.MoeError) as e:
            call()
        assert e.value.code == -1
    assert calls == []


def test_gradient_lists_are_checked(calls):
    ws, norm = FakeTensor(1 << 20), _f32(1)
    g = [_f32(5, 3), _bf(7), _f32(0)]
    api.moe_grad_norm(g, norm, ws)
    api.moe_grad_clip(g, norm, 1.0)
    api.moe_grad_clip(g, norm, 1.0, outs=[_f32(15), _bf(7), _f32(0)])
    assert calls == ["moe_grad_norm", "moe_grad_clip", "moe_grad_clip"]
    for t in g:
        t.index = 1
        with pytest.raises(ValueError):
            api.moe_grad_norm(g, norm, ws)
        t.index = 0
    for outs in ([_f32(15), _bf(7)], [_f32(15), _f32(7), _f32(0)], [_f32(14), _bf(7), _f32(0)]):
        with pytest.raises(ValueError):
            api.moe_grad_clip(g, norm, 1.0, outs=outs)
    with pytest.raises(ValueError):
        api.moe_grad_norm([FakeTensor(3, dtype=torch.float16)], norm, ws)
    assert len(calls) == 3


@pytest.mark.parametrize("scale", [1e39, -1e300, math.inf, math.nan, 10 ** 40])
def test_scales_without_an_fp32_form_are_refused_as_others_are(calls, scale):
    made = _calls()
    for call in (api.moe_attention_forward, api.moe_attention_backward):
        with pytest.raises(api.MoeError) as e:
            call(*made[call], scale=scale)
        assert e.value.code == -1
    assert calls == []
