"""Calls that the step operators refuse at the edges of their ranges: scales whose scores leave fp32's range,
gradients that would be scaled twice.  No GPU needed."""
import math

import numpy as np
import pytest
import torch

from moe_expert_layer_05_gb300 import api, lm
from test_step_ops_abi import bwd, config, fwd, tensors

NO_GPU = not torch.cuda.is_available()


@pytest.mark.parametrize("scale", [2.0 ** -65, 1e-38, 1e-44, 2.0 ** 65, 3e38])
def test_scales_out_of_range_are_refused(scale):
    """The gradients' kernels form lse / scale, the forward scale * log2 e: both have to have fp32 values."""
    lib = api.load()
    c = config(scale=scale)
    assert lib.moe_attention_workspace_bytes(c) == 0
    assert fwd(lib, c) == -1 and bwd(lib, c) == -1


@pytest.mark.skipif(not NO_GPU, reason="fake pointers")
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** 64])
def test_scales_at_the_ends_of_the_range_are_taken(scale):
    lib = api.load()
    assert fwd(lib, config(scale=scale)) == -2 and bwd(lib, config(scale=scale)) == -2


def _many(n, first=1 << 20, step=64):
    return [(first + step * i, 16, 1) for i in range(n)]        # 16 fp32 values each, end to end


@pytest.mark.parametrize("n", [2, 64, 65, 600])
def test_what_is_scaled_twice_is_refused(n):
    lib = api.load()
    def clip(grads, outs=None):
        return lib.moe_grad_clip(tensors(*grads), tensors(*outs) if outs else None, len(grads), 16, 1.0, None)
    taken = -2 if NO_GPU else None
    grads, outs = _many(n), _many(n, first=1 << 30)
    again, into = list(grads), list(grads)
    again[-1] = grads[0]                                        # the same gradient twice
    into[-1] = (grads[0][0] + 48, 16, 1)                        # one that begins inside another
    assert clip(again) == -1 and clip(into) == -1
    twice = list(outs)
    twice[0] = (outs[1][0] - 16, 16, 1)                         # outputs that overlap
    assert clip(grads, twice) == -1
    assert clip(grads, grads) == -1                             # an output that is a gradient
    reaching = list(outs)
    reaching[0] = (grads[-1][0] + 48, 16, 1)
    assert clip(grads, reaching) == -1
    if NO_GPU:                                                  # (the pointers are fakes)
        assert clip(grads) == taken and clip(grads, outs) == taken
        assert clip(again, outs) == taken                       # a gradient that is only read, twice
        empty = list(grads)
        empty[0] = (grads[1][0], 0, 1)                          # nothing of it
        assert clip(empty) == taken


@pytest.mark.parametrize("heads,cu", [(0, torch.tensor([0, 9], dtype=torch.int32)), (2, torch.zeros(0, dtype=torch.int32)),
                                      (2, torch.tensor([0, 9])), (2, torch.tensor([[0, 9]], dtype=torch.int32))])
def test_a_model_refuses_boundaries_that_it_cannot_use(heads, cu):
    """Before anything is launched: none at all (an index into an empty tensor fails on the device), another type, or a
    model without attention, which would have left them unread."""
    m = lm.MoEModel.__new__(lm.MoEModel)
    m.T, m.heads = 9, heads
    tokens = torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_seqlens"):
        m.forward(tokens, tokens, cu)


# ---------------------------------------------------------------- rotary frequencies by parts
def _by_parts(R, base, factor, length, fast=32.0, slow=1.0):
    """The ramp over the pairs' indices, from the last whole pair that turns `fast` times to the first that turns `slow` times."""
    freq = base ** (-np.arange(0, R, 2) / R)

    def pair(turns):                                   # length base^(-2 i / R) = 2 pi turns
        return R / 2 * math.log(length / (2 * math.pi * turns)) / math.log(base)

    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
    slowed = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return freq * (1 - slowed) + freq / factor * slowed, slowed


@pytest.mark.parametrize("R,base,factor,length,fast,slow", [
    (64, 10000.0, 8.0, 4096, 32.0, 1.0), (128, 500000.0, 32.0, 8192, 32.0, 1.0), (16, 10000.0, 4.0, 512, 16.0, 2.0),
    (512, 1e6, 1.0, 32768, 32.0, 1.0), (48, 10000.0, 40.0, 100, 32.0, 1.0), (64, 10.0, 2.0, 4096, 32.0, 1.0),
    (64, 10000.0, 8.0, 4096, 7.3, 7.3)])
def test_the_ramp_between_the_parts(R, base, factor, length, fast, slow):
    freq, scale = api.moe_rotary_frequencies(R, base, "by_parts", factor, length, fast, slow, device="cpu")
    want, slowed = _by_parts(R, base, factor, length, fast, slow)
    assert ((slowed > 0) & (slowed < 1)).any() or R == 64 and (base == 10.0 or fast == slow)
    # pow and log to a few units of fp64 each, the ramp's ends whole numbers
    np.testing.assert_allclose(freq.numpy(), want, rtol=1e-13)
    assert abs(scale - (0.1 * math.log(factor) + 1)) <= 2.0 ** -23


@pytest.mark.parametrize("length,slow", [(1, 1.0), (4, 1.0), (6, 1.0), (100, 16.0), (4096, 1e6)])
def test_pairs_that_all_turn_less_than_the_slow_ones_are_all_slowed(length, slow):
    """The first pair turns length / (2 pi) times, fewer than `slow`: it is divided by the factor as the others are."""
    assert length / (2 * math.pi) < slow
    freq, _ = api.moe_rotary_frequencies(64, 10000.0, "by_parts", 8.0, length, max(slow, 32.0), slow, device="cpu")
    np.testing.assert_allclose(freq.numpy(), 10000.0 ** (-np.arange(0, 64, 2) / 64) / 8, rtol=1e-13)
