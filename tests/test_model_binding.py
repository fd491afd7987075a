"""The binding's checks of the embedding, layer-norm and cross-entropy calls that
need no GPU: sizes past 32 bits are refused, not cut off; tensors of a GPU other
than the current one are refused."""
import pytest

from moe_expert_layer_05_gb300 import api

PAST = 2 ** 32 + 8             # its low 32 bits are a size that would be accepted


class FakeTensor:
    """As much of a CUDA tensor as the checks look at, of any size."""

    def __init__(self, *shape, dtype=api._BF16, device=0):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, f"cuda:{device}", True
        self.index = device

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return 1

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 16


@pytest.fixture
def calls(monkeypatch):
    """The names of the library calls that got past the checks (none of them runs)."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(api, "load", lambda: Library())
    monkeypatch.setattr(api, "stream_ptr", lambda *a: None)
    monkeypatch.setattr(api, "_device", lambda: 0, raising=False)
    return made


def _bf(*shape):
    return FakeTensor(*shape)


def _f32(*shape):
    return FakeTensor(*shape, dtype=api._F32)


def _i32(*shape):
    return FakeTensor(*shape, dtype=api._I32)


def test_sizes_past_32_bits_are_refused(calls):
    ws = FakeTensor(1 << 20)
    refused = [
        lambda: api.moe_embedding_forward(_i32(PAST), _bf(8, 64), _bf(PAST, 64), ws),
        lambda: api.moe_embedding_forward(_i32(4), _bf(PAST, 64), _bf(4, 64), ws),
        lambda: api.moe_embedding_forward(_i32(4), _bf(8, PAST), _bf(4, PAST), ws),
        lambda: api.moe_embedding_backward(_i32(PAST), _bf(PAST, 64), _f32(8, 64), ws),
        lambda: api.moe_embedding_backward(_i32(4), _bf(4, 64), _f32(PAST, 64), ws),
        lambda: api.moe_layer_norm_forward(_bf(PAST, 64), _bf(64), None, _bf(PAST, 64), _f32(PAST), _f32(PAST)),
        lambda: api.moe_layer_norm_backward(_bf(PAST, 64), _bf(PAST, 64), _bf(64), _f32(PAST), _f32(PAST),
                                            _bf(PAST, 64), _f32(64), None, ws),
        lambda: api.moe_cross_entropy_forward(_bf(PAST, 64), _bf(9, 64), _i32(PAST), _f32(PAST), _f32(PAST), ws),
        lambda: api.moe_cross_entropy_forward(_bf(4, 64), _bf(PAST, 64), _i32(4), _f32(4), _f32(4), ws),
        lambda: api.moe_cross_entropy_backward(_bf(4, 64), _bf(PAST, 64), _i32(4), _f32(4), _f32(4), _bf(4, 64),
                                               _bf(PAST, 64), ws),
        lambda: api.moe_cross_entropy_backward(_bf(4, 64), _bf(9, 64), _i32(4), _f32(4), _f32(4), _bf(4, 64),
                                               _bf(9, 64), ws, piece=2 ** 32 + 256),
    ]
    for call in refused:
        with pytest.raises(api.MoeError) as e:
            call()
        assert e.value.code == -1
    assert calls == []
    # the same calls at sizes that fit do reach the library
    api.moe_embedding_forward(_i32(4), _bf(8, 64), _bf(4, 64), ws)
    api.moe_cross_entropy_backward(_bf(4, 64), _bf(9, 64), _i32(4), _f32(4), _f32(4), _bf(4, 64), _bf(9, 64), ws,
                                   piece=256)
    assert calls == ["moe_embedding_forward", "moe_cross_entropy_backward"]


def test_workspaces_of_sizes_past_32_bits_are_zero():
    for n, V, H in ((PAST, 8, 64), (8, PAST, 64), (8, 8, 2 ** 32 + 64)):
        assert api.moe_embedding_workspace_bytes(n, V, H) == 0
        assert api.moe_cross_entropy_workspace_bytes(n, H, V) == 0
    assert api.moe_layer_norm_workspace_bytes(PAST, 64) == 0 and api.moe_layer_norm_workspace_bytes(8, 2 ** 32 + 64) == 0
    assert api.moe_cross_entropy_workspace_bytes(8, 64, 8, 2 ** 32 + 256) == 0
    assert api.moe_embedding_workspace_bytes(8, 8, 64) > 0


def test_tensors_of_another_gpu_are_refused(calls):
    """Each tensor of each call on GPU 1 while GPU 0 is the current one, whose kernel could not read it."""
    ws = FakeTensor(1 << 20)
    by_call = {
        api.moe_embedding_forward: [_i32(4), _bf(8, 64), _bf(4, 64), ws],
        api.moe_embedding_backward: [_i32(4), _bf(4, 64), _f32(8, 64), ws],
        api.moe_layer_norm_forward: [_bf(4, 64), _bf(64), _bf(64), _bf(4, 64), _f32(4), _f32(4)],
        api.moe_layer_norm_backward: [_bf(4, 64), _bf(4, 64), _bf(64), _f32(4), _f32(4), _bf(4, 64), _f32(64), _f32(64),
                                      ws],
        api.moe_cross_entropy_forward: [_bf(4, 64), _bf(9, 64), _i32(4), _f32(4), _f32(4), ws],
        api.moe_cross_entropy_backward: [_bf(4, 64), _bf(9, 64), _i32(4), _f32(4), _f32(4), _bf(4, 64), _bf(9, 64), ws],
    }
    optional = {api.moe_embedding_backward: {"base": _bf(8, 64)},
                api.moe_layer_norm_forward: {"residual": _bf(4, 64), "sum_out": _bf(4, 64)},
                api.moe_layer_norm_backward: {"dsum": _bf(4, 64)}}
    for call, args in by_call.items():
        named = optional.get(call, {})
        call(*args, **named)
        assert calls.pop() == call.__name__
        for t in [*args, *named.values()]:
            t.index = 1
            with pytest.raises(ValueError):
                call(*args, **named)
            t.index = 0
        assert calls == []
