"""Refusals of the embedding, layer-norm and cross-entropy calls, before any
launch (no GPU needed: the device check comes after the argument checks, and
every call here fails an argument check or names fake pointers where no GPU
could be reached)."""
import pytest
import torch

from moe_expert_layer_05_gb300 import api

BIG = 1 << 40
NO_GPU = not torch.cuda.is_available()
BAD_H = [0, -8, 4, 100, 1001, 16392]


@pytest.mark.parametrize("H", BAD_H)
def test_bad_hidden_sizes_refused(H):
    lib = api.load()
    assert lib.moe_embedding_workspace_bytes(8, 8, H) == 0
    assert lib.moe_layer_norm_workspace_bytes(8, H) == 0
    assert lib.moe_cross_entropy_workspace_bytes(8, H, 8, 0) == 0
    assert lib.moe_embedding_forward(16, 8, 16, 8, H, 1.0, 16, 16, None) == -1
    assert lib.moe_embedding_backward(16, 8, 16, 8, H, 1.0, None, 16, 16, BIG, None) == -1
    assert lib.moe_layer_norm_forward(16, None, 16, None, 8, H, 1e-5, 16, None, 16, 16, None) == -1
    assert lib.moe_layer_norm_backward(16, 16, 16, 16, 16, None, 8, H, 16, 16, 16, 16, BIG, None) == -1
    assert lib.moe_cross_entropy_forward(16, 16, 16, 8, H, 8, 16, 16, 16, BIG, None) == -1
    assert lib.moe_cross_entropy_backward(16, 16, 16, 16, 16, 8, H, 8, 0, 16, 16, 16, BIG, None) == -1


@pytest.mark.parametrize("n,V", [(-1, 8), (8, 0), (8, -3), ((1 << 24) + 1, 8), (8, (1 << 24) + 1)])
def test_bad_counts_refused(n, V):
    lib = api.load()
    assert lib.moe_embedding_workspace_bytes(n, V, 64) == 0
    assert lib.moe_embedding_forward(16, n, 16, V, 64, 1.0, 16, 16, None) == -1
    assert lib.moe_embedding_backward(16, n, 16, V, 64, 1.0, None, 16, 16, BIG, None) == -1
    assert lib.moe_cross_entropy_workspace_bytes(n, 64, V, 0) == 0
    assert lib.moe_cross_entropy_forward(16, 16, 16, n, 64, V, 16, 16, 16, BIG, None) == -1
    assert lib.moe_cross_entropy_backward(16, 16, 16, 16, 16, n, 64, V, 0, 16, 16, 16, BIG, None) == -1


@pytest.mark.parametrize("T", [-1, (1 << 30) + 1])
def test_bad_row_counts_refused(T):
    lib = api.load()
    assert lib.moe_layer_norm_workspace_bytes(T, 64) == 0
    assert lib.moe_layer_norm_forward(16, None, 16, None, T, 64, 1e-5, 16, None, 16, 16, None) == -1
    assert lib.moe_layer_norm_backward(16, 16, 16, 16, 16, None, T, 64, 16, 16, 16, 16, BIG, None) == -1


def _each_pointer(call, required, optional=()):
    """Every required pointer missing or misaligned, every optional one misaligned."""
    for i in required:
        assert call(i, None) == -1, (i, "missing")
        assert call(i, 24) == -1, (i, "misaligned")
    for i in optional:
        assert call(i, 24) == -1, (i, "misaligned")


def test_pointers_checked():
    lib = api.load()

    def replaced(args):
        def call_of(fn):
            return lambda i, v: fn(*[v if j == i else a for j, a in enumerate(args)])
        return call_of

    _each_pointer(replaced([16, 8, 16, 8, 64, 1.0, 16, 16, None])(lib.moe_embedding_forward), [0, 2, 6, 7])
    _each_pointer(replaced([16, 8, 16, 8, 64, 1.0, None, 16, 16, BIG, None])(lib.moe_embedding_backward),
                  [0, 2, 7, 8], [6])
    _each_pointer(replaced([16, 16, 16, 16, 8, 64, 1e-5, 16, 16, 16, 16, None])(lib.moe_layer_norm_forward),
                  [0, 2, 7, 8, 9, 10], [1, 3])
    _each_pointer(replaced([16, 16, 16, 16, 16, 16, 8, 64, 16, 16, 16, 16, BIG, None])(lib.moe_layer_norm_backward),
                  [0, 1, 2, 3, 4, 8, 9, 11], [5, 10])
    _each_pointer(replaced([16, 16, 16, 8, 64, 8, 16, 16, 16, BIG, None])(lib.moe_cross_entropy_forward),
                  [0, 1, 2, 6, 7, 8])
    _each_pointer(replaced([16, 16, 16, 16, 16, 8, 64, 8, 0, 16, 16, 16, BIG, None])(lib.moe_cross_entropy_backward),
                  [0, 1, 2, 3, 4, 9, 10, 11])
    # a sum output without a residual to add; a negative or NaN eps; a negative piece
    assert lib.moe_layer_norm_forward(16, None, 16, None, 8, 64, 1e-5, 16, 16, 16, 16, None) == -1
    assert lib.moe_layer_norm_forward(16, None, 16, None, 8, 64, -1.0, 16, None, 16, 16, None) == -1
    assert lib.moe_layer_norm_forward(16, None, 16, None, 8, 64, float("nan"), 16, None, 16, 16, None) == -1
    assert lib.moe_cross_entropy_backward(16, 16, 16, 16, 16, 8, 64, 8, -1, 16, 16, 16, BIG, None) == -1


def test_small_workspaces_refused():
    lib = api.load()
    for n, V, H in ((0, 8, 8), (1, 8, 8), (1000, 5003, 1000), (100000, 100, 64)):
        need = lib.moe_embedding_workspace_bytes(n, V, H)
        assert need >= 256 + 16 * n + V
        assert lib.moe_embedding_backward(16, n, 16, V, H, 1.0, None, 16, 16, need - 1, None) == -4
    for T, H in ((1, 8), (5000, 7168)):
        need = lib.moe_layer_norm_workspace_bytes(T, H)
        assert lib.moe_layer_norm_backward(16, 16, 16, 16, 16, None, T, H, 16, 16, 16, 16, need - 1, None) == -4
    for T, H, V, piece in ((1, 8, 8, 0), (1003, 1000, 5003, 0), (4096, 4096, 131072, 0), (64, 128, 5003, 1000)):
        need = lib.moe_cross_entropy_workspace_bytes(T, H, V, piece)
        rows = min(-(-(piece or 256) // 256), -(-V // 256)) * 256
        assert need >= 256 + T * rows * 2 + T * H * 4
        assert lib.moe_cross_entropy_backward(16, 16, 16, 16, 16, T, H, V, piece, 16, 16, 16, need - 1, None) == -4
        assert lib.moe_cross_entropy_forward(16, 16, 16, T, H, V, 16, 16, 16, 256, None) == -4
    # the gradient's memory does not grow with the vocabulary beyond a piece and the forward's statistics
    big, small = (lib.moe_cross_entropy_workspace_bytes(4096, 4096, v, 0) for v in (1 << 20, 1 << 17))
    assert big < 4096 * (1 << 20) and big <= small + 16 * 4096 * ((1 << 20) // 256)


@pytest.mark.skipif(not NO_GPU, reason="fake pointers")
def test_good_arguments_reach_the_device_check():
    lib = api.load()
    assert lib.moe_embedding_forward(16, 8, 16, 8, 64, 1.0, 16, 16, None) == -2
    assert lib.moe_embedding_backward(None, 0, None, 8, 64, 1.0, None, 16, 16, BIG, None) == -2
    assert lib.moe_layer_norm_forward(None, None, 16, None, 0, 64, 1e-5, None, None, None, None, None) == -2
    assert lib.moe_layer_norm_backward(16, 16, 16, 16, 16, None, 8, 64, 16, 16, None, 16, BIG, None) == -2
    assert lib.moe_cross_entropy_forward(16, 16, 16, 8, 64, 8, 16, 16, 16, BIG, None) == -2
    assert lib.moe_cross_entropy_backward(16, 16, 16, 16, 16, 8, 64, 8, 0, 16, 16, 16, BIG, None) == -2


def test_binding_refuses_wrong_tensors():
    """Type, shape, layout and device are checked in the binding; all on the CPU here, so every call is refused."""
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    tok, x = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.moe_embedding_forward(tok, x, x, ws)
    with pytest.raises(ValueError):
        api.moe_embedding_backward(tok.long(), x, x.float(), ws)
    with pytest.raises(ValueError):
        api.moe_layer_norm_forward(x, x[0], None, x, x[:, 0].float(), x[:, 0].float())
    with pytest.raises(ValueError):
        api.moe_cross_entropy_forward(x[0], x, tok, x[:, 0].float(), x[:, 0].float(), ws)
