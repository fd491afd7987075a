"""The bounded waits of the vocabulary head's logits GEMM, with a limit of 1 ns
that no wait for a long contraction can meet (as in test_gpu_timeout.py): the call
returns, records MOE_ERR_TIMEOUT, and the same context then computes correctly."""
import numpy as np
import pytest
import torch

from gpu_helpers import f64
from moe_expert_layer_05_gb300 import api
from oracle import model_oracle as M
from test_gpu_model import DEV, U, _bf, _dz, _within, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [4096, 16384])              # whole contractions, and in segments
def test_cross_entropy_wait_limit_gives_timeout_status_and_the_context_recovers(lib, H):
    T, V = 100, 3000                                      # one-CTA tiles of 64 or 256 k-blocks
    rng = np.random.default_rng(H)
    x, w = _bf(rng, T, H), _bf(rng, V, H, std=1 / np.sqrt(H))
    lab = rng.integers(0, V, T).astype(np.int32)
    xd, wd, ld = x.to(DEV), w.to(DEV), torch.from_numpy(lab).to(DEV)
    loss, lse = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
    ws = _ws(api.moe_cross_entropy_workspace_bytes(T, H, V))
    api.moe_debug_set_wait_limit_ns(1)
    try:
        api.moe_cross_entropy_forward(xd, wd, ld, loss, lse, ws)
        torch.cuda.synchronize()
    finally:
        api.moe_debug_set_wait_limit_ns(0)
    assert api.moe_read_device_status(ws) == -6           # MOE_ERR_TIMEOUT
    words = ws[:256].view(torch.int32).cpu()
    assert int(words[32]) == 0 and int(words[33]) == 0    # the tile counter is back at zero
    api.moe_workspace_init(ws[:256])
    api.moe_cross_entropy_forward(xd, wd, ld, loss, lse, ws)
    assert api.moe_read_device_status(ws) == 0
    ref = M.cross_entropy(f64(x), f64(w), lab)
    _within(f64(lse), ref["lse"], _dz(ref) + (V / 16 + 64) * U, "lse")
