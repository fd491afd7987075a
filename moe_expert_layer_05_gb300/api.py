"""Python binding of libmoe_gb300.so (ctypes): the C-ABI calls under the same
names, plus a small buffer holder that uses PyTorch only to allocate device
memory and to pick the stream.  Every step of the layer runs in the library's
CUDA kernels; there is no fallback path — if the library is missing or the GPU
is not a GB300 the calls raise.
"""
from __future__ import annotations

import array
import ctypes
import os
import struct

import torch

from . import build as _build

MOE_OK = 0
STATUS_NAMES = {0: "ok", -1: "invalid argument", -2: "unsupported", -3: "CUDA error", -4: "workspace too small",
                -5: "bad expert index", -6: "device wait timed out"}
SCORE = {"softmax": 0, "sigmoid": 1}
GEMM_DTYPE = {"bf16": 0, "mxfp8": 1, "nvfp4": 2}

(GG_FC1_SWIGLU, GG_FC2, GG_DGRAD_FC2, GG_DGRAD_FC1, GG_WGRAD_FC1, GG_WGRAD_FC2, GG_FC1_SWIGLU_GATHERED,
 GG_FC2_COMBINE) = range(8)
ROTARY_SCALING = {"plain": 0, "linear": 1, "by_parts": 2}
MX_ROWS, MX_COLS_T, MX_ROWS_GATE_UP, MX_ROWS_G224, MX_COLS_T_G224 = range(5)

c_i32 = ctypes.c_int32
c_vp = ctypes.c_void_p
c_sz = ctypes.c_size_t
c_f32 = ctypes.c_float
c_f64 = ctypes.c_double


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", c_i32), ("H", c_i32), ("E", c_i32), ("k", c_i32), ("F", c_i32), ("S", c_i32),
                ("score", c_i32), ("dtype", c_i32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("w_router", c_vp), ("router_bias", c_vp), ("w1", c_vp), ("w2", c_vp),
                ("w1_shared", c_vp), ("w2_shared", c_vp), ("mx", c_vp)]


class MoeGrads(ctypes.Structure):
    _fields_ = [("dw_router", c_vp), ("dw1", c_vp), ("dw2", c_vp), ("dw1_shared", c_vp), ("dw2_shared", c_vp)]


_LAYOUT_FIELDS = ["logits", "topk_idx", "topk_gate", "counts", "offsets", "poffsets", "slot_row", "row_src",
                  "row_gate", "x_perm", "z", "h", "o", "zs", "hs", "os", "dy_perm", "dz", "dx_perm",
                  "dgate_part", "dlogits", "row_dlogit", "dzs", "dxs", "dz_qt", "dz_qt_sf", "h_qt",
                  "h_qt_sf"]


class MoeActLayout(ctypes.Structure):
    _fields_ = [(n, c_sz) for n in _LAYOUT_FIELDS] + [("total", c_sz), ("cap", c_i32), ("backward", c_i32)]


class MoeGemmArgs(ctypes.Structure):
    _fields_ = [("op", c_i32), ("dense_rows", c_i32), ("a", c_vp), ("b", c_vp), ("c", c_vp), ("c2", c_vp),
                ("aux", c_vp), ("row_gate", c_vp), ("dgate_part", c_vp), ("poffsets", c_vp),
                ("a_scales", c_vp), ("b_scales", c_vp), ("a_amax", c_vp), ("b_amax", c_vp), ("a_rows", c_vp),
                ("slot_row", c_vp), ("b_scale_group", c_i32), ("q_codes", c_vp), ("q_scales", c_vp),
                ("qt_codes", c_vp), ("qt_scales", c_vp)]


_P = ctypes.POINTER
_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [c_i32]),
    "moe_version": (c_i32, []),
    "moe_kernel_launches": (ctypes.c_uint64, []),
    "moe_debug_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "moe_capacity_rows": (c_i32, [_P(MoeConfig)]),
    "moe_activation_layout": (c_i32, [_P(MoeConfig), c_i32, _P(MoeActLayout)]),
    "moe_workspace_bytes": (c_sz, [_P(MoeConfig)]),
    "moe_workspace_init": (c_i32, [c_vp, c_sz, c_vp]),
    "moe_read_device_status": (c_i32, [c_vp, _P(c_i32), c_vp]),
    "moe_router_topk": (c_i32, [_P(MoeConfig), c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "moe_topk_gating": (c_i32, [_P(MoeConfig), c_vp, c_vp, c_vp, c_vp, c_vp]),
    "moe_permute": (c_i32, [_P(MoeConfig), c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32,
                            c_vp, c_vp]),
    "moe_permute_noalloc": (c_i32, [_P(MoeConfig), c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                    c_i32, c_vp]),
    "moe_grouped_gemm": (c_i32, [_P(MoeConfig), _P(MoeGemmArgs), c_vp, c_vp]),
    "moe_unpermute": (c_i32, [_P(MoeConfig), c_vp, c_vp, c_vp, c_vp, c_vp]),
    "moe_quantize_mxfp8": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp]),
    "moe_mxfp8_weights_bytes": (c_sz, [_P(MoeConfig)]),
    "moe_prepare_mxfp8_weights": (c_i32, [_P(MoeConfig), _P(MoeWeights), c_vp, c_sz, c_vp]),
    "moe_quantize_nvfp4": (c_i32, [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]),
    "moe_nvfp4_weights_bytes": (c_sz, [_P(MoeConfig)]),
    "moe_prepare_nvfp4_weights": (c_i32, [_P(MoeConfig), _P(MoeWeights), c_vp, c_sz, c_vp]),
    "moe_layer_forward": (c_i32, [_P(MoeConfig), _P(MoeWeights), c_vp, c_vp, c_vp, c_sz, c_i32, c_vp, c_sz,
                                  c_vp]),
    "moe_layer_backward_dgrad": (c_i32, [_P(MoeConfig), _P(MoeWeights), c_vp, c_vp, c_vp, c_vp, c_vp, c_sz,
                                         c_vp, c_sz, c_vp]),
    "moe_layer_backward_wgrad": (c_i32, [_P(MoeConfig), _P(MoeWeights), c_vp, c_vp, _P(MoeGrads), c_vp, c_sz,
                                         c_vp, c_sz, c_vp]),
    "moe_embedding_workspace_bytes": (c_sz, [c_i32, c_i32, c_i32]),
    "moe_embedding_forward": (c_i32, [c_vp, c_i32, c_vp, c_i32, c_i32, c_f32, c_vp, c_vp, c_vp]),
    "moe_embedding_backward": (c_i32, [c_vp, c_i32, c_vp, c_i32, c_i32, c_f32, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "moe_layer_norm_forward": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "moe_layer_norm_workspace_bytes": (c_sz, [c_i32, c_i32]),
    "moe_layer_norm_backward": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp,
                                        c_sz, c_vp]),
    "moe_cross_entropy_workspace_bytes": (c_sz, [c_i32, c_i32, c_i32, c_i32]),
    "moe_cross_entropy_forward": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "moe_cross_entropy_backward": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp,
                                           c_vp, c_sz, c_vp]),
    "moe_attention_workspace_bytes": (c_sz, [c_vp]),
    "moe_attention_forward": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp,
                                      c_vp, c_vp, c_vp, c_sz, c_vp]),
    "moe_attention_backward": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp,
                                       c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                       c_vp, c_sz, c_vp]),
    "moe_rotary_frequencies": (c_i32, [c_i32, c_f64, c_i32, c_f64, c_i32, c_f64, c_f64, _P(c_f64), _P(c_f32)]),
    "moe_rotary": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_f32, c_i32, c_vp,
                           c_vp]),
    "moe_balance_loss_workspace_bytes": (c_sz, [c_i32, c_i32]),
    "moe_balance_loss_forward": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_sz,
                                         c_vp]),
    "moe_balance_loss_backward": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp]),
    "moe_grad_norm_workspace_bytes": (c_sz, [c_i32]),
    "moe_grad_norm": (c_i32, [c_vp, c_i32, c_vp, c_vp, c_sz, c_vp]),
    "moe_grad_clip": (c_i32, [c_vp, c_vp, c_i32, c_vp, c_f32, c_vp]),
}

_lib = None


def library_path() -> str:
    """libmoe_gb300.so built in-tree, or the file MOE_GB300_LIBRARY names."""
    return os.environ.get("MOE_GB300_LIBRARY") or _build.LIB_PATH


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libmoe_gb300.so (building it first if absent).  Raises if it cannot."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libmoe_gb300.so not built ({path}); run __graft_entry__.build()")
        _build.build()
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)} ({code})")
        self.code = code


def check(code: int, what: str) -> None:
    if code != MOE_OK:
        raise MoeError(code, what)


def ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without a Stream object around it (0.1 us against
# 3 us of a call's 8-11 us on the host), where this torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_ptr(stream=None, dev: int | None = None) -> int | None:
    """Handle of `stream`, or of the current stream of the current GPU (dev, where the caller has asked already)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if dev is None else dev)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def make_config(T, H, E, k, F, S=0, score="softmax", dtype="bf16") -> MoeConfig:
    return MoeConfig(T, H, E, k, F, S, SCORE[score] if isinstance(score, str) else int(score),
                     GEMM_DTYPE[dtype] if isinstance(dtype, str) else int(dtype))


def config_of(workload, tokens: int | None = None) -> MoeConfig:
    w = workload
    return make_config(w.T if tokens is None else tokens, w.H, w.E, w.k, w.F, w.S, w.score, w.dtype)


# ---------------------------------------------------------------- C calls, same names
def moe_capacity_rows(cfg: MoeConfig) -> int:
    return load().moe_capacity_rows(ctypes.byref(cfg))


def moe_activation_layout(cfg: MoeConfig, with_backward: bool) -> MoeActLayout:
    L = MoeActLayout()
    check(load().moe_activation_layout(ctypes.byref(cfg), int(with_backward), ctypes.byref(L)),
          "moe_activation_layout")
    return L


def moe_workspace_bytes(cfg: MoeConfig) -> int:
    return load().moe_workspace_bytes(ctypes.byref(cfg))


def moe_workspace_init(ws: torch.Tensor, stream=None) -> None:
    check(load().moe_workspace_init(ptr(ws), ws.numel() * ws.element_size(), stream_ptr(stream)),
          "moe_workspace_init")


def moe_read_device_status(ws: torch.Tensor, stream=None) -> int:
    code = c_i32(0)
    check(load().moe_read_device_status(ptr(ws), ctypes.byref(code), stream_ptr(stream)), "moe_read_device_status")
    return code.value


def moe_router_topk(cfg, x, w_router, bias, logits, topk_idx, topk_gate, ws, stream=None) -> None:
    check(load().moe_router_topk(ctypes.byref(cfg), ptr(x), ptr(w_router), ptr(bias), ptr(logits), ptr(topk_idx),
                                 ptr(topk_gate), ptr(ws), stream_ptr(stream)), "moe_router_topk")


def moe_topk_gating(cfg, logits, bias, topk_idx, topk_gate, stream=None) -> None:
    check(load().moe_topk_gating(ctypes.byref(cfg), ptr(logits), ptr(bias), ptr(topk_idx), ptr(topk_gate),
                                 stream_ptr(stream)), "moe_topk_gating")


def moe_permute(cfg, x, topk_idx, topk_gate, counts, offsets, poffsets, slot_row, row_src, row_gate, x_perm,
                zero_pad, ws, stream=None) -> None:
    check(load().moe_permute(ctypes.byref(cfg), ptr(x), ptr(topk_idx), ptr(topk_gate), ptr(counts), ptr(offsets),
                             ptr(poffsets), ptr(slot_row), ptr(row_src), ptr(row_gate), ptr(x_perm), int(zero_pad),
                             ptr(ws), stream_ptr(stream)), "moe_permute")


def moe_permute_noalloc(cfg, x, topk_idx, topk_gate, counts, offsets, poffsets, slot_row, row_src, row_gate,
                        x_perm, zero_pad, stream=None) -> None:
    """moe_permute for callers that cannot allocate: no workspace argument;
    the scratch is a fixed 1 MiB device array inside the library."""
    check(load().moe_permute_noalloc(ctypes.byref(cfg), ptr(x), ptr(topk_idx), ptr(topk_gate), ptr(counts),
                                     ptr(offsets), ptr(poffsets), ptr(slot_row), ptr(row_src), ptr(row_gate),
                                     ptr(x_perm), int(zero_pad), stream_ptr(stream)), "moe_permute_noalloc")


def moe_grouped_gemm(cfg, op, a, b, c, ws, c2=None, aux=None, row_gate=None, dgate_part=None, poffsets=None,
                     dense_rows=0, a_scales=None, b_scales=None, a_amax=None, b_amax=None, a_rows=None,
                     slot_row=None, b_scale_group=0, q_codes=None, q_scales=None, qt_codes=None, qt_scales=None,
                     stream=None) -> None:
    args = MoeGemmArgs(op, dense_rows, ptr(a), ptr(b), ptr(c), ptr(c2), ptr(aux), ptr(row_gate), ptr(dgate_part),
                       ptr(poffsets), ptr(a_scales), ptr(b_scales), ptr(a_amax), ptr(b_amax), ptr(a_rows),
                       ptr(slot_row), int(b_scale_group), ptr(q_codes), ptr(q_scales), ptr(qt_codes), ptr(qt_scales))
    check(load().moe_grouped_gemm(ctypes.byref(cfg), ctypes.byref(args), ptr(ws), stream_ptr(stream)),
          "moe_grouped_gemm")


def moe_quantize_mxfp8(src, batch, rows, cols, mode, codes, scales, stream=None) -> None:
    check(load().moe_quantize_mxfp8(ptr(src), batch, rows, cols, mode, ptr(codes), ptr(scales),
                                    stream_ptr(stream)), "moe_quantize_mxfp8")


def moe_mxfp8_weights_bytes(cfg) -> int:
    return int(load().moe_mxfp8_weights_bytes(ctypes.byref(cfg)))


def moe_prepare_mxfp8_weights(cfg, weights: MoeWeights, mx, stream=None) -> None:
    check(load().moe_prepare_mxfp8_weights(ctypes.byref(cfg), ctypes.byref(weights), ptr(mx),
                                           mx.numel() * mx.element_size(), stream_ptr(stream)),
          "moe_prepare_mxfp8_weights")


def moe_quantize_nvfp4(src, batch, rows, cols, mode, codes, scales, amax, stream=None) -> None:
    check(load().moe_quantize_nvfp4(ptr(src), batch, rows, cols, mode, ptr(codes), ptr(scales), ptr(amax),
                                    stream_ptr(stream)), "moe_quantize_nvfp4")


def moe_nvfp4_weights_bytes(cfg) -> int:
    return int(load().moe_nvfp4_weights_bytes(ctypes.byref(cfg)))


def moe_prepare_nvfp4_weights(cfg, weights: MoeWeights, buf, stream=None) -> None:
    check(load().moe_prepare_nvfp4_weights(ctypes.byref(cfg), ctypes.byref(weights), ptr(buf),
                                           buf.numel() * buf.element_size(), stream_ptr(stream)),
          "moe_prepare_nvfp4_weights")


def moe_unpermute(cfg, o_perm, slot_row, shared_out, y, stream=None) -> None:
    check(load().moe_unpermute(ctypes.byref(cfg), ptr(o_perm), ptr(slot_row), ptr(shared_out), ptr(y),
                               stream_ptr(stream)), "moe_unpermute")


def moe_layer_forward(cfg, weights: MoeWeights, x, y, act, with_backward, ws, stream=None) -> None:
    check(load().moe_layer_forward(ctypes.byref(cfg), ctypes.byref(weights), ptr(x), ptr(y), ptr(act),
                                   act.numel() * act.element_size(), int(with_backward), ptr(ws),
                                   ws.numel() * ws.element_size(), stream_ptr(stream)), "moe_layer_forward")


def moe_layer_backward_dgrad(cfg, weights: MoeWeights, x, dy, dx, dgate, act, ws, stream=None) -> None:
    check(load().moe_layer_backward_dgrad(ctypes.byref(cfg), ctypes.byref(weights), ptr(x), ptr(dy), ptr(dx),
                                          ptr(dgate), ptr(act), act.numel() * act.element_size(), ptr(ws),
                                          ws.numel() * ws.element_size(), stream_ptr(stream)),
          "moe_layer_backward_dgrad")


def moe_layer_backward_wgrad(cfg, weights: MoeWeights, x, dy, grads: MoeGrads, act, ws, stream=None) -> None:
    check(load().moe_layer_backward_wgrad(ctypes.byref(cfg), ctypes.byref(weights), ptr(x), ptr(dy),
                                          ctypes.byref(grads), ptr(act), act.numel() * act.element_size(),
                                          ptr(ws), ws.numel() * ws.element_size(), stream_ptr(stream)),
          "moe_layer_backward_wgrad")


# ---------------------------------------------------------------- around the layer
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device() -> int:
    """The current GPU, on which a call's kernels run and its tensors have to be (-2, no tensor's, without one)."""
    try:
        return _get_device()
    except (RuntimeError, AssertionError):
        return -2


def _tensor(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on GPU `dev`; raises ValueError otherwise."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous tensor {tuple(shape)} of {dtype} on the current GPU, got "
                     f"{tuple(t.shape)} of {t.dtype} on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))


# Sizes cross the C ABI in 32 bits; ctypes would cut a larger one off without a word.
_MAX_SIZE = 2 ** 31 - 1


def _fits(size: int, name: str) -> int:
    if not -_MAX_SIZE <= size <= _MAX_SIZE:
        raise MoeError(-1, name)
    return size


def _sized(a: int, b: int, c: int = 0, d: int = 0) -> bool:
    return (-_MAX_SIZE <= a <= _MAX_SIZE and -_MAX_SIZE <= b <= _MAX_SIZE and -_MAX_SIZE <= c <= _MAX_SIZE
            and -_MAX_SIZE <= d <= _MAX_SIZE)


def _matrix(t, name: str) -> torch.Size:
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected two dimensions, got {tuple(shape)}")
    if shape[0] > _MAX_SIZE or shape[1] > _MAX_SIZE:
        raise MoeError(-1, name)
    return shape


def _scratch(ws, dev: int) -> tuple[int, int]:
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on the current GPU, got one on {ws.device}")
    nbytes = ws.numel() * ws.element_size()
    if nbytes < 256:
        raise MoeError(-4, "ws")
    return ws.data_ptr(), nbytes


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def moe_embedding_workspace_bytes(n: int, V: int, H: int) -> int:
    return int(load().moe_embedding_workspace_bytes(n, V, H)) if _sized(n, V, H) else 0


def moe_embedding_forward(tokens, table, out, ws, scale: float = 1.0, stream=None) -> None:
    """out[i] = scale * table[tokens[i]] (bf16); a zero row where tokens[i] is -1."""
    dev = _device()
    V, H = rows = _matrix(table, "table")
    n = _fits(tokens.numel(), "tokens")
    check(load().moe_embedding_forward(_tensor(tokens, "tokens", _I32, (n,), dev), n,
                                       _tensor(table, "table", _BF16, rows, dev), V, H, scale,
                                       _tensor(out, "out", _BF16, (n, H), dev), _scratch(ws, dev)[0],
                                       stream_ptr(stream, dev)),
          "moe_embedding_forward")


def moe_embedding_backward(tokens, dy, dtable, ws, scale: float = 1.0, base=None, stream=None) -> None:
    """dtable[v] = base[v] + scale * (sum of dy[i] over tokens[i] == v), fp32, every row written."""
    dev = _device()
    V, H = _matrix(dtable, "dtable")
    n = _fits(tokens.numel(), "tokens")
    wp, wn = _scratch(ws, dev)
    check(load().moe_embedding_backward(_tensor(tokens, "tokens", _I32, (n,), dev), n,
                                        _tensor(dy, "dy", _BF16, (n, H), dev), V, H, scale,
                                        None if base is None else _tensor(base, "base", _BF16, (V, H), dev),
                                        _tensor(dtable, "dtable", _F32, (V, H), dev), wp, wn, stream_ptr(stream, dev)),
          "moe_embedding_backward")


def moe_layer_norm_forward(x, weight, bias, y, mean, rstd, residual=None, sum_out=None, eps: float = 1e-5,
                           stream=None) -> None:
    """y = norm(s) * weight + bias with s = x + residual (written to sum_out); mean and rstd for the backward."""
    dev = _device()
    T, H = rows = _matrix(x, "x")
    check(load().moe_layer_norm_forward(_tensor(x, "x", _BF16, rows, dev),
                                        None if residual is None else _tensor(residual, "residual", _BF16, rows, dev),
                                        _tensor(weight, "weight", _BF16, (H,), dev),
                                        None if bias is None else _tensor(bias, "bias", _BF16, (H,), dev),
                                        T, H, eps, _tensor(y, "y", _BF16, rows, dev),
                                        None if sum_out is None else _tensor(sum_out, "sum_out", _BF16, rows, dev),
                                        _tensor(mean, "mean", _F32, (T,), dev), _tensor(rstd, "rstd", _F32, (T,), dev),
                                        stream_ptr(stream, dev)), "moe_layer_norm_forward")


def moe_layer_norm_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_layer_norm_workspace_bytes(T, H)) if _sized(T, H) else 0


def moe_layer_norm_backward(dy, s, weight, mean, rstd, dx, dweight, dbias, ws, dsum=None, stream=None) -> None:
    """dx = the gradient of s (plus dsum, the stream's own); dweight and dbias (or None), fp32."""
    dev = _device()
    T, H = rows = _matrix(s, "s")
    wp, wn = _scratch(ws, dev)
    check(load().moe_layer_norm_backward(_tensor(dy, "dy", _BF16, rows, dev), _tensor(s, "s", _BF16, rows, dev),
                                         _tensor(weight, "weight", _BF16, (H,), dev),
                                         _tensor(mean, "mean", _F32, (T,), dev), _tensor(rstd, "rstd", _F32, (T,), dev),
                                         None if dsum is None else _tensor(dsum, "dsum", _BF16, rows, dev),
                                         T, H, _tensor(dx, "dx", _BF16, rows, dev),
                                         _tensor(dweight, "dweight", _F32, (H,), dev),
                                         None if dbias is None else _tensor(dbias, "dbias", _F32, (H,), dev), wp, wn,
                                         stream_ptr(stream, dev)),
          "moe_layer_norm_backward")


def moe_cross_entropy_workspace_bytes(T: int, H: int, V: int, piece: int = 0) -> int:
    return int(load().moe_cross_entropy_workspace_bytes(T, H, V, piece)) if _sized(T, H, V, piece) else 0


def moe_cross_entropy_forward(x, w, labels, loss, lse, ws, stream=None) -> None:
    """loss[t] = lse[t] - <x[t], w[labels[t]]>, 0 where labels[t] is -1; the logits are not kept."""
    dev = _device()
    T, H = _matrix(x, "x")
    V = _matrix(w, "w")[0]
    wp, wn = _scratch(ws, dev)
    check(load().moe_cross_entropy_forward(_tensor(x, "x", _BF16, (T, H), dev), _tensor(w, "w", _BF16, (V, H), dev),
                                           _tensor(labels, "labels", _I32, (T,), dev), T, H, V,
                                           _tensor(loss, "loss", _F32, (T,), dev),
                                           _tensor(lse, "lse", _F32, (T,), dev), wp, wn, stream_ptr(stream, dev)),
          "moe_cross_entropy_forward")


def moe_cross_entropy_backward(x, w, labels, lse, dloss, dx, dw, ws, piece: int = 0, stream=None) -> None:
    """dx and dw (bf16) of sum_t dloss[t] * loss[t], `piece` vocabulary entries at a time (0: chosen by size)."""
    dev = _device()
    T, H = _matrix(x, "x")
    V = _matrix(w, "w")[0]
    wp, wn = _scratch(ws, dev)
    check(load().moe_cross_entropy_backward(_tensor(x, "x", _BF16, (T, H), dev), _tensor(w, "w", _BF16, (V, H), dev),
                                            _tensor(labels, "labels", _I32, (T,), dev),
                                            _tensor(lse, "lse", _F32, (T,), dev),
                                            _tensor(dloss, "dloss", _F32, (T,), dev), T, H, V, _fits(piece, "piece"),
                                            _tensor(dx, "dx", _BF16, (T, H), dev),
                                            _tensor(dw, "dw", _BF16, (V, H), dev), wp, wn, stream_ptr(stream, dev)),
          "moe_cross_entropy_backward")


# ---------------------------------------------------------------- attention
# moe_heads, moe_tensor and moe_attention_config cross as packed bytes: a ctypes structure takes 1 us to make.
def _heads(t, name: str, shape, dev: int) -> tuple[int, int, int]:
    """The fields of moe_heads for a [T, heads, width] bf16 tensor on GPU `dev` with a contiguous last dimension."""
    strides = t.stride()
    if t.dtype is _BF16 and t.shape == shape and t.get_device() == dev and (strides[2] == 1 or shape[2] == 1):
        return t.data_ptr(), strides[0], strides[1]
    raise ValueError(f"{name}: expected {tuple(shape)} of {_BF16} on the current GPU, its last dimension contiguous, "
                     f"got {tuple(t.shape)} of {t.dtype} on {t.device}, strides {strides}")


def _attention(q, k, cu_seqlens, scale):
    """Bytes of the config, number of sequences, shapes of q and of k and v."""
    if len(q.shape) != 3 or len(k.shape) != 3:
        raise ValueError(f"q, k: expected three dimensions, got {tuple(q.shape)} and {tuple(k.shape)}")
    T, Hq, D = q.shape
    Hkv, n = k.shape[1], cu_seqlens.numel() - 1
    if n < 0:
        raise ValueError("cu_seqlens: expected the sequences' first rows and the last one's end")
    if not (_sized(T, Hq, Hkv, D) and n <= _MAX_SIZE):
        raise MoeError(-1, "q, k, cu_seqlens")
    if scale is None:
        scale = D ** -0.5 if D > 0 else 1.0
    elif not abs(scale) < 2.0 ** 127:         # (struct has no fp32 form of more, the call none of 2^65)
        raise MoeError(-1, "scale")
    return struct.pack("5if", T, n, Hq, Hkv, D, scale), n, (T, Hq, D), (T, Hkv, D)


def moe_attention_workspace_bytes(T: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    if not _sized(T, q_heads, kv_heads, head_dim):
        return 0
    return load().moe_attention_workspace_bytes(struct.pack("5if", T, 1, q_heads, kv_heads, head_dim, 1.0))


def moe_attention_forward(q, k, v, cu_seqlens, out, lse, ws, scale: float | None = None, stream=None) -> None:
    """Causal attention of each packed sequence; lse for the backward pass.

    q, out [T, q_heads, D] and k, v [T, kv_heads, D] bf16 in any strides; cu_seqlens int32, the sequences' first
    rows and the last one's end; lse [q_heads, T] fp32; scale 1/sqrt(D) unless given.
    """
    dev = _device()
    cfg, n, sq, sk = _attention(q, k, cu_seqlens, scale)
    wp, wn = _scratch(ws, dev)
    heads = array.array("q", _heads(q, "q", sq, dev) + _heads(k, "k", sk, dev) + _heads(v, "v", sk, dev)
                        + _heads(out, "out", sq, dev))
    at = heads.buffer_info()[0]
    check(load().moe_attention_forward(cfg, at, at + 24, at + 48, _tensor(cu_seqlens, "cu_seqlens", _I32, (n + 1,), dev),
                                       at + 72, _tensor(lse, "lse", _F32, (sq[1], sq[0]), dev), wp, wn,
                                       stream_ptr(stream, dev)), "moe_attention_forward")


def moe_attention_backward(q, k, v, cu_seqlens, out, lse, dout, dq, dk, dv, ws, scale: float | None = None,
                           stream=None) -> None:
    """dq, dk, dv of sum <dout, out>; q, k, v, out, lse (and scale) as in the forward call."""
    dev = _device()
    cfg, n, sq, sk = _attention(q, k, cu_seqlens, scale)
    wp, wn = _scratch(ws, dev)
    heads = array.array("q", _heads(q, "q", sq, dev) + _heads(k, "k", sk, dev) + _heads(v, "v", sk, dev)
                        + _heads(out, "out", sq, dev) + _heads(dout, "dout", sq, dev) + _heads(dq, "dq", sq, dev)
                        + _heads(dk, "dk", sk, dev) + _heads(dv, "dv", sk, dev))
    at = heads.buffer_info()[0]
    check(load().moe_attention_backward(cfg, at, at + 24, at + 48, _tensor(cu_seqlens, "cu_seqlens", _I32, (n + 1,), dev),
                                        at + 72, _tensor(lse, "lse", _F32, (sq[1], sq[0]), dev), at + 96, at + 120,
                                        at + 144, at + 168, wp, wn, stream_ptr(stream, dev)),
          "moe_attention_backward")


def moe_rotary_frequencies(R: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                           original_length: int = 0, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(freq, scale) for moe_rotary: the angle per position of each pair (fp64, on `device`), the values' factor."""
    if not _sized(R, original_length):
        raise MoeError(-1, "moe_rotary_frequencies")
    freq, scale = (c_f64 * max(R // 2, 1))(), c_f32(1.0)
    check(load().moe_rotary_frequencies(R, base, ROTARY_SCALING[scaling], factor, original_length, fast, slow, freq,
                                        ctypes.byref(scale)), "moe_rotary_frequencies")
    return torch.tensor(list(freq), dtype=torch.float64, device=device), scale.value


def moe_rotary(x, positions, freq, out, interleaved: bool = False, scale: float = 1.0, inverse: bool = False,
               stream=None) -> None:
    """out = the first 2 len(freq) values of every head of x turned by positions * freq, the others copied.

    x, out [T, heads, width] bf16 in any strides (out may be x); inverse: by the negative angles, the gradient.
    """
    dev = _device()
    if len(x.shape) != 3:
        raise ValueError(f"x: expected three dimensions, got {tuple(x.shape)}")
    T, heads, width = shape = x.shape
    pairs = freq.numel()
    if not _sized(T, heads, width, 2 * pairs):
        raise MoeError(-1, "x, freq")
    both = array.array("q", _heads(x, "x", shape, dev) + _heads(out, "out", shape, dev))
    at = both.buffer_info()[0]
    check(load().moe_rotary(at, _tensor(positions, "positions", _I32, (T,), dev),
                            _tensor(freq, "freq", torch.float64, (pairs,), dev), T, heads, width, 2 * pairs,
                            1 if interleaved else 0, scale, 1 if inverse else 0, at + 24, stream_ptr(stream, dev)),
          "moe_rotary")


# ---------------------------------------------------------------- balance loss
def moe_balance_loss_workspace_bytes(T: int, E: int) -> int:
    return int(load().moe_balance_loss_workspace_bytes(T, E)) if _sized(T, E) else 0


def moe_balance_loss_forward(logits, topk_idx, loss, counts, slope, ws, tokens=None, score: str = "softmax",
                             stream=None) -> None:
    """loss [1] of the router's choices topk_idx [T, k] among logits [T, E]; counts [E] per expert; slope [E] for
    the backward.  tokens [T]: rows below 0 are padding."""
    dev = _device()
    T, E = _matrix(logits, "logits")
    k = _matrix(topk_idx, "topk_idx")[1]
    wp, wn = _scratch(ws, dev)
    check(load().moe_balance_loss_forward(_tensor(logits, "logits", _F32, (T, E), dev),
                                          _tensor(topk_idx, "topk_idx", _I32, (T, k), dev),
                                          None if tokens is None else _tensor(tokens, "tokens", _I32, (T,), dev),
                                          T, E, k, SCORE[score], _tensor(loss, "loss", _F32, (1,), dev),
                                          _tensor(counts, "counts", _I32, (E,), dev),
                                          _tensor(slope, "slope", _F32, (E,), dev), wp, wn, stream_ptr(stream, dev)),
          "moe_balance_loss_forward")


def moe_balance_loss_backward(logits, slope, dloss, dlogits, tokens=None, score: str = "softmax", stream=None) -> None:
    """dlogits [T, E] of dloss[0] times the loss; zero rows for padding."""
    dev = _device()
    T, E = rows = _matrix(logits, "logits")
    check(load().moe_balance_loss_backward(_tensor(logits, "logits", _F32, rows, dev),
                                           _tensor(slope, "slope", _F32, (E,), dev),
                                           None if tokens is None else _tensor(tokens, "tokens", _I32, (T,), dev),
                                           T, E, SCORE[score], _tensor(dloss, "dloss", _F32, (1,), dev),
                                           _tensor(dlogits, "dlogits", _F32, rows, dev), stream_ptr(stream, dev)),
          "moe_balance_loss_backward")


# ---------------------------------------------------------------- gradient norm
def _tensors(ts, name: str, dev: int) -> array.array:
    """moe_tensor of each contiguous bf16 or fp32 tensor on GPU `dev`, as 64-bit words (the type in the low half)."""
    words = []
    for t in ts:
        dtype = t.dtype
        if (dtype is not _F32 and dtype is not _BF16) or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous tensors of {_F32} or {_BF16} on the current GPU, got one of "
                             f"{dtype} on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))
        words += (t.data_ptr(), t.numel(), 1 if dtype is _F32 else 0)
    return array.array("q", words)


def moe_grad_norm_workspace_bytes(n: int) -> int:
    return int(load().moe_grad_norm_workspace_bytes(n)) if _sized(n, 0) else 0


def moe_grad_norm(grads, norm, ws, stream=None) -> None:
    """norm [1] = the 2-norm of all tensors of the list (bf16 or fp32) together."""
    dev = _device()
    wp, wn = _scratch(ws, dev)
    words = _tensors(grads, "grads", dev)
    check(load().moe_grad_norm(words.buffer_info()[0], len(grads), _tensor(norm, "norm", _F32, (1,), dev), wp, wn,
                               stream_ptr(stream, dev)), "moe_grad_norm")


def moe_grad_clip(grads, norm, limit: float, outs=None, stream=None) -> None:
    """Every tensor times min(1, limit / (norm + 1e-6)), in place or into outs (tensors of the same sizes and types)."""
    dev = _device()
    words = _tensors(grads, "grads", dev)
    to = None if outs is None else _tensors(outs, "outs", dev)
    if to is not None and (to[1::3] != words[1::3] or to[2::3] != words[2::3]):
        raise ValueError("outs: expected as many tensors as the gradients, of the same sizes and types")
    check(load().moe_grad_clip(words.buffer_info()[0], None if to is None else to.buffer_info()[0], len(grads),
                               _tensor(norm, "norm", _F32, (1,), dev), limit, stream_ptr(stream, dev)), "moe_grad_clip")


# ---------------------------------------------------------------- buffers
class MoELayer:
    """Device buffers for one layer shape (weights are the caller's tensors).

    Owns the activation buffer and the workspace (torch.uint8 device tensors)
    and exposes views of the activation fields for inspection.
    """

    def __init__(self, cfg: MoeConfig, weights: dict, with_backward: bool = False, device="cuda"):
        self.cfg = cfg
        self.with_backward = with_backward
        self.w = weights
        self.layout = moe_activation_layout(cfg, with_backward)
        self.act = torch.empty(self.layout.total, dtype=torch.uint8, device=device)
        self.ws = torch.zeros(max(moe_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)
        moe_workspace_init(self.ws)
        self.cw = MoeWeights(ptr(weights["w_router"]), ptr(weights.get("bias")), ptr(weights["w1"]),
                             ptr(weights["w2"]), ptr(weights.get("w1_shared")), ptr(weights.get("w2_shared")),
                             None)
        self.mx = None
        if cfg.dtype == GEMM_DTYPE["mxfp8"]:
            self.mx = torch.empty(moe_mxfp8_weights_bytes(cfg), dtype=torch.uint8, device=device)
        elif cfg.dtype == GEMM_DTYPE["nvfp4"]:
            self.mx = torch.empty(moe_nvfp4_weights_bytes(cfg), dtype=torch.uint8, device=device)
        if self.mx is not None:
            self.cw.mx = ptr(self.mx)
            self.prepare_weights()

    def prepare_weights(self, stream=None) -> None:
        """(MXFP8 / NVFP4) quantise the weights into the layer's buffer; call after a weight update."""
        if self.cfg.dtype == GEMM_DTYPE["nvfp4"]:
            moe_prepare_nvfp4_weights(self.cfg, self.cw, self.mx, stream)
        else:
            moe_prepare_mxfp8_weights(self.cfg, self.cw, self.mx, stream)

    def view(self, name: str, dtype, shape) -> torch.Tensor:
        off = getattr(self.layout, name)
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.act[off:off + nbytes].view(dtype).view(*shape)

    def fields(self) -> dict:
        c = self.cfg
        cap = self.layout.cap
        d = {
            "logits": self.view("logits", torch.float32, (c.T, c.E)),
            "topk_idx": self.view("topk_idx", torch.int32, (c.T, c.k)),
            "topk_gate": self.view("topk_gate", torch.float32, (c.T, c.k)),
            "counts": self.view("counts", torch.int32, (c.E,)),
            "offsets": self.view("offsets", torch.int32, (c.E + 1,)),
            "poffsets": self.view("poffsets", torch.int32, (c.E + 1,)),
            "slot_row": self.view("slot_row", torch.int32, (c.T, c.k)),
            "row_src": self.view("row_src", torch.int32, (cap,)),
            "row_gate": self.view("row_gate", torch.float32, (cap,)),
            "x_perm": self.view("x_perm", torch.bfloat16, (cap, c.H)),
            "z": self.view("z", torch.bfloat16, (cap, 2 * c.F)),
            "h": self.view("h", torch.bfloat16, (cap, c.F)),
            "o": self.view("o", torch.bfloat16, (cap, c.H)),
        }
        if self.with_backward:
            d.update({
                "dy_perm": self.view("dy_perm", torch.bfloat16, (cap, c.H)),
                "dz": self.view("dz", torch.bfloat16, (cap, 2 * c.F)),
                "dx_perm": self.view("dx_perm", torch.bfloat16, (cap, c.H)),
                "dlogits": self.view("dlogits", torch.float32, (c.T, c.E)),
            })
        return d

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if y is None:
            y = torch.empty_like(x)
        moe_layer_forward(self.cfg, self.cw, x, y, self.act, self.with_backward, self.ws, stream)
        return y

    def backward(self, x, dy, grads: dict | None = None, dx=None, dgate=None, stream=None):
        c = self.cfg
        dev = x.device
        if dx is None:
            dx = torch.empty_like(x)
        if dgate is None:
            dgate = torch.empty((c.T, c.k), dtype=torch.float32, device=dev)
        if grads is None:
            grads = {"dw_router": torch.empty((c.E, c.H), dtype=torch.float32, device=dev),
                     "dw1": torch.empty((c.E, 2 * c.F, c.H), dtype=torch.float32, device=dev),
                     "dw2": torch.empty((c.E, c.H, c.F), dtype=torch.float32, device=dev)}
            if c.S > 0:
                grads["dw1_shared"] = torch.empty((2 * c.S, c.H), dtype=torch.float32, device=dev)
                grads["dw2_shared"] = torch.empty((c.H, c.S), dtype=torch.float32, device=dev)
        moe_layer_backward_dgrad(c, self.cw, x, dy, dx, dgate, self.act, self.ws, stream)
        g = MoeGrads(ptr(grads["dw_router"]), ptr(grads["dw1"]), ptr(grads["dw2"]), ptr(grads.get("dw1_shared")),
                     ptr(grads.get("dw2_shared")))
        moe_layer_backward_wgrad(c, self.cw, x, dy, g, self.act, self.ws, stream)
        return dx, dgate, grads


def moe_debug_set_wait_limit_ns(ns: int) -> None:
    """Test hook: the grouped GEMMs' pipeline waits give up after ns (0: 2 s)."""
    load().moe_debug_set_wait_limit_ns(int(ns))


def moe_kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().moe_kernel_launches())


def moe_status_string(code: int) -> str:
    return load().moe_status_string(int(code)).decode()


def moe_version() -> int:
    return int(load().moe_version())
