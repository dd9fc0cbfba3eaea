"""Python binding of libmoe_gb300.so, the GB300 (sm_103a) routed MoE FFN forward.

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  Functions carry the C ABI's names (include/moe.h) and take
torch CUDA tensors for device memory (plus the current torch stream by
default); each raises MoeError when the library returns a non-OK status.

The library must have been built (``build.build()`` or
``__graft_entry__.build()``); the first call into it raises RuntimeError if it
is missing - there is no other implementation to fall back on.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_gb300.so")

# moe_status
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_ERR_DEVICE_BOUNDS = 6
# moe_quant
MOE_BF16 = 0
MOE_FP8_PER_TENSOR = 1
MOE_FP8_BLOCK128 = 2
MOE_MXFP8 = 3
# moe_path
MOE_PATH_AUTO = 0
MOE_PATH_GROUPED = 1
MOE_PATH_ROUTE_DIRECT = 2

# moe_dtype
MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_F16 = 2
MOE_DTYPE_E4M3 = 3
# moe_score_fn
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
# moe_norm_kind
MOE_NORM_NONE = 0
MOE_NORM_RMS = 1
MOE_NORM_LAYER = 2
# moe_gate_kind
MOE_GATE_NONE = 0
MOE_GATE_CHANNEL = 1
MOE_GATE_TOKEN = 2
MOE_GATE_FULL = 3
# moe_act
MOE_ACT_NONE = 0
MOE_ACT_RELU = 1
MOE_ACT_SILU = 2
MOE_ACT_GELU = 3
MOE_ACT_GELU_TANH = 4

QUANT_BY_NAME = {"bf16": MOE_BF16, "fp8_tensor": MOE_FP8_PER_TENSOR, "fp8_block": MOE_FP8_BLOCK128,
                 "mxfp8": MOE_MXFP8}
GEMM_BM = 128  # row-tile height of the grouped GEMMs (tile map of moe_forward)


class moe_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int), ("H", ctypes.c_int),
                ("I", ctypes.c_int), ("quant", ctypes.c_int), ("path", ctypes.c_int)]


class moe_views(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("ids", "w", "counts", "offsets", "perm", "inv", "tiles", "num_tiles", "xs", "x_scale",
                 "amax_x")]


class moe_forward_options(ctypes.Structure):
    _fields_ = [("n_shared", ctypes.c_int), ("w1_shared", ctypes.c_void_p), ("w2_shared", ctypes.c_void_p),
                ("w1_shared_scale", ctypes.c_void_p), ("w2_shared_scale", ctypes.c_void_p), ("y_fp32", ctypes.c_int),
                ("mx_weight_scales_blocked", ctypes.c_int)]


class moe_stage_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("total_ms", ctypes.c_double), ("launches", ctypes.c_int)]


_vp, _sz, _i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_ll, _f = ctypes.c_longlong, ctypes.c_float


class moe_route_options(ctypes.Structure):
    _fields_ = [("score_fn", _i), ("renormalise", _i), ("scale", _f), ("n_group", _i), ("topk_group", _i),
                ("group_best", _i), ("bias", _vp), ("dtype", _i), ("ld", _ll), ("ld_grad", _ll)]


class moe_norm_problem(ctypes.Structure):
    _fields_ = [("T", _i), ("H", _i), ("post_norm", _i), ("pre_norm", _i), ("gate", _i), ("h_dtype", _i),
                ("o_dtype", _i), ("w_dtype", _i), ("eps", _f), ("alpha", _f), ("beta", _f), ("ld_h", _ll),
                ("ld_o", _ll)]


class moe_linear_problem(ctypes.Structure):
    _fields_ = [("M", _i), ("N", _i), ("K", _i), ("dtype", _i), ("out_dtype", _i), ("bias_dtype", _i), ("act", _i),
                ("alpha", _f), ("ld_x", _ll), ("ld_w", _ll), ("ld_y", _ll)]


class moe_gated_problem(ctypes.Structure):
    _fields_ = [("M", _i), ("N", _i), ("K", _i), ("dtype", _i), ("out_dtype", _i), ("bias_dtype", _i), ("act", _i),
                ("ld_x", _ll), ("ld_w", _ll), ("ld_h", _ll)]


class moe_quantise_problem(ctypes.Structure):
    _fields_ = [("M", _i), ("K", _i), ("dtype", _i), ("block_rows", _i), ("ld_x", _ll), ("ld_q", _ll)]


_P = ctypes.POINTER(moe_problem)
_O = ctypes.POINTER(moe_forward_options)
_RO = ctypes.POINTER(moe_route_options)
_NP = ctypes.POINTER(moe_norm_problem)
_LP = ctypes.POINTER(moe_linear_problem)
_GP = ctypes.POINTER(moe_gated_problem)
_QP = ctypes.POINTER(moe_quantise_problem)
_SIGS = {
    "moe_route": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp]),
    "moe_shuffle_workspace_size": (_sz, [_i, _i, _i]),
    "moe_shuffle": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_shuffle_noalloc": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "moe_tile_map": (_i, [_vp, _i, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "moe_select_path": (_i, [_P]),
    "moe_workspace_size": (_sz, [_P]),
    "moe_forward": (_i, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_forward_views": (_i, [_P, _vp, _sz, ctypes.POINTER(moe_views)]),
    "moe_workspace_size_ex": (_sz, [_P, _O]),
    "moe_forward_ex": (_i, [_P, _O, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_forward_routed": (_i, [_P, _O, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_forward_views_ex": (_i, [_P, _O, _vp, _sz, ctypes.POINTER(moe_views)]),
    "moe_round_bf16": (_i, [_vp, _vp, _sz, _vp]),
    "moe_mx_blocked_bytes": (_sz, [_i, _i, _i]),
    "moe_mx_weight_scales_bytes": (_sz, [_i, _i, _i, _i]),
    "moe_mx_weight_scales": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
    "moe_mx_blocked_workspace_size": (_sz, [_i, _i]),
    "moe_mx_blocked_scales": (_i, [_vp, _i, _i, _vp, _i, _vp, _sz, _vp, _vp, _sz, _vp]),
    "moe_route_ex": (_i, [_RO, _vp, _i, _i, _i, _vp, _vp, _vp]),
    "moe_route_backward": (_i, [_RO, _vp, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "moe_norm_forward": (_i, [_NP] + [_vp] * 10),
    "moe_norm_backward_workspace_size": (_sz, [_NP]),
    "moe_norm_backward": (_i, [_NP] + [_vp] * 16 + [_sz, _vp]),
    "moe_linear_workspace_size": (_sz, [_LP]),
    "moe_linear": (_i, [_LP] + [_vp] * 7 + [_sz, _vp]),
    "moe_linear_backward_workspace_size": (_sz, [_LP]),
    "moe_linear_backward": (_i, [_LP] + [_vp] * 8 + [_sz, _vp]),
    "moe_gated_workspace_size": (_sz, [_GP]),
    "moe_gated": (_i, [_GP] + [_vp] * 6 + [_sz, _vp]),
    "moe_gated_backward_workspace_size": (_sz, [_GP]),
    "moe_gated_backward": (_i, [_GP] + [_vp] * 8 + [_sz, _vp]),
    "moe_quantise": (_i, [_QP] + [_vp] * 4),
    "moe_linear_fp8_workspace_size": (_sz, [_LP]),
    "moe_linear_fp8": (_i, [_LP] + [_vp] * 8 + [_sz, _vp]),
    "moe_gated_fp8_workspace_size": (_sz, [_GP]),
    "moe_gated_fp8": (_i, [_GP] + [_vp] * 8 + [_sz, _vp]),
    "moe_read_device_status": (_i, [_vp, _vp]),
    "moe_profile_start": (_i, []),
    "moe_profile_start_stage": (_i, [ctypes.c_char_p]),
    "moe_profile_stop": (_i, [ctypes.POINTER(moe_stage_time), _i]),
    "moe_status_string": (ctypes.c_char_p, [_i]),
}
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with mixture_experts_layer_index_gb300.build.build() "
                "(the CUDA library is the only implementation)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(handle, name)
            f.restype = res
            f.argtypes = args
        _lib = handle
    return _lib


EXPORTED = tuple(_SIGS)


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {moe_status_string(status)} (status {status})")


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t) -> Optional[int]:
    """Device pointer of a contiguous CUDA tensor (None -> NULL; ints pass through)."""
    if t is None or type(t) is int:
        return t
    try:
        on_device = t.is_cuda
    except AttributeError:
        if isinstance(t, int):  # its subclasses
            return int(t)
        raise
    if not on_device:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


_current_stream = None  # the raw handle of the current device's current stream


def _find_current_stream():
    global _current_stream
    import torch

    device = torch.cuda.current_device  # starts CUDA, or raises where there is none
    device()
    # the Stream object that torch.cuda.current_stream() builds around the handle costs more than a
    # small launch (2.9 us; the handle alone 0.2)
    device, handle = getattr(torch._C, "_cuda_getDevice", device), torch._C._cuda_getCurrentRawStream
    _current_stream = lambda: handle(device())  # noqa: E731


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _current_stream is None:
            _find_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def problem(T: int, E: int, k: int, H: int, I: int, quant=MOE_BF16, path=MOE_PATH_AUTO) -> moe_problem:
    if isinstance(quant, str):
        quant = QUANT_BY_NAME[quant]
    return moe_problem(T, E, k, H, I, int(quant), int(path))


def moe_route(scores, T, E, k, ids, w, stream=None) -> None:
    _check(lib().moe_route(_ptr(scores), T, E, k, _ptr(ids), _ptr(w), _stream(stream)), "moe_route")


def moe_shuffle_workspace_size(T, E, k) -> int:
    return int(lib().moe_shuffle_workspace_size(T, E, k))


def moe_shuffle(ids, T, E, k, counts, offsets, perm, inv, ws, ws_bytes=None, stream=None) -> None:
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_shuffle(_ptr(ids), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(ws), nb,
                            _stream(stream)), "moe_shuffle")


def moe_shuffle_noalloc(ids, T, E, k, counts, offsets, perm, inv, stream=None) -> None:
    """moe_shuffle with the library's fixed scratch array instead of a workspace
    (for callers that cannot allocate device memory; see include/moe.h)."""
    _check(lib().moe_shuffle_noalloc(_ptr(ids), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                                     _stream(stream)), "moe_shuffle_noalloc")


def moe_tile_map(counts, E, BM, tiles, num_tiles, max_tiles, ws, ws_bytes=None, stream=None) -> None:
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_tile_map(_ptr(counts), E, BM, _ptr(tiles), _ptr(num_tiles), max_tiles, _ptr(ws), nb,
                             _stream(stream)), "moe_tile_map")


def moe_select_path(p: moe_problem) -> int:
    return int(lib().moe_select_path(ctypes.byref(p)))


def moe_workspace_size(p: moe_problem) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(p)))


def moe_forward(p: moe_problem, x, scores, w1, w2, w1_scale, w2_scale, y, ws, ws_bytes=None, stream=None) -> None:
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_forward(ctypes.byref(p), _ptr(x), _ptr(scores), _ptr(w1), _ptr(w2), _ptr(w1_scale),
                            _ptr(w2_scale), _ptr(y), _ptr(ws), nb, _stream(stream)), "moe_forward")


def forward_options(n_shared=0, w1_shared=None, w2_shared=None, w1_shared_scale=None, w2_shared_scale=None,
                    y_fp32=False, mx_weight_scales_blocked=False) -> moe_forward_options:
    return moe_forward_options(int(n_shared), _ptr(w1_shared), _ptr(w2_shared), _ptr(w1_shared_scale),
                               _ptr(w2_shared_scale), 1 if y_fp32 else 0, 1 if mx_weight_scales_blocked else 0)


def _opt_ref(opt):
    return None if opt is None else ctypes.byref(opt)


def moe_workspace_size_ex(p: moe_problem, opt: Optional[moe_forward_options]) -> int:
    return int(lib().moe_workspace_size_ex(ctypes.byref(p), _opt_ref(opt)))


def moe_forward_ex(p: moe_problem, opt: Optional[moe_forward_options], x, scores, w1, w2, w1_scale, w2_scale, y, ws,
                   ws_bytes=None, stream=None) -> None:
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_forward_ex(ctypes.byref(p), _opt_ref(opt), _ptr(x), _ptr(scores), _ptr(w1), _ptr(w2),
                               _ptr(w1_scale), _ptr(w2_scale), _ptr(y), _ptr(ws), nb, _stream(stream)),
           "moe_forward_ex")


def moe_forward_routed(p: moe_problem, opt: Optional[moe_forward_options], x, ids, w, w1, w2, w1_scale, w2_scale, y,
                       ws, ws_bytes=None, stream=None) -> None:
    """moe_forward_ex with a given routing (ids, w), e.g. of moe_route_ex."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_forward_routed(ctypes.byref(p), _opt_ref(opt), _ptr(x), _ptr(ids), _ptr(w), _ptr(w1), _ptr(w2),
                                    _ptr(w1_scale), _ptr(w2_scale), _ptr(y), _ptr(ws), nb, _stream(stream)),
           "moe_forward_routed")


def moe_forward_views_ex(p: moe_problem, opt: Optional[moe_forward_options], ws, ws_bytes=None) -> moe_views:
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    v = moe_views()
    _check(lib().moe_forward_views_ex(ctypes.byref(p), _opt_ref(opt), _ptr(ws), nb, ctypes.byref(v)),
           "moe_forward_views_ex")
    return v


def moe_round_bf16(y32, y, n=None, stream=None) -> None:
    n = y32.numel() if n is None else n
    _check(lib().moe_round_bf16(_ptr(y32), _ptr(y), n, _stream(stream)), "moe_round_bf16")


def moe_mx_weight_scales_bytes(E: int, H: int, I: int, which: int) -> int:
    return int(lib().moe_mx_weight_scales_bytes(E, H, I, which))


def moe_mx_weight_scales(w1_scale, w2_scale, E, H, I, w1_blocked, w2_blocked, stream=None) -> None:
    """MXFP8 weight scales converted once into the forward's blocked layouts."""
    _check(lib().moe_mx_weight_scales(_ptr(w1_scale), _ptr(w2_scale), E, H, I, _ptr(w1_blocked), _ptr(w2_blocked),
                                     _stream(stream)), "moe_mx_weight_scales")


def moe_mx_blocked_bytes(rows: int, cols: int, groups: int) -> int:
    return int(lib().moe_mx_blocked_bytes(rows, cols, groups))


def moe_mx_blocked_workspace_size(rows: int, groups: int) -> int:
    return int(lib().moe_mx_blocked_workspace_size(rows, groups))


def moe_mx_blocked_scales(scales, rows, cols, group_offsets, groups, out, group_starts, ws, out_bytes=None,
                          ws_bytes=None, stream=None) -> None:
    """Per-group blocked layout of MX scales (see include/moe.h)."""
    ob = out.numel() * out.element_size() if out_bytes is None else out_bytes
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_mx_blocked_scales(_ptr(scales), rows, cols, _ptr(group_offsets), groups, _ptr(out), ob,
                                      _ptr(group_starts), _ptr(ws), nb, _stream(stream)), "moe_mx_blocked_scales")


def moe_forward_views(p: moe_problem, ws, ws_bytes=None) -> moe_views:
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    v = moe_views()
    _check(lib().moe_forward_views(ctypes.byref(p), _ptr(ws), nb, ctypes.byref(v)), "moe_forward_views")
    return v


def _rows(t, name: str, width: int, ld: int = 0) -> Optional[int]:
    """Device pointer of a CUDA tensor of rows of `width` values, `ld` elements apart (0: `width`) as the
    descriptor says; None -> NULL; ints pass through."""
    if t is None or type(t) is int:
        return t
    try:
        on_device = t.is_cuda
    except AttributeError:
        if isinstance(t, int):  # its subclasses
            return int(t)
        raise
    if not on_device:
        raise ValueError(f"{name}: device tensor expected")
    if not t.is_contiguous() or (ld != 0 and ld != width):
        _check_rows(t, name, ld or width)
    return t.data_ptr()


def _check_rows(t, name: str, ld: int) -> None:
    """Rows of t lie ld elements apart (over all its leading dimensions; a 1-D tensor is taken as it is)."""
    shape, stride = t.shape, t.stride()
    if 0 in shape:
        return
    if len(shape) and shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n > 1 and s != ld:
            raise ValueError(f"{name}: rows lie {s} elements apart, the descriptor says {ld}")
        ld *= n


def route_options(score="softmax", bias=None, n_group=1, topk_group=1, group_best=1, renormalise=True, scale=1.0,
                  dtype=MOE_DTYPE_F32, ld=0, ld_grad=0) -> moe_route_options:
    """Routing rule of moe_route_ex (see include/moe.h).  The bias tensor must outlive the options."""
    fn = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}[score] if isinstance(score, str) else int(score)
    return moe_route_options(fn, 1 if renormalise else 0, float(scale), int(n_group), int(topk_group),
                             int(group_best), _ptr(bias), int(dtype), int(ld), int(ld_grad))


def moe_route_ex(opt: moe_route_options, scores, T, E, k, ids, w, stream=None) -> None:
    """Routing with a score function, selection bias, expert groups and renormalised weights."""
    _check(lib().moe_route_ex(opt, _rows(scores, "scores", E, opt.ld), T, E, k, _ptr(ids), _ptr(w), _stream(stream)), "moe_route_ex")


def moe_route_backward(opt: moe_route_options, scores, T, E, k, ids, dw, dscores, stream=None) -> None:
    """Gradient of moe_route_ex's weights into the scores."""
    _check(lib().moe_route_backward(opt, _rows(scores, "scores", E, opt.ld), T, E, k, _ptr(ids), _ptr(dw),
                                    _rows(dscores, "dscores", E, opt.ld_grad), _stream(stream)), "moe_route_backward")


def norm_problem(T, H, post_norm=MOE_NORM_RMS, pre_norm=MOE_NORM_RMS, gate=MOE_GATE_NONE, h_dtype=MOE_DTYPE_BF16,
                 o_dtype=MOE_DTYPE_BF16, w_dtype=MOE_DTYPE_F32, eps=1e-6, alpha=1.0, beta=1.0, ld_h=0,
                 ld_o=0) -> moe_norm_problem:
    return moe_norm_problem(T, H, post_norm, pre_norm, gate, h_dtype, o_dtype, w_dtype, eps, alpha, beta, ld_h, ld_o)


def _gate(p: moe_norm_problem, t, name: str) -> Optional[int]:
    """A gate or its gradient: rows like o's, or a vector."""
    return _rows(t, name, p.H, p.ld_o) if p.gate == MOE_GATE_FULL else _ptr(t)


def moe_norm_forward(p: moe_norm_problem, h, o, gate, w_post, b_post, w_pre, b_pre, h_out, x_out,
                     stream=None) -> None:
    """h_out = beta h + alpha gate N_post(o), x_out = N_pre(h_out)."""
    H, ld_h, ld_o = p.H, p.ld_h, p.ld_o
    _check(lib().moe_norm_forward(p, _rows(h, "h", H, ld_h), _rows(o, "o", H, ld_o), _gate(p, gate, "gate"),
                                  _ptr(w_post), _ptr(b_post), _ptr(w_pre), _ptr(b_pre),
                                  _rows(h_out, "h_out", H, ld_h), _rows(x_out, "x_out", H, ld_o), _stream(stream)),
           "moe_norm_forward")


def moe_norm_backward_workspace_size(p: moe_norm_problem) -> int:
    return int(lib().moe_norm_backward_workspace_size(p))


def moe_norm_backward(p: moe_norm_problem, dh_out, dx_out, h_out, o, gate, w_post, b_post, w_pre, dh, d_o, dgate,
                      dw_post, db_post, dw_pre, db_pre, ws, ws_bytes=None, stream=None) -> None:
    """Gradient of moe_norm_forward; outputs given as None are left out."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    H, ld_h, ld_o = p.H, p.ld_h, p.ld_o
    _check(lib().moe_norm_backward(p, _rows(dh_out, "dh_out", H, ld_h), _rows(dx_out, "dx_out", H, ld_o),
                                   _rows(h_out, "h_out", H, ld_h), _rows(o, "o", H, ld_o), _gate(p, gate, "gate"),
                                   _ptr(w_post), _ptr(b_post), _ptr(w_pre), _rows(dh, "dh", H, ld_h),
                                   _rows(d_o, "d_o", H, ld_o), _gate(p, dgate, "dgate"), _ptr(dw_post), _ptr(db_post),
                                   _ptr(dw_pre), _ptr(db_pre), _ptr(ws), nb, _stream(stream)), "moe_norm_backward")


def linear_problem(M, N, K, dtype=MOE_DTYPE_BF16, out_dtype=MOE_DTYPE_BF16, bias_dtype=MOE_DTYPE_F32,
                   act=MOE_ACT_NONE, alpha=1.0, ld_x=0, ld_w=0, ld_y=0) -> moe_linear_problem:
    return moe_linear_problem(M, N, K, dtype, out_dtype, bias_dtype, act, alpha, ld_x, ld_w, ld_y)


def moe_linear_workspace_size(p: moe_linear_problem) -> int:
    return int(lib().moe_linear_workspace_size(p))


def moe_linear(p: moe_linear_problem, x, w, bias, residual, y, z, ws, ws_bytes=None, stream=None) -> None:
    """y = alpha act(x w^T + bias) + residual; z keeps the pre-activation."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    N, K, ld_y = p.N, p.K, p.ld_y
    _check(lib().moe_linear(p, _rows(x, "x", K, p.ld_x), _rows(w, "w", K, p.ld_w), _ptr(bias),
                            _rows(residual, "residual", N, ld_y), _rows(y, "y", N, ld_y), _ptr(z), _ptr(ws), nb,
                            _stream(stream)), "moe_linear")


def moe_linear_backward_workspace_size(p: moe_linear_problem) -> int:
    return int(lib().moe_linear_backward_workspace_size(p))


def moe_linear_backward(p: moe_linear_problem, dy, x, w, z, dx, dw, dbias, ws, ws_bytes=None, stream=None) -> None:
    """Gradient of moe_linear; outputs given as None are left out."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    K = p.K
    _check(lib().moe_linear_backward(p, _rows(dy, "dy", p.N, p.ld_y), _rows(x, "x", K, p.ld_x), _rows(w, "w", K, p.ld_w),
                                     _ptr(z), _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(ws), nb, _stream(stream)),
           "moe_linear_backward")


def gated_problem(M, N, K, dtype=MOE_DTYPE_BF16, out_dtype=MOE_DTYPE_BF16, bias_dtype=MOE_DTYPE_F32, act=MOE_ACT_SILU,
                  ld_x=0, ld_w=0, ld_h=0) -> moe_gated_problem:
    return moe_gated_problem(M, N, K, dtype, out_dtype, bias_dtype, act, ld_x, ld_w, ld_h)


def moe_gated_workspace_size(p: moe_gated_problem) -> int:
    return int(lib().moe_gated_workspace_size(p))


def moe_gated(p: moe_gated_problem, x, w, bias, h, z, ws, ws_bytes=None, stream=None) -> None:
    """h = act(g) u for [g, u] = x w^T + bias, N gate rows and N up rows in w; z keeps [g, u]."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    K = p.K
    _check(lib().moe_gated(p, _rows(x, "x", K, p.ld_x), _rows(w, "w", K, p.ld_w), _ptr(bias), _rows(h, "h", p.N, p.ld_h),
                           _ptr(z), _ptr(ws), nb, _stream(stream)), "moe_gated")


def moe_gated_backward_workspace_size(p: moe_gated_problem) -> int:
    return int(lib().moe_gated_backward_workspace_size(p))


def moe_gated_backward(p: moe_gated_problem, dh, x, w, z, dx, dw, dbias, ws, ws_bytes=None, stream=None) -> None:
    """Gradient of moe_gated; outputs given as None are left out."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    K = p.K
    _check(lib().moe_gated_backward(p, _rows(dh, "dh", p.N, p.ld_h), _rows(x, "x", K, p.ld_x), _rows(w, "w", K, p.ld_w),
                                    _ptr(z), _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(ws), nb, _stream(stream)),
           "moe_gated_backward")


def quantise_problem(M, K, dtype=MOE_DTYPE_BF16, block_rows=1, ld_x=0, ld_q=0) -> moe_quantise_problem:
    return moe_quantise_problem(M, K, dtype, block_rows, ld_x, ld_q)


def moe_quantise(p: moe_quantise_problem, x, q, scale, stream=None) -> None:
    """e4m3 codes q and fp32 scales of x, per (row, 128 columns) or per 128 x 128 block."""
    _check(lib().moe_quantise(p, _rows(x, "x", p.K, p.ld_x), _rows(q, "q", p.K, p.ld_q), _ptr(scale), _stream(stream)),
           "moe_quantise")


def moe_linear_fp8_workspace_size(p: moe_linear_problem) -> int:
    return int(lib().moe_linear_fp8_workspace_size(p))


def moe_linear_fp8(p: moe_linear_problem, x, x_scale, w, w_scale, bias, residual, y, ws, ws_bytes=None, stream=None) -> None:
    """y = alpha act(x w^T + bias) + residual for e4m3 operands with block scales."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    N, K, ld_y = p.N, p.K, p.ld_y
    _check(lib().moe_linear_fp8(p, _rows(x, "x", K, p.ld_x), _ptr(x_scale), _rows(w, "w", K, p.ld_w), _ptr(w_scale),
                                _ptr(bias), _rows(residual, "residual", N, ld_y), _rows(y, "y", N, ld_y), _ptr(ws), nb,
                                _stream(stream)), "moe_linear_fp8")


def moe_gated_fp8_workspace_size(p: moe_gated_problem) -> int:
    return int(lib().moe_gated_fp8_workspace_size(p))


def moe_gated_fp8(p: moe_gated_problem, x, x_scale, w, w_scale, bias, h, h_scale, ws, ws_bytes=None, stream=None) -> None:
    """moe_gated for e4m3 operands with block scales; h in codes with h_scale, or in out_dtype with None."""
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    K = p.K
    _check(lib().moe_gated_fp8(p, _rows(x, "x", K, p.ld_x), _ptr(x_scale), _rows(w, "w", K, p.ld_w), _ptr(w_scale),
                               _ptr(bias), _rows(h, "h", p.N, p.ld_h), _ptr(h_scale), _ptr(ws), nb, _stream(stream)),
           "moe_gated_fp8")


def moe_read_device_status(ws, stream=None) -> int:
    return int(lib().moe_read_device_status(_ptr(ws), _stream(stream)))


def moe_profile_start() -> None:
    lib().moe_profile_start()


def moe_profile_start_stage(stage: str) -> None:
    """Profile only the launches of one stage (e.g. "gateup_gemm")."""
    lib().moe_profile_start_stage(stage.encode() if stage else None)


def moe_profile_stop(max_stages: int = 32) -> dict:
    """Stops stage timing; returns {stage name: (total_ms, launches)} in launch order."""
    arr = (moe_stage_time * max_stages)()
    n = int(lib().moe_profile_stop(arr, max_stages))
    if n < 0:
        raise MoeError(MOE_ERR_CUDA, "moe_profile_stop")
    return {arr[i].name.decode(): (float(arr[i].total_ms), int(arr[i].launches)) for i in range(min(n, max_stages))}


def raw_status(fn_name: str, *args) -> int:
    """Call an entry point with raw arguments and return its status code
    (used by boundary tests that pass NULL or misaligned pointers)."""
    return int(getattr(lib(), fn_name)(*args))
