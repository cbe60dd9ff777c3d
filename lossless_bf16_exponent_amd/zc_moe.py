"""Python binding of the C ABI in include/zc_moe.h (argument marshalling only).

Every function has the name of the C entry point it calls and its arguments in
the same order; pointer and stream arguments are those of ``zc`` (an integer
device address or anything with ``data_ptr()``; None is NULL).  A nonzero status
raises ``zc.ZcError``.  A product is summed in full (ZC_FP8_SUM_FULL) unless the
caller asks for the faster sums.  All work runs in the HIP kernels of libzc.so:
there is no fallback path.
"""
from __future__ import annotations

import ctypes

from .zc import ZC_OK, _lib, ZcError  # noqa: F401  (raises when libzc.so is not built)

ZC_F32, ZC_BF16, ZC_FP8_E4M3, ZC_FP8_E5M2 = range(4)
ZC_SCORE_SOFTMAX, ZC_SCORE_SIGMOID = range(2)
ZC_FP8_SUM_FAST, ZC_FP8_SUM_FULL = range(2)
ZC_MAX_EXPERTS = 1024
ZC_MAX_TOP_K = 32
ZC_MAX_EXPERT_GROUPS = 64
ZC_FP8_BLOCK = 128
ZC_MOE_ROW_SLACK = 262144
ZC_FP8_MATMUL_WORKSPACE_MAX = 64 << 20


class zc_route_config(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_uint32), ("top_k", ctypes.c_uint32), ("score", ctypes.c_uint32),
                ("groups", ctypes.c_uint32), ("group_top", ctypes.c_uint32), ("group_score", ctypes.c_uint32),
                ("renormalise", ctypes.c_uint32), ("scale", ctypes.c_float)]


# The calls of a serving step take a few microseconds: no object is made for the
# current stream, and nothing is imported, once torch is loaded.
_raw_stream = _device = None


def _stream(s) -> int:
    global _raw_stream, _device
    if s is None:
        if _raw_stream is None:
            import torch
            torch.cuda.current_stream()  # initialises the device
            _raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        return _raw_stream(_device())
    return s if isinstance(s, int) else int(s.cuda_stream)


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def _check(rc: int, where: str) -> None:
    if rc != ZC_OK:
        raise ZcError(rc, where)


_P, _U32, _U64, _CFG = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.POINTER(zc_route_config)

_SIGNATURES = {
    "zc_route": (ctypes.c_int, [_P, _U32, _U64, _U64, _P, _CFG, _P, _P, _P]),
    "zc_route_backward": (ctypes.c_int, [_P, _U32, _U64, _U64, _CFG, _P, _P, _P, _U64, _P]),
    "zc_dispatch_workspace_bytes": (_U64, [_U64, _U32, _U32]),
    "zc_dispatch_plan": (ctypes.c_int, [_P, _U64, _U32, _U32, _P, _U64, _P, _P, _P, _P]),
    "zc_dispatch": (ctypes.c_int, [_P, _U64, _U64, _U64, _P, _U32, _P, _U64, _U64, _P]),
    "zc_combine": (ctypes.c_int, [_P, _U64, _U64, _U64, _P, _P, _U64, _U32, _P, _U64, _P]),
    "zc_combine_backward": (ctypes.c_int, [_P, _U64, _P, _U64, _U64, _U64, _P, _P, _U64, _U32, _P, _U64, _P, _P]),
    "zc_fp8_stride": (_U64, [_U64]),
    "zc_fp8_scale_stride": (_U64, [_U64]),
    "zc_fp8_padded_rows": (_U64, [_U64, _U32]),
    "zc_fp8_quantize": (ctypes.c_int, [_P, _U64, _U64, _U64, _U32, _U32, _P, _P, _P]),
    "zc_fp8_quantize_t": (ctypes.c_int, [_P, _P, _U32, _U64, _U64, _U64, _U32, _P, _U32, _P, _P, _U64, _P]),
    "zc_fp8_transpose": (ctypes.c_int, [_P, _P, _U64, _U64, _U64, _P, _P, _P]),
    "zc_fp8_matmul_workspace_bytes": (_U64, [_U64, _U64, _U64, _U32]),
    "zc_fp8_matmul": (ctypes.c_int, [_P, _P, _U32, _U64, _P, _P, _U32, _U64, _U64, _U32, _P, _P, _U32, _U64, _U32, _P,
                                     _U64, _P]),
    "zc_fp8_matmul_wgrad": (ctypes.c_int, [_P, _P, _U32, _U64, _P, _P, _U32, _U64, _U64, _U64, _U32, _P, _P, _U32,
                                           _U32, _P]),
    "zc_swiglu": (ctypes.c_int, [_P, _U64, _U64, _U64, _P, _U64, _P, _P, _P, _P, _P]),
    "zc_swiglu_backward": (ctypes.c_int, [_P, _P, _U64, _U64, _P, _U64, _P, _U64, _P]),
}
EXPORTED = tuple(_SIGNATURES)

for _name, (_res, _args) in _SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args


def route_config(experts, top_k, score="softmax", groups=1, group_top=1, group_score=1, renormalise=True,
                 scale=1.0) -> zc_route_config:
    """How a token's experts are chosen; score: "softmax", "sigmoid" or a ZC_SCORE_ value."""
    score = {"softmax": ZC_SCORE_SOFTMAX, "sigmoid": ZC_SCORE_SIGMOID}.get(score, score)
    return zc_route_config(int(experts), int(top_k), int(score), int(groups), int(group_top), int(group_score),
                           int(renormalise), float(scale))


def zc_route(d_logits, logits_type, tokens, logits_stride, d_bias, cfg, d_ids, d_weights, stream=None) -> None:
    _check(_lib.zc_route(_ptr(d_logits), logits_type, tokens, logits_stride, _ptr(d_bias), ctypes.byref(cfg),
                         _ptr(d_ids), _ptr(d_weights), _stream(stream)), "zc_route")


def zc_route_backward(d_logits, logits_type, tokens, logits_stride, cfg, d_ids, d_dweights, d_dlogits, dlogits_stride,
                      stream=None) -> None:
    _check(_lib.zc_route_backward(_ptr(d_logits), logits_type, tokens, logits_stride, ctypes.byref(cfg), _ptr(d_ids),
                                  _ptr(d_dweights), _ptr(d_dlogits), dlogits_stride, _stream(stream)),
           "zc_route_backward")


def zc_dispatch_workspace_bytes(tokens, top_k, experts) -> int:
    return int(_lib.zc_dispatch_workspace_bytes(tokens, top_k, experts))


def zc_dispatch_plan(d_ids, tokens, top_k, experts, d_workspace, workspace_bytes, d_offsets, d_position,
                     d_source=None, stream=None) -> None:
    _check(_lib.zc_dispatch_plan(_ptr(d_ids), tokens, top_k, experts, _ptr(d_workspace), workspace_bytes,
                                 _ptr(d_offsets), _ptr(d_position), _ptr(d_source), _stream(stream)),
           "zc_dispatch_plan")


def zc_dispatch(d_x, tokens, hidden, x_stride, d_position, top_k, d_out, rows, out_stride, stream=None) -> None:
    _check(_lib.zc_dispatch(_ptr(d_x), tokens, hidden, x_stride, _ptr(d_position), top_k, _ptr(d_out), rows,
                            out_stride, _stream(stream)), "zc_dispatch")


def zc_combine(d_z, rows, hidden, z_stride, d_position, d_weights, tokens, top_k, d_y, y_stride, stream=None) -> None:
    _check(_lib.zc_combine(_ptr(d_z), rows, hidden, z_stride, _ptr(d_position), _ptr(d_weights), tokens, top_k,
                           _ptr(d_y), y_stride, _stream(stream)), "zc_combine")


def zc_combine_backward(d_dy, dy_stride, d_z, rows, hidden, z_stride, d_position, d_weights, tokens, top_k, d_dz,
                        dz_stride, d_dweights, stream=None) -> None:
    _check(_lib.zc_combine_backward(_ptr(d_dy), dy_stride, _ptr(d_z), rows, hidden, z_stride, _ptr(d_position),
                                    _ptr(d_weights), tokens, top_k, _ptr(d_dz), dz_stride, _ptr(d_dweights),
                                    _stream(stream)), "zc_combine_backward")


def zc_fp8_stride(cols) -> int:
    return int(_lib.zc_fp8_stride(cols))


def zc_fp8_scale_stride(cols) -> int:
    return int(_lib.zc_fp8_scale_stride(cols))


def zc_fp8_padded_rows(rows, groups) -> int:
    return int(_lib.zc_fp8_padded_rows(rows, groups))


def zc_fp8_quantize(d_x, rows, cols, x_stride, type, block_rows, d_q, d_scales, stream=None) -> None:
    _check(_lib.zc_fp8_quantize(_ptr(d_x), rows, cols, x_stride, type, block_rows, _ptr(d_q), _ptr(d_scales),
                                _stream(stream)), "zc_fp8_quantize")


def zc_fp8_quantize_t(d_x, d_x_scales, x_type, rows, cols, x_stride, groups, d_offsets, type, d_q, d_scales,
                      padded_rows, stream=None) -> None:
    _check(_lib.zc_fp8_quantize_t(_ptr(d_x), _ptr(d_x_scales), x_type, rows, cols, x_stride, groups, _ptr(d_offsets),
                                  type, _ptr(d_q), _ptr(d_scales), padded_rows, _stream(stream)), "zc_fp8_quantize_t")


def zc_fp8_transpose(d_q, d_scales, batch, rows, cols, d_qt, d_scales_t, stream=None) -> None:
    _check(_lib.zc_fp8_transpose(_ptr(d_q), _ptr(d_scales), batch, rows, cols, _ptr(d_qt), _ptr(d_scales_t),
                                 _stream(stream)), "zc_fp8_transpose")


def zc_fp8_matmul_workspace_bytes(m, n, k, groups) -> int:
    return int(_lib.zc_fp8_matmul_workspace_bytes(m, n, k, groups))


def zc_fp8_matmul(d_a, d_a_scales, a_type, m, d_b, d_b_scales, b_type, n, k, groups, d_offsets, d_out, out_type,
                  out_stride, sum_mode=ZC_FP8_SUM_FULL, d_workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.zc_fp8_matmul(_ptr(d_a), _ptr(d_a_scales), a_type, m, _ptr(d_b), _ptr(d_b_scales), b_type, n, k, groups,
                              _ptr(d_offsets), _ptr(d_out), out_type, out_stride, sum_mode, _ptr(d_workspace),
                              workspace_bytes, _stream(stream)), "zc_fp8_matmul")


def zc_fp8_matmul_wgrad(d_a, d_a_scales, a_type, n, d_b, d_b_scales, b_type, k, padded_rows, rows, groups, d_offsets,
                        d_out, out_type, sum_mode=ZC_FP8_SUM_FULL, stream=None) -> None:
    _check(_lib.zc_fp8_matmul_wgrad(_ptr(d_a), _ptr(d_a_scales), a_type, n, _ptr(d_b), _ptr(d_b_scales), b_type, k,
                                    padded_rows, rows, groups, _ptr(d_offsets), _ptr(d_out), out_type,
                                    sum_mode, _stream(stream)), "zc_fp8_matmul_wgrad")


def zc_swiglu(d_gate_up, rows, cols, gu_stride, d_h, h_stride, d_hq, d_hq_scales, d_kept, d_kept_scales,
              stream=None) -> None:
    _check(_lib.zc_swiglu(_ptr(d_gate_up), rows, cols, gu_stride, _ptr(d_h), h_stride, _ptr(d_hq), _ptr(d_hq_scales),
                          _ptr(d_kept), _ptr(d_kept_scales), _stream(stream)), "zc_swiglu")


def zc_swiglu_backward(d_kept, d_kept_scales, rows, cols, d_dh, dh_stride, d_dgate_up, gu_stride,
                       stream=None) -> None:
    _check(_lib.zc_swiglu_backward(_ptr(d_kept), _ptr(d_kept_scales), rows, cols, _ptr(d_dh), dh_stride,
                                   _ptr(d_dgate_up), gu_stride, _stream(stream)), "zc_swiglu_backward")
