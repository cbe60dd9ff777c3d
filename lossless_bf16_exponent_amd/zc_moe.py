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
ZC_NORM_NONE, ZC_NORM_RMS, ZC_NORM_LAYER = range(3)
ZC_ACT_NONE, ZC_ACT_RELU, ZC_ACT_SILU, ZC_ACT_GELU, ZC_ACT_GELU_TANH, ZC_ACT_SIGMOID = range(6)
ZC_NORM_MAX_COLS = 16384
ZC_MAX_SEQUENCES = 1024
ZC_MATMUL_WORKSPACE_MAX = 64 << 20
ZC_BALANCE_WORKSPACE_MAX = 64 << 20
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


class zc_norm_params(ctypes.Structure):
    _fields_ = [("d_weight", ctypes.c_void_p), ("d_bias", ctypes.c_void_p), ("kind", ctypes.c_uint32),
                ("type", ctypes.c_uint32), ("eps", ctypes.c_float)]


class zc_norm_config(ctypes.Structure):
    _fields_ = [("after", zc_norm_params), ("before", zc_norm_params), ("d_gate", ctypes.c_void_p),
                ("d_row_gate", ctypes.c_void_p), ("gate_type", ctypes.c_uint32), ("scale", ctypes.c_float)]


class zc_norm_grads(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("d_weight_after", "d_bias_after", "d_gate", "d_weight_before",
                                                     "d_bias_before", "d_row_gate")]


class zc_epilogue(ctypes.Structure):
    _fields_ = [("d_bias", ctypes.c_void_p), ("d_residual", ctypes.c_void_p), ("d_pre", ctypes.c_void_p),
                ("residual_stride", ctypes.c_uint64), ("pre_stride", ctypes.c_uint64), ("bias_type", ctypes.c_uint32),
                ("residual_type", ctypes.c_uint32), ("activation", ctypes.c_uint32), ("scale", ctypes.c_float)]


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
_F32, _NORM = ctypes.c_float, ctypes.POINTER(zc_norm_config)

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
    "zc_norm": (ctypes.c_int, [_P, _U32, _U64, _U64, _U64, _P, _U64, _NORM, _P, _U64, _P, _U64, _P, _P, _P]),
    "zc_norm_backward_workspace_bytes": (_U64, [_U64, _U64]),
    "zc_norm_backward": (ctypes.c_int, [_P, _U32, _U64, _U64, _U64, _P, _U64, _NORM, _P, _U64, _P, _U64, _P, _U64, _P,
                                        _U64, ctypes.POINTER(zc_norm_grads), _P, _U64, _P]),
    "zc_matmul_workspace_bytes": (_U64, [_U64, _U64, _U64]),
    "zc_matmul": (ctypes.c_int, [_P, _U64, _U64, _P, _U64, _U64, _U64, ctypes.POINTER(zc_epilogue), _P, _U32, _U64, _P,
                                 _U64, _P]),
    "zc_activation_backward_workspace_bytes": (_U64, [_U64, _U64]),
    "zc_activation_backward": (ctypes.c_int, [_P, _U32, _U64, _U64, _U64, _P, _U64, _U32, _F32, _P, _U64, _P, _P, _U64,
                                              _P]),
    "zc_matmul_dgrad": (ctypes.c_int, [_P, _U64, _U64, _U64, _P, _U64, _U64, _P, _U32, _U64, _P, _U32, _U64, _P, _U64,
                                       _P]),
    "zc_matmul_wgrad": (ctypes.c_int, [_P, _U64, _U64, _U64, _P, _U64, _U64, _P, _U32, _U64, _P, _U32, _U64, _P, _U64,
                                       _P]),
    "zc_balance_workspace_bytes": (_U64, [_U64, _U32, _U32]),
    "zc_balance": (ctypes.c_int, [_P, _U32, _U64, _U64, _CFG, _P, _P, _U32, _P, _P, _U64, _P, _P, _P, _P, _P]),
    "zc_balance_backward": (ctypes.c_int, [_P, _U32, _U64, _U64, _CFG, _P, _U32, _P, _P, _P, _P, _P, _P, _U64, _P, _U64,
                                           _P]),
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


_types = {}  # of torch, once it is loaded


def _type_of(x, given) -> int:
    """The ZC_ type of a parameter: as given, or that of a float32 or bfloat16 tensor; ZC_F32 where there is none."""
    if given is not None:
        return given
    if x is None:
        return ZC_F32
    if isinstance(x, int):
        raise TypeError("the type of an address has to be given")
    if not _types:
        import torch
        _types.update({torch.float32: ZC_F32, torch.bfloat16: ZC_BF16})
    if x.dtype not in _types:
        raise TypeError("a parameter is float32 or bfloat16, not %s" % x.dtype)
    return _types[x.dtype]


# The structures hold addresses: `keep` holds what they belong to for as long.  They are made within a few
# microseconds too.

def norm_params(kind, weight=None, bias=None, eps=1e-6, type=None) -> zc_norm_params:
    """One norm; kind: a ZC_NORM_ value; type: of weight and bias, by default their tensors'."""
    t = _type_of(bias if weight is None else weight, type)
    if type is None and weight is not None and bias is not None and _type_of(bias, None) != t:
        raise TypeError("weight and bias have different types")
    p = zc_norm_params(_ptr(weight), _ptr(bias), kind, t, eps)
    p.keep = weight, bias
    return p


_no_norm = norm_params(ZC_NORM_NONE)


def norm_config(after=None, before=None, gate=None, row_gate=None, scale=1.0, gate_type=None) -> zc_norm_config:
    """after, before: norm_params, or None for no norm."""
    c = zc_norm_config(after or _no_norm, before or _no_norm, _ptr(gate), _ptr(row_gate), _type_of(gate, gate_type), scale)
    c.keep = after, before, gate, row_gate
    return c


def norm_grads(weight_after=None, bias_after=None, gate=None, weight_before=None, bias_before=None,
               row_gate=None) -> zc_norm_grads:
    g = zc_norm_grads(_ptr(weight_after), _ptr(bias_after), _ptr(gate), _ptr(weight_before), _ptr(bias_before), _ptr(row_gate))
    g.keep = weight_after, bias_after, gate, weight_before, bias_before, row_gate
    return g


def epilogue(bias=None, activation=ZC_ACT_NONE, residual=None, residual_stride=0, pre=None, pre_stride=0, scale=1.0,
             bias_type=None, residual_type=None) -> zc_epilogue:
    """bias_type, residual_type: by default those of their tensors."""
    e = zc_epilogue(_ptr(bias), _ptr(residual), _ptr(pre), residual_stride, pre_stride, _type_of(bias, bias_type),
                    _type_of(residual, residual_type), activation, scale)
    e.keep = bias, residual, pre
    return e


def zc_norm(d_x, stream_type, rows, cols, x_stride, d_z, z_stride, cfg, d_r, r_stride, d_y=None, y_stride=0, d_yq=None,
            d_yq_scales=None, stream=None) -> None:
    _check(_lib.zc_norm(_ptr(d_x), stream_type, rows, cols, x_stride, _ptr(d_z), z_stride, ctypes.byref(cfg), _ptr(d_r),
                        r_stride, _ptr(d_y), y_stride, _ptr(d_yq), _ptr(d_yq_scales), _stream(stream)), "zc_norm")


def zc_norm_backward_workspace_bytes(rows, cols) -> int:
    return int(_lib.zc_norm_backward_workspace_bytes(rows, cols))


def zc_norm_backward(d_r, stream_type, rows, cols, r_stride, d_z, z_stride, cfg, d_dr, dr_stride, d_dy, dy_stride, d_dx,
                     dx_stride, d_dz, dz_stride, grads=None, d_workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.zc_norm_backward(_ptr(d_r), stream_type, rows, cols, r_stride, _ptr(d_z), z_stride, ctypes.byref(cfg),
                                 _ptr(d_dr), dr_stride, _ptr(d_dy), dy_stride, _ptr(d_dx), dx_stride, _ptr(d_dz),
                                 dz_stride, None if grads is None else ctypes.byref(grads), _ptr(d_workspace),
                                 workspace_bytes, _stream(stream)), "zc_norm_backward")


def zc_matmul_workspace_bytes(rows, cols, contraction) -> int:
    return int(_lib.zc_matmul_workspace_bytes(rows, cols, contraction))


def zc_matmul(d_a, m, a_stride, d_w, n, k, w_stride, epilogue, d_out, out_type, out_stride, d_workspace=None,
              workspace_bytes=0, stream=None) -> None:
    _check(_lib.zc_matmul(_ptr(d_a), m, a_stride, _ptr(d_w), n, k, w_stride,
                          None if epilogue is None else ctypes.byref(epilogue), _ptr(d_out), out_type, out_stride,
                          _ptr(d_workspace), workspace_bytes, _stream(stream)), "zc_matmul")


def zc_activation_backward_workspace_bytes(rows, cols) -> int:
    return int(_lib.zc_activation_backward_workspace_bytes(rows, cols))


def zc_activation_backward(d_dout, dout_type, rows, cols, dout_stride, d_pre, pre_stride, activation, scale, d_dpre,
                           dpre_stride, d_dbias=None, d_workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.zc_activation_backward(_ptr(d_dout), dout_type, rows, cols, dout_stride, _ptr(d_pre), pre_stride,
                                       activation, scale, _ptr(d_dpre), dpre_stride, _ptr(d_dbias), _ptr(d_workspace),
                                       workspace_bytes, _stream(stream)), "zc_activation_backward")


def zc_matmul_dgrad(d_dpre, m, n, dpre_stride, d_w, k, w_stride, d_add, add_type, add_stride, d_dx, dx_type, dx_stride,
                    d_workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.zc_matmul_dgrad(_ptr(d_dpre), m, n, dpre_stride, _ptr(d_w), k, w_stride, _ptr(d_add), add_type,
                                add_stride, _ptr(d_dx), dx_type, dx_stride, _ptr(d_workspace), workspace_bytes,
                                _stream(stream)), "zc_matmul_dgrad")


def zc_matmul_wgrad(d_dpre, m, n, dpre_stride, d_a, k, a_stride, d_add, add_type, add_stride, d_dw, dw_type, dw_stride,
                    d_workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.zc_matmul_wgrad(_ptr(d_dpre), m, n, dpre_stride, _ptr(d_a), k, a_stride, _ptr(d_add), add_type,
                                add_stride, _ptr(d_dw), dw_type, dw_stride, _ptr(d_workspace), workspace_bytes,
                                _stream(stream)), "zc_matmul_wgrad")


def zc_balance_workspace_bytes(tokens, experts, sequences) -> int:
    return int(_lib.zc_balance_workspace_bytes(tokens, experts, sequences))


def zc_balance(d_logits, logits_type, tokens, logits_stride, cfg, d_ids, d_mask, sequences, d_offsets, d_workspace,
               workspace_bytes, d_counts, d_used, d_loss=None, d_zloss=None, stream=None) -> None:
    _check(_lib.zc_balance(_ptr(d_logits), logits_type, tokens, logits_stride, ctypes.byref(cfg), _ptr(d_ids),
                           _ptr(d_mask), sequences, _ptr(d_offsets), _ptr(d_workspace), workspace_bytes, _ptr(d_counts),
                           _ptr(d_used), _ptr(d_loss), _ptr(d_zloss), _stream(stream)), "zc_balance")


def zc_balance_backward(d_logits, logits_type, tokens, logits_stride, cfg, d_mask, sequences, d_offsets, d_counts, d_used,
                        d_dloss, d_dzloss, d_add, add_stride, d_dlogits, dlogits_stride, stream=None) -> None:
    _check(_lib.zc_balance_backward(_ptr(d_logits), logits_type, tokens, logits_stride, ctypes.byref(cfg), _ptr(d_mask),
                                    sequences, _ptr(d_offsets), _ptr(d_counts), _ptr(d_used), _ptr(d_dloss),
                                    _ptr(d_dzloss), _ptr(d_add), add_stride, _ptr(d_dlogits), dlogits_stride,
                                    _stream(stream)), "zc_balance_backward")
