"""An error that another call left pending in the HIP runtime is not a call's own."""
import ctypes

import numpy as np
import pytest
import torch

from moe_gpu import Out, device, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


def leave_an_error(zc):
    """The runtime refuses a device that does not exist and keeps the error until somebody asks for it."""
    assert zc._lib.hipSetDevice(ctypes.c_int(1 << 20)) != 0


def calls(zc):
    bf, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    e4, t, e, k, h = zc.ZC_FP8_E4M3, 40, 16, 2, 256
    cfg = zc.route_config(e, k, "sigmoid")
    x = torch.ones(t * k, h, dtype=bf, device="cuda")
    logits = torch.zeros(t, e, device="cuda")
    ids, w = torch.zeros(t, k, dtype=i32, device="cuda"), torch.zeros(t, k, dtype=f32, device="cuda")
    off, pos = Out((e + 1,), i32), torch.arange(t * k, dtype=i32, device="cuda")
    ws = Out((zc.zc_dispatch_workspace_bytes(t, k, e),), u8)
    q, s = torch.zeros(t * k, h, dtype=u8, device="cuda"), torch.zeros(t * k, 4, dtype=u8, device="cuda")
    qt, st = torch.zeros(h, 128, dtype=u8, device="cuda"), torch.zeros(h, 4, dtype=u8, device="cuda")
    kept, ks = torch.zeros(t * k, h, dtype=u8, device="cuda"), torch.zeros(t * k, 4, dtype=u8, device="cuda")
    rows = device(np.array([0, t * k], dtype=np.int32))
    out, wide = Out((t * k, h), bf), Out((h, h), f32)
    yield "zc_route", (logits, zc.ZC_F32, t, e, None, cfg, ids, w)
    yield "zc_route_backward", (logits, zc.ZC_F32, t, e, cfg, ids, w, Out((t, e), f32), e)
    yield "zc_dispatch_plan", (ids, t, k, e, ws, ws.n, off, Out((t, k), i32), None)
    yield "zc_dispatch_plan", (None, 0, k, e, None, 0, off, None, None)
    yield "zc_dispatch", (x, t, h, h, pos, k, out, t * k, h)
    yield "zc_combine", (x, t * k, h, h, pos, w, t, k, out, h)
    yield "zc_combine_backward", (x, h, x, t * k, h, h, pos, w, t, k, out, h, Out((t, k), f32))
    yield "zc_fp8_quantize", (x, t * k, h, h, e4, 1, q, s)
    yield "zc_fp8_quantize_t", (x, None, zc.ZC_BF16, t * k, h, h, 1, rows, e4, qt, st, 128)
    yield "zc_fp8_transpose", (q, s, 1, t * k, h, qt, st)
    yield "zc_fp8_matmul", (q, s, e4, t * k, q, s, e4, t * k, h, 1, None, out, zc.ZC_BF16, h)
    yield "zc_fp8_matmul_wgrad", (qt, st, e4, h, qt, st, e4, h, 128, t * k, 1, None, wide, zc.ZC_F32)
    yield "zc_swiglu", (x, t * k, h // 2, h, None, 0, None, None, kept, ks)
    yield "zc_swiglu_backward", (kept, ks, t * k, h // 2, x, h, out, h)


def test_a_pending_error_is_not_reported(zc):
    for name, args in calls(zc):
        torch.cuda.synchronize()
        leave_an_error(zc)
        getattr(zc, name)(*args)  # raises zc.ZcError for anything but ZC_OK
    torch.cuda.synchronize()
