"""Host-side checks of the norms, products and balance losses that need no GPU: sizes, and every argument they refuse,
before anything is enqueued."""
import ctypes
import os

import numpy as np
import pytest

from lossless_bf16_exponent_amd import _build

P = 1 << 20  # an address that passes the alignment checks and is never read
INVALID, CAPACITY, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(_build.LIB):
        _build.build()
    from lossless_bf16_exponent_amd import zc_moe
    return zc_moe


@pytest.fixture(scope="module")
def zc():
    from lossless_bf16_exponent_amd import zc as mod
    return mod


def call(zc, fn, args):
    return zc.raw_status(fn, *[ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args])


def side(moe, kind=1, weight=P, bias=P, eps=1e-6, type=1):
    return moe.norm_params(kind, weight, bias, eps, type)


def config(moe, after=None, before=None, **kw):
    base = dict(gate=P, row_gate=P, scale=1.0, gate_type=1)
    base.update(kw)
    return moe.norm_config(after or side(moe), before or side(moe), **base)


def test_sizes(moe):
    for rows, cols in ((1, 1), (8192, 7168), (5, 16384), (1 << 30, 64)):
        n = moe.zc_norm_backward_workspace_bytes(rows, cols)
        assert n % 256 == 0 and 0 < n <= 1 << 28, (rows, cols)
    assert moe.zc_norm_backward_workspace_bytes(0, 64) == 0
    assert moe.zc_norm_backward_workspace_bytes(1, moe.ZC_NORM_MAX_COLS + 1) == 0
    g = np.random.default_rng(0)
    for _ in range(500):
        r, c, k = (int(2 ** g.uniform(0, 15)) for _ in range(3))
        n = moe.zc_matmul_workspace_bytes(r, c, k)
        assert n <= moe.ZC_MATMUL_WORKSPACE_MAX and n % 16 == 0
    assert moe.zc_matmul_workspace_bytes(0, 5, 5) == 0 and moe.zc_matmul_workspace_bytes(1 << 31, 5, 5) == 0
    assert moe.zc_matmul_workspace_bytes(256, 256, 8192) > 0
    assert moe.zc_activation_backward_workspace_bytes(8192, 4096) % 256 == 0
    assert moe.zc_activation_backward_workspace_bytes(8192, 4096) >= 4 * 4096
    for t, e, s in ((0, 8, 1), (1, 1, 1), (8192, 256, 1), (1 << 20, 1024, 1024), (100, 1024, 1024)):
        n = moe.zc_balance_workspace_bytes(t, e, s)
        assert n % 256 == 0 and 0 < n <= moe.ZC_BALANCE_WORKSPACE_MAX
    assert moe.zc_balance_workspace_bytes(8, 0, 1) == 0 and moe.zc_balance_workspace_bytes(8, 1025, 1) == 0
    assert moe.zc_balance_workspace_bytes(8, 8, 0) == 0 and moe.zc_balance_workspace_bytes(8, 8, 1025) == 0


def refusals(moe):
    cfg, grads, rc = config(moe), moe.norm_grads(P, P, P, P, P, P), moe.route_config(64, 4)
    ep = moe.epilogue(P, 2, P, 64, P, 64, bias_type=0, residual_type=1)
    big = 1 << 41
    yield "zc_norm", [P, 1, 4, 64, 64, P, 64, cfg, P, 64, P, 64, P, P, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 2, INVALID), (2, 1 << 31, INVALID), (3, 16385, INVALID),
        (4, 63, INVALID), (4, big, INVALID), (5, P + 1, MISALIGNED), (6, 63, INVALID), (7, None, INVALID),
        (8, P + 1, MISALIGNED), (9, 63, INVALID), (10, P + 1, MISALIGNED), (11, 63, INVALID), (12, None, INVALID),
        (12, P + 8, MISALIGNED), (13, None, INVALID), (13, P + 2, MISALIGNED)]
    yield "zc_norm", [P, 0, 4, 64, 64, P, 64, cfg, P, 64, P, 64, P, P, None], [
        (0, P + 2, MISALIGNED), (8, P + 2, MISALIGNED)]
    yield "zc_norm_backward", [P, 1, 4, 64, 64, P, 64, cfg, P, 64, P, 64, P, 64, P, 64, grads, P, 1 << 28, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 2, INVALID), (2, 1 << 31, INVALID), (3, 16385, INVALID),
        (4, 63, INVALID), (5, None, INVALID), (6, 63, INVALID), (7, None, INVALID), (8, P + 1, MISALIGNED), (9, 63, INVALID),
        (10, P + 1, MISALIGNED), (11, 63, INVALID), (12, P + 1, MISALIGNED), (13, 63, INVALID), (14, P + 1, MISALIGNED),
        (15, 63, INVALID), (17, None, INVALID), (17, P + 8, MISALIGNED), (18, 8, CAPACITY)]
    for name in ("weight_after", "bias_after", "gate", "weight_before", "bias_before", "row_gate"):
        yield "zc_norm_backward", [P, 1, 4, 64, 64, P, 64, cfg, P, 64, P, 64, P, 64, P, 64, grads, P, 1 << 28, None], [
            (16, moe.norm_grads(**{name: P + 2}), MISALIGNED)]
    yield "zc_matmul", [P, 8, 128, P, 64, 128, 128, ep, P, 1, 64, P, 0, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 1 << 31, INVALID), (2, 127, INVALID), (2, big, INVALID),
        (3, None, INVALID), (3, P + 1, MISALIGNED), (4, 1 << 29, INVALID), (5, 1 << 29, INVALID), (6, 127, INVALID),
        (8, None, INVALID), (8, P + 1, MISALIGNED), (9, 2, INVALID), (10, 63, INVALID), (11, P + 8, MISALIGNED)]
    yield "zc_activation_backward", [P, 1, 8, 64, 64, P, 64, 2, 1.0, P, 64, P, P, 1 << 28, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 2, INVALID), (2, 1 << 31, INVALID), (3, 1 << 29, INVALID),
        (4, 63, INVALID), (5, None, INVALID), (5, P + 1, MISALIGNED), (6, 63, INVALID), (7, 6, INVALID),
        (8, float("nan"), INVALID), (9, P + 1, MISALIGNED), (10, 63, INVALID), (11, P + 2, MISALIGNED), (12, None, INVALID),
        (12, P + 8, MISALIGNED), (13, 8, CAPACITY)]
    for fn in ("zc_matmul_dgrad", "zc_matmul_wgrad"):
        # both operands 128 wide at least
        yield fn, [P, 128, 128, 128, P, 128, 128, P, 0, 128, P, 1, 128, P, 0, None], [
            (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 1 << 31, INVALID), (2, 1 << 29, INVALID), (3, 127, INVALID),
            (4, None, INVALID), (4, P + 1, MISALIGNED), (5, 1 << 29, INVALID), (6, 127, INVALID), (7, P + 2, MISALIGNED),
            (8, 2, INVALID), (9, 127, INVALID), (10, None, INVALID), (10, P + 1, MISALIGNED), (11, 2, INVALID),
            (12, 127, INVALID), (13, P + 8, MISALIGNED)]
    yield "zc_balance", [P, 0, 40, 64, rc, P, P, 2, P, P, 1 << 26, P, P, P, P, None], [
        (0, None, INVALID), (0, P + 2, MISALIGNED), (1, 2, INVALID), (2, 1 << 31, INVALID), (3, 63, INVALID), (4, None, INVALID),
        (5, None, INVALID), (5, P + 2, MISALIGNED), (7, 0, INVALID), (7, 1025, INVALID), (8, None, INVALID),
        (8, P + 2, MISALIGNED), (9, None, INVALID), (9, P + 8, MISALIGNED), (10, 64, CAPACITY), (11, None, INVALID),
        (11, P + 2, MISALIGNED), (12, None, INVALID), (12, P + 1, MISALIGNED), (13, P + 2, MISALIGNED), (14, P + 2, MISALIGNED)]
    yield "zc_balance_backward", [P, 0, 40, 64, rc, P, 2, P, P, P, P, P, P, 64, P, 64, None], [
        (0, None, INVALID), (0, P + 2, MISALIGNED), (1, 2, INVALID), (2, 1 << 31, INVALID), (3, 63, INVALID), (4, None, INVALID),
        (6, 0, INVALID), (6, 1025, INVALID), (7, None, INVALID), (7, P + 2, MISALIGNED), (8, None, INVALID), (9, None, INVALID),
        (9, P + 2, MISALIGNED), (10, P + 2, MISALIGNED), (11, P + 2, MISALIGNED), (12, P + 2, MISALIGNED), (13, 63, INVALID),
        (14, None, INVALID), (14, P + 2, MISALIGNED), (15, 63, INVALID)]


def test_refusals(zc, moe):
    for fn, good, bad in refusals(moe):
        for index, value, status in bad:
            args = list(good)
            args[index] = value
            assert call(zc, fn, args) == status, (fn, index, value)


@pytest.mark.parametrize("kw", [dict(kind=3), dict(type=2), dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(eps=1e-39)])
def test_refused_norms(zc, moe, kw):
    for cfg in (config(moe, after=side(moe, **kw)), config(moe, before=side(moe, **kw))):
        assert call(zc, "zc_norm", [P, 1, 4, 64, 64, P, 64, cfg, P, 64, P, 64, P, P, None]) == INVALID
        assert call(zc, "zc_norm_backward", [P, 1, 4, 64, 64, P, 64, cfg, P, 64, P, 64, P, 64, P, 64, None, P, 0, None]) == INVALID
    # what is not read is not looked at: the first half without a block's output, and all but the kind of no norm
    cfg = config(moe, after=side(moe, **kw))
    assert call(zc, "zc_norm", [None, 1, 0, 64, 64, None, 0, cfg, P, 64, P, 64, P, P, None]) == 0
    if "kind" not in kw:
        cfg = config(moe, after=side(moe, **{**kw, "kind": 0}), before=side(moe, **{**kw, "kind": 0}))
        assert call(zc, "zc_norm", [None, 1, 0, 64, 64, P, 64, cfg, P, 64, P, 64, P, P, None]) == 0


@pytest.mark.parametrize("kw", [dict(scale=float("nan")), dict(scale=float("inf")), dict(gate_type=2)])
def test_refused_gates(zc, moe, kw):
    assert call(zc, "zc_norm", [P, 1, 4, 64, 64, P, 64, config(moe, **kw), P, 64, P, 64, P, P, None]) == INVALID
    for kw, status in ((dict(gate=P + 1), MISALIGNED), (dict(row_gate=P + 2), MISALIGNED), (dict(gate=P + 2, gate_type=0), MISALIGNED),
                       (dict(after=side(moe, weight=P + 1)), MISALIGNED), (dict(before=side(moe, bias=P + 2, type=0)), MISALIGNED)):
        assert call(zc, "zc_norm", [P, 1, 4, 64, 64, P, 64, config(moe, **kw), P, 64, P, 64, P, P, None]) == status


@pytest.mark.parametrize("kw,status", [(dict(activation=6), INVALID), (dict(scale=float("nan")), INVALID),
                                       (dict(bias=P, bias_type=2), INVALID), (dict(bias=P + 2, bias_type=0), MISALIGNED),
                                       (dict(residual=P, residual_type=2, residual_stride=64), INVALID),
                                       (dict(residual=P, residual_type=1, residual_stride=63), INVALID),
                                       (dict(residual=P + 1, residual_type=1, residual_stride=64), MISALIGNED),
                                       (dict(pre=P, pre_stride=63), INVALID), (dict(pre=P + 1, pre_stride=64), MISALIGNED)])
def test_refused_epilogues(zc, moe, kw, status):
    assert call(zc, "zc_matmul", [P, 8, 128, P, 64, 128, 128, moe.epilogue(**kw), P, 1, 64, None, 0, None]) == status


@pytest.mark.parametrize("kw", [dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=33), dict(score=2)])
def test_refused_balance(zc, moe, kw):
    rc = moe.route_config(**{**dict(experts=64, top_k=4), **kw})
    assert call(zc, "zc_balance", [P, 0, 40, 2048, rc, P, P, 2, P, P, 1 << 26, P, P, P, P, None]) == INVALID
    assert call(zc, "zc_balance_backward", [P, 0, 40, 2048, rc, P, 2, P, P, P, P, P, P, 2048, P, 2048, None]) == INVALID


def test_nothing_to_do_is_ok(zc, moe):
    """Counts of zero return ZC_OK without a launch (there is no GPU to launch on here)."""
    cfg, rc = config(moe), moe.route_config(64, 4)
    for fn, args in (("zc_norm", [None, 1, 0, 64, 64, None, 64, cfg, None, 64, None, 64, None, None, None]),
                     ("zc_norm", [P, 1, 4, 0, 64, P, 64, cfg, P, 64, P, 64, P, P, None]),
                     ("zc_norm", [P, 1, 4, 64, 64, P, 64, cfg, None, 0, None, 0, None, None, None]),
                     ("zc_norm_backward", [None, 1, 0, 64, 64, None, 64, cfg] + [None, 64] * 4 + [None, None, 0, None]),
                     ("zc_norm_backward", [P, 1, 4, 64, 64, None, 64, cfg] + [None, 64] * 4 + [None, None, 0, None]),
                     ("zc_matmul", [None, 0, 64, None, 64, 64, 64, None, None, 1, 64, None, 0, None]),
                     ("zc_matmul", [P, 8, 64, P, 0, 64, 64, None, P, 1, 64, None, 0, None]),
                     ("zc_activation_backward", [None, 1, 0, 64, 64, None, 64, 2, 1.0, P, 64, None, None, 0, None]),
                     ("zc_activation_backward", [P, 1, 8, 64, 64, P, 64, 2, 1.0, None, 0, None, None, 0, None]),
                     ("zc_matmul_dgrad", [None, 0, 64, 64, P, 64, 64, None, 0, 0, None, 1, 64, None, 0, None]),
                     ("zc_matmul_wgrad", [P, 8, 0, 64, P, 64, 64, None, 0, 0, None, 1, 64, None, 0, None]),
                     ("zc_balance_backward", [None, 0, 0, 64, rc, None, 1, None, None, None, None, None, None, 0, None, 64, None])):
        assert call(zc, fn, args) == 0, fn


def test_types_come_from_tensors(moe):
    torch = pytest.importorskip("torch")
    f, b = torch.zeros(4), torch.zeros(4, dtype=torch.bfloat16)
    assert moe.norm_params(1, f).type == moe.ZC_F32 and moe.norm_params(1, b).type == moe.ZC_BF16
    assert moe.norm_params(1, None, b).type == moe.ZC_BF16
    with pytest.raises(TypeError):
        moe.norm_params(1, f, b)
    with pytest.raises(TypeError):
        moe.norm_params(1, 4096)
    with pytest.raises((TypeError, KeyError)):
        moe.epilogue(bias=torch.zeros(4, dtype=torch.float16))
    e = moe.epilogue(bias=b, residual=f, residual_stride=4)
    assert (e.bias_type, e.residual_type, e.d_bias, e.d_residual) == (moe.ZC_BF16, moe.ZC_F32, b.data_ptr(), f.data_ptr())
    c = moe.norm_config(moe.norm_params(2, f), None, gate=b)
    assert (c.after.kind, c.before.kind, c.gate_type, c.d_gate) == (2, 0, moe.ZC_BF16, b.data_ptr())


def test_types_of_parameters(moe):
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        moe.norm_params(moe.ZC_NORM_RMS, torch.ones(8, dtype=torch.float16))
    with pytest.raises(TypeError):
        moe.epilogue(bias=torch.ones(8, dtype=torch.float64))
    assert moe.norm_params(moe.ZC_NORM_RMS, torch.ones(8, dtype=torch.bfloat16)).type == moe.ZC_BF16
