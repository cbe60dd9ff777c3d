"""The gated activation, its 8-bit checkpoint and its gradient from the checkpoint
against 64 bits."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from moe_gpu import Out, bf16_device, close, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


SHAPES = [(1, 1, 0), (1, 128, 0), (3, 130, 0), (8, 2048, 0), (17, 1000, 8), (40, 333, 1), (5, 64, 64), (130, 264, 0)]


def inputs(m, f, scale=2.0):
    g = np.random.default_rng([m, f])
    return ref.bf16(g.standard_normal((m, 2 * f)) * scale), ref.bf16(g.standard_normal((m, f)))


# The exponential's argument is rounded (|g| log2 e steps of 2^-24), the exponential, the reciprocal and the products
# add a few half steps; results below 2^-126 may be flushed in the exponential.
def tolerance(value, size, g):
    return ref.BF16_HALF_STEP * np.abs(value) + (10 + 4 * np.abs(g)) * 2 * ref.F32_HALF_STEP * size + 2.0 ** -120


def forward(zc, gu, f, gap, h=True, hq=True, kept=True):
    m = gu.shape[0]
    fs = zc.zc_fp8_stride(f)
    o = dict(h=Out((m, f + gap), torch.bfloat16), hq=Out((m, fs), torch.uint8),
             hs=Out((m, zc.zc_fp8_scale_stride(f)), torch.uint8), kq=Out((m, 2 * fs), torch.uint8),
             ks=Out((m, zc.zc_fp8_scale_stride(2 * fs)), torch.uint8))
    zc.zc_swiglu(bf16_device(gu, 2 * f + gap), m, f, 2 * f + gap, o["h"] if h else None, f + gap,
                 o["hq"] if hq else None, o["hs"] if hq else None, o["kq"] if kept else None, o["ks"] if kept else None)
    return o


@pytest.mark.parametrize("m,f,gap", SHAPES)
def test_forward(zc, m, f, gap):
    gu, _ = inputs(m, f)
    o = forward(zc, gu, f, gap)
    h = o["h"].numpy()[:, :f]
    want = ref.swiglu(gu[:, :f], gu[:, f:])
    close(h, want, tolerance(want, np.abs(want), gu[:, :f]), "h")
    # the 8-bit h is the blocks of the BF16 h, and the checkpoint those of the input: exactly
    want_q, want_s = ref.quantize(h, ref.E4M3)
    assert np.array_equal(o["hq"].numpy(), want_q) and np.array_equal(o["hs"].numpy(), want_s)
    fs = zc.zc_fp8_stride(f)
    nb = fs // 128
    kq, ks = o["kq"].numpy(), o["ks"].numpy()
    for half in range(2):
        want_q, want_s = ref.quantize(gu[:, half * f:(half + 1) * f], ref.E4M3)
        assert np.array_equal(kq[:, half * fs:(half + 1) * fs], want_q)
        assert np.array_equal(ks[:, half * nb:(half + 1) * nb], want_s[:, :nb])
    assert not ks[:, 2 * nb:].any()


@pytest.mark.parametrize("which", [("h",), ("hq",), ("kept",), ("h", "kept"), ()])
def test_results_left_out(zc, which):
    m, f = 20, 200
    gu, _ = inputs(m, f)
    full = {k: v.numpy().copy() for k, v in forward(zc, gu, f, 0).items()}
    part = forward(zc, gu, f, 0, **{k: k in which for k in ("h", "hq", "kept")})
    for key, owner in (("h", "h"), ("hq", "hq"), ("hs", "hq"), ("kq", "kept"), ("ks", "kept")):
        got = part[key].numpy()
        if owner in which:
            assert np.array_equal(got, full[key]), key
        else:
            assert bool((part[key].raw == 0xA5).all()), key


@pytest.mark.parametrize("m,f,gap", SHAPES)
def test_backward(zc, m, f, gap):
    gu, dh = inputs(m, f)
    o = forward(zc, gu, f, gap, h=False, hq=False)
    out = Out((m, 2 * f + gap), torch.bfloat16)
    zc.zc_swiglu_backward(o["kq"], o["ks"], m, f, bf16_device(dh, f + gap), f + gap, out, 2 * f + gap)
    got = out.numpy()
    fs = zc.zc_fp8_stride(f)
    nb = fs // 128
    kq, ks = o["kq"].numpy(), o["ks"].numpy()
    g = ref.values(kq[:, :fs], ks[:, :nb], ref.E4M3, f)
    u = ref.values(kq[:, fs:], ks[:, nb:2 * nb], ref.E4M3, f)
    dg, du, size = ref.swiglu_backward(g, u, dh)
    close(got[:, :f], dg, tolerance(dg, size, g), "dgate")
    close(got[:, f:2 * f], du, tolerance(du, np.abs(du), g), "dup")


def test_backward_against_differences(zc):
    """Central differences of the 64-bit activation at the kept values."""
    m, f = 4, 128
    gu, dh = inputs(m, f, 1.0)
    o = forward(zc, gu, f, 0, h=False, hq=False)
    out = Out((m, 2 * f), torch.bfloat16)
    zc.zc_swiglu_backward(o["kq"], o["ks"], m, f, bf16_device(dh), f, out, 2 * f)
    got = out.numpy()
    kq, ks = o["kq"].numpy(), o["ks"].numpy()
    g, u = ref.values(kq[:, :128], ks[:, :1], ref.E4M3, f), ref.values(kq[:, 128:], ks[:, 1:2], ref.E4M3, f)
    e = 1e-5
    dg = dh * (ref.swiglu(g + e, u) - ref.swiglu(g - e, u)) / (2 * e)
    du = dh * (ref.swiglu(g, u + e) - ref.swiglu(g, u - e)) / (2 * e)
    slack = 1e-8 * (1 + np.abs(dh) * (1 + np.abs(u)))  # e^2 times a third derivative, and 64-bit roundings over e
    _, _, size = ref.swiglu_backward(g, u, dh)
    close(got[:, :f], dg, tolerance(dg, size, g) + slack, "dgate")
    close(got[:, f:], du, tolerance(du, np.abs(du), g) + slack, "dup")


def test_extreme_gates(zc):
    """Gates far on both sides, infinities and NaN: the value the formula has, or NaN where it has none."""
    g = np.array([-1e38, -200.0, -100.0, -88.0, -20.0, -0.0, 0.0, 20.0, 100.0, 1e38, np.inf, np.nan] + [0.0] * 4)
    u = np.full(16, 2.0)
    o = forward(zc, np.concatenate([g, u])[None], 16, 0)
    h = o["h"].numpy()[0]
    assert np.isnan(h[11]) and h[10] == np.inf
    with np.errstate(over="ignore"):
        want = np.where(np.isfinite(g), g / (1 + np.exp(-g)) * 2, 0.0)
    close(h[:10], ref.bf16(want[:10]), tolerance(want, np.abs(want), np.minimum(np.abs(g), 200.0))[:10], "h")
    out = Out((1, 32), torch.bfloat16)
    dh = np.ones((1, 16))
    zc.zc_swiglu_backward(o["kq"], o["ks"], 1, 16, bf16_device(dh), 16, out, 32)
    assert np.isfinite(out.numpy()[0, :10]).all()


def test_gates_whose_sigmoid_is_below_the_normal_numbers(zc):
    """sigmoid(-88) to sigmoid(-104) have few or no digits in 32 bits; their products with large values have all of theirs."""
    m, f = 6, 128
    r = np.random.default_rng(104)
    g = ref.bf16(-r.uniform(88.0, 104.0, (m, f)))
    u = ref.bf16(r.standard_normal((m, f)) * 2.0 ** np.array([20, 40, 50, 70, 90, 110])[:, None])
    gu = np.concatenate([g, u], axis=1)
    o = forward(zc, gu, f, 0)
    want = ref.swiglu(g, u)
    close(o["h"].numpy(), want, tolerance(want, np.abs(want), g), "h")
    dh = ref.bf16(r.standard_normal((m, f)) * 2.0 ** np.array([60, 50, 30, 20, 10, 5])[:, None])
    out = Out((m, 2 * f), torch.bfloat16)
    zc.zc_swiglu_backward(o["kq"], o["ks"], m, f, bf16_device(dh), f, out, 2 * f)
    got, kq, ks = out.numpy(), o["kq"].numpy(), o["ks"].numpy()
    g, u = ref.values(kq[:, :f], ks[:, :1], ref.E4M3, f), ref.values(kq[:, f:], ks[:, 1:2], ref.E4M3, f)
    dg, du, size = ref.swiglu_backward(g, u, dh)
    close(got[:, :f], dg, tolerance(dg, size, g), "dgate")
    close(got[:, f:], du, tolerance(du, np.abs(du), g), "dup")
