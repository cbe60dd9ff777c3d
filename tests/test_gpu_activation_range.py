"""Activations and their slopes at the ends of their range against 64 bits: gradients beside vanishing slopes, infinities, and the
digits of 32-bit results."""
import numpy as np
import pytest
import torch

import block_ref as ref
from moe_gpu import Out, close, device, moe

pytestmark = pytest.mark.gpu
EPS = ref.EPS32
RELU, SILU, GELU, GELU_TANH, SIGMOID = range(1, 6)
LOWEST = float(torch.finfo(torch.bfloat16).min)


@pytest.fixture(scope="module")
def zc():
    return moe()


def values(zc, v, act):
    """The activation of 32-bit values: an empty contraction, and the values as the bias."""
    out = Out((1, v.size), torch.float32)
    e = zc.epilogue(device(v).float(), act)
    zc.zc_matmul(None, 1, 0, None, v.size, 0, 0, e, out, zc.ZC_F32, v.size)
    return out.numpy()[0]


def slopes(zc, d, v, act, scale=1.0):
    """scale * d * slope at BF16 values, through the bias sum of a single row."""
    n = v.size
    dbias = Out((n,), torch.float32)
    ws = torch.full((zc.zc_activation_backward_workspace_bytes(1, n),), 0xFF, dtype=torch.uint8, device="cuda")
    zc.zc_activation_backward(device(np.broadcast_to(d, v.shape)[None]).float(), zc.ZC_F32, 1, n, n, device(v[None]).bfloat16(), n,
                              act, scale, None, 0, dbias, ws, ws.numel())
    return dbias.numpy()


@pytest.mark.parametrize("d", [4.0, -100.0, 2.0 ** 80, -2.0 ** 126])
@pytest.mark.parametrize("act", [RELU, SILU, GELU, GELU_TANH, SIGMOID])
def test_large_gradients_beside_vanishing_slopes(zc, act, d):
    """Finite values and gradients have finite slopes times gradients, 0 where the slope is, the lowest BF16 value among
    the values.  Past |v| = 300 every slope is 1 or 0 in 32 bits, whatever the gradient; before it, where 2^126 times the slope's
    own 2^-149 could be seen, only the size is looked at."""
    v = ref.bf16(np.concatenate([[LOWEST, -1e38, -1e37, -1e30, -1e10, -1000.0, -310.0], -np.geomspace(90, 300, 60)]))
    v = np.concatenate([v, -v])
    got = slopes(zc, d, v, act)
    assert np.isfinite(got).all()
    far = np.abs(v) > 300
    want = d * np.where(v > 0, 0.0 if act == SIGMOID else 1.0, 0.0)
    assert np.array_equal(got[far], want[far])
    # |slope - its limit| <= (1 + |v|) e^-|v| < 1e-37 past 90
    close(got[~far], want[~far], 2 * EPS * np.abs(want[~far]) + abs(d) * 1e-37, "slopes")


@pytest.mark.parametrize("act", [RELU, SILU, GELU, GELU_TANH, SIGMOID])
def test_infinities(zc, act):
    """The activations' limits, and their slopes'; NaN stays, beside values that are what they are without it."""
    v = np.array([np.inf, 1.0, -np.inf, -1.0, np.nan, 2.0, LOWEST, -LOWEST])
    got = values(zc, v, act)
    plain = values(zc, np.array([1.0, -1.0, 2.0]), act)
    top = 1.0 if act == SIGMOID else np.inf
    assert np.array_equal(got[[0, 2]], [top, 0.0])
    assert np.isnan(got[4]) and np.array_equal(got[[1, 3, 5]], plain)
    assert np.array_equal(got[[6, 7]], [0.0, 1.0 if act == SIGMOID else -LOWEST])
    for d in (1.0, -3.0, 2.0 ** 100):
        got = slopes(zc, d, v, act)
        plain = slopes(zc, d, np.array([1.0, -1.0, 2.0]), act)
        one = 0.0 if act == SIGMOID else d
        assert np.array_equal(got[[0, 2]], [one, 0.0]) and np.array_equal(got[[6, 7]], [0.0, one])
        assert np.isnan(got[4]) and np.array_equal(got[[1, 3, 5]], plain)


@pytest.mark.parametrize("act", [RELU, SILU, GELU, GELU_TANH])
def test_infinite_gradients(zc, act):
    """A gradient that has left the range of a float is multiplied by the slope: an infinity of its sign right of 0."""
    v = ref.bf16(np.array([0.5, 3.0, 20.0, 30.0, 100.0, 1e30]))
    for d in (np.inf, -np.inf):
        assert np.array_equal(slopes(zc, d, v, act), np.full(v.size, d))


@pytest.mark.parametrize("m", [1, 40, 200])
def test_infinite_sums(zc, m):
    """GELU of an infinite sum in the kernels of few rows, of tiles and of split contractions."""
    for n, k in ((40, 64), (128, 8192)):
        a, w = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda"), torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
        a[0, 3] = float("inf")
        ws = torch.full((max(16, zc.zc_matmul_workspace_bytes(m, n, k)),), 0xFF, dtype=torch.uint8, device="cuda")
        out = Out((m, n), torch.bfloat16)
        zc.zc_matmul(a, m, k, w, n, k, k, zc.epilogue(activation=GELU), out, zc.ZC_BF16, n, ws, ws.numel())
        got = out.numpy()
        assert np.isposinf(got[0]).all() and not got[1:].any()


def far_and_near(low, high):
    """32-bit values, spread evenly and towards 0."""
    g = np.random.default_rng(11)
    v = np.concatenate([g.uniform(low, high, 20000), [-5.0, -20.0, -80.0], np.geomspace(1e-6, 1, 500), -np.geomspace(1e-6, 1, 500)])
    return ref.f32(v[(v >= low) & (v <= high)])


@pytest.mark.parametrize("act", [SILU, SIGMOID])
def test_digits_of_sigmoids(zc, act):
    """sigmoid = m r 2^2h, m = 2^f with |f| <= 1 known to 2^-24 (0.7 half steps of m), the hardware's 2^f and 1 / x a unit each (2 half
    steps), one for 1 + e and one for m r, e's own 2.7 in 1 + e: 6.7 half steps, and one for the product with v."""
    v = far_and_near(-86.0, 30.0)
    want = ref.activation(v, act)[0]
    close(values(zc, v, act), want, 8 * EPS * np.abs(want), "activation %d" % act)


@pytest.mark.parametrize("act", [SILU, SIGMOID])
def test_digits_of_their_slopes(zc, act):
    """SILU: q = s (1 - |v| r) left of 0 and 1 - q right of it, with s = sigmoid(-|v|) off by 5.7 half steps, r = 1 - s by 4.4, one for the
    difference and each product.  SIGMOID: s r."""
    v = np.unique(ref.bf16(far_and_near(-85.0, 30.0)))
    want = ref.activation(v, act)[1]
    s, q = ref._sigmoid(v), ref._sigmoid(-v)
    tol = 14 * EPS * np.abs(want) if act == SIGMOID else EPS * (12 * np.abs(want) + 8 * np.abs(v) * q * s)
    close(slopes(zc, 1.0, v, act), want, tol, "slope %d" % act)


def test_digits_of_gelu(zc):
    """v Phi(v), left of 0 the tail m root^2: t = 1 / (1 + x / 2) is off by 3.5 half steps, which count 1 + |t p'(t) / p(t)| <= 2.26
    times; the polynomial's steps and coefficients by 5.6, its fit by 0.2, m's product by one, each root by 3 (the hardware's unit and the
    carried rest), three products, and half of one for a constant: 25 half steps.  Right of 0 the tail is taken off v."""
    v = far_and_near(-12.5, 12.5)
    want = ref.activation(v, GELU)[0]
    tail = np.abs(v) * (0.5 * ref._erfc(np.abs(v) / 2 ** 0.5))
    close(values(zc, v, GELU), want, EPS * (25 * tail + 2 * np.where(v > 0, want, 0)), "gelu")
    v = np.unique(ref.bf16(v))
    want = ref.activation(v, GELU)[1]
    tail, bell = 0.5 * ref._erfc(np.abs(v) / 2 ** 0.5), np.abs(v) * np.exp(-v * v / 2) / (2 * np.pi) ** 0.5
    # the tail's 16 half steps before its roots, six for the roots and three products for both terms, three for sum and result
    close(slopes(zc, 1.0, v, GELU), want, EPS * (13 * np.abs(want) + 25 * tail + 13 * bell), "slope")
