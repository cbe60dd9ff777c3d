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
