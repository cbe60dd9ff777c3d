"""Norms in the form that users of BF16 results call, and rows that are constant or fill the range of a float, against 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from moe_gpu import bf16_device, close, moe
from test_gpu_norm import KINDS, SHAPES, Case, half_step, stream_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


def with_rows(zc, x, z, f32, **kw):
    """A case of the given rows."""
    c = Case(zc, *x.shape, f32=f32, z=z is not None, **kw)
    c.x, c.z = x, z
    c.dx, c.dz = stream_device(x, f32, x.shape[1]), None if z is None else bf16_device(z, x.shape[1])
    return c


def test_nearly_constant_rows(zc):
    """One value of a row a few steps from the others: the deviation is theirs, not that of a rounded mean."""
    for n in (300, 700, 5125, 7168):
        x = np.full((4, n), 1e6)
        x[0, 5] += 0.0625 * 3
        x[1, :7] -= 0.0625
        x[2, n // 2:] += 0.0625
        x[3, -1] = 1e6 + 1
        c = with_rows(zc, x, None, True, after=ref.NONE, before=ref.LAYER, eps=1e-12, weights=False)
        hat = c.before.apply(x)[0]
        y = c.forward()["y"].numpy()
        # the mean, its correction and the deviation: about a hundred half steps of the deviation and of one step of 1e6
        rs = ref.stat(x, ref.LAYER, 1e-12)[1]
        tol = ref.BF16_HALF_STEP * np.abs(hat) + ref.EPS32 * 128 * (np.abs(hat) + 1 + 0.0625 * 64 * rs)
        close(y, hat, tol, "y of %d columns" % n)
