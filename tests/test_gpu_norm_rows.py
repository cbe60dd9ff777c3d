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


def check_plain(c):
    """Sum and norm without the 8-bit blocks, and nothing written between the rows."""
    o = c.forward()
    r, er, y, ey = ref.norm(c.x, c.z, c.after, c.before, c.gate, c.row_gate, c.scale)
    close(o["r"].numpy()[:, :c.cols], r, half_step(c.f32) * np.abs(r) + 2 * er, "r")
    close(o["y"].numpy()[:, :c.cols], y, ref.BF16_HALF_STEP * np.abs(y) + 2 * ey, "y")
    if c.gap:
        for v in (o["r"], o["y"]):
            assert bool((v.t[:, c.cols:].contiguous().view(torch.uint8) == 0xA5).all())


# rows on 16 bytes and off them, whole pieces of eight and tails, every team, and more rows than the blocks take at once
FORMS = SHAPES + [(5, 7168, 8, 8), (4, 7168, 1, 0), (3, 4097, 7, 5), (3, 16383, 2, 1), (5000, 72, 0, 0), (1500, 1100, 3, 1)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,gap,offset", FORMS)
def test_forward_without_blocks(zc, m, n, gap, offset, f32):
    check_plain(Case(zc, m, n, gap=gap, offset=offset, f32=f32, params_f32=f32, row_gate=True))
    check_plain(Case(zc, m, n, gap=gap, offset=offset, f32=f32, params_f32=not f32, bias=True, after=ref.LAYER, before=ref.LAYER))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kw", KINDS + [dict(weights=False), dict(gate=False), dict(z=False), dict(z=False, before=ref.LAYER),
                                        dict(gate=False, row_gate=True, bias=True), dict(scale=0.0), dict(scale=-3.0),
                                        dict(params_f32=True, bias=True)])
def test_kinds_without_blocks(zc, kw, f32):
    for m, n, gap, offset in ((5, 200, 0, 0), (5, 203, 2, 1), (3, 2500, 0, 0), (3, 2504, 8, 8)):
        check_plain(Case(zc, m, n, gap=gap, offset=offset, f32=f32, **kw))


def test_rows_in_turn(zc):
    """More rows than the grid's teams: every row is what it is alone."""
    c = Case(zc, 2300, 4100, gap=1, offset=1, row_gate=True, bias=True)
    check_plain(c)


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


# constant rows: sums that fit a float and sums that do not, of either sign, small and 0
CONSTANTS = [2.0 ** 50, 1e20, -1e30, 1e37, -3e38, 3.0, 2.0 ** -100, 0.0]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [1e-6, 1e-20, 1e-30])
@pytest.mark.parametrize("n", [1, 64, 700, 1030, 2500, 5125, 7168, 16384])
def test_constant_rows_under_a_layer_norm(zc, n, eps, f32):
    """A constant row differs from its mean nowhere: its norm is the bias, whatever its size and that of eps."""
    v = (ref.f32 if f32 else ref.bf16)(np.repeat(np.array(CONSTANTS)[:, None], n, axis=1))
    # beside rows that are not
    v[5] = ref.bf16(np.random.default_rng(n).standard_normal(n))
    still = [i for i in range(len(CONSTANTS)) if i != 5]
    for bias in (True, False):
        c = with_rows(zc, v, None, f32, after=ref.NONE, before=ref.LAYER, eps=eps, bias=bias)
        y = c.forward(q=True)["y"].numpy()
        want = ref.bf16(c.before.b) if bias else np.zeros(n)
        assert np.array_equal(y[still], np.broadcast_to(want, y[still].shape))
        assert np.array_equal(c.forward()["y"].numpy(), y)
        o = c.backward(dr=False)
        assert np.isfinite(o["dx"].numpy()).all()
        if n > 1:  # (of one column the gradient is what rounding leaves of 0)
            c.check_backward()
        c.dy = c.dy * (np.arange(len(CONSTANTS)) != 5)[:, None]
        assert not c.backward()["dw2"].numpy().any()
    # the block's output
    z = ref.bf16(v)
    c = with_rows(zc, np.zeros_like(v), z, f32, after=ref.LAYER, before=ref.NONE, eps=eps, gate=False, scale=1.0, bias=True)
    for q in (False, True):
        r = c.forward(q=q)["r"].numpy()
        assert np.array_equal(r[still], np.broadcast_to(half(c.after.b, f32), r[still].shape))
    if n > 1:
        c.check_backward()


def half(v, f32):
    return ref.f32(v) if f32 else ref.bf16(v)


def wide_rows(n, f32):
    """Rows whose values lie further from their mean than the largest float."""
    big = 3e38
    x = np.full((5, n), -big)
    x[0, 0] = big
    x[1] = big
    x[1, n // 2] = -big
    x[2, ::2] = big
    x[3] = np.random.default_rng(n).uniform(-big, big, n)
    x[4] = np.random.default_rng(n).standard_normal(n)
    return (ref.f32 if f32 else ref.bf16)(x)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", [9, 700, 1030, 5125, 7168])
def test_layer_norm_over_the_whole_range(zc, n, f32):
    x = wide_rows(n, f32)
    c = with_rows(zc, x, None, f32, after=ref.NONE, before=ref.LAYER, bias=True)
    c.check_forward()
    check_plain(c)
    c.check_backward()
    z = wide_rows(n, False)
    # (a large scale: the gradient, divided by the deviation, stays above the smallest normal number)
    c = with_rows(zc, np.zeros((5, n)), z, f32, after=ref.LAYER, before=ref.NONE, scale=2.0 ** 60, gate=False)
    c.check_forward()
    check_plain(c)
    c.check_backward()


@pytest.mark.parametrize("after", [ref.RMS, ref.LAYER])
@pytest.mark.parametrize("n", [64, 700, 5125, 7168])
def test_both_halves_out_of_range_at_once(zc, n, after):
    """Both norms measured again, in some of the rows that a workgroup holds and not in others."""
    x, z = wide_rows(n, True), wide_rows(n, False)[[4, 0, 1, 4, 2]]
    c = with_rows(zc, x, z, True, after=after, before=ref.LAYER, scale=2.0 ** 60, bias=True, row_gate=True)
    c.check_forward()
    check_plain(c)
    c.check_backward()
