"""Balance and z losses at the ends of their range: few roundings where the sums are exact, and infinite logits."""
import numpy as np
import pytest

import block_ref as ref
from moe_gpu import moe
from test_gpu_balance import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (4, 3), (64, 6), (256, 7)])
def test_losses_of_exact_sums_are_rounded_once(zc, experts, top_k, sigmoid):
    """Equal logits: every score is 1 / experts, a power of two, and sums of them, and of whole squares, are exact.  What is left is
    the quotient."""
    lengths = np.arange(1, 90)
    tokens = int(lengths.sum())
    c = Case(zc, tokens, experts, top_k, sigmoid, offsets=[0, *np.cumsum(lengths)])
    c.x = np.zeros((tokens, experts))
    if experts == 1:  # the logarithm of the sum is the logit
        c.x[:, 0] = np.random.default_rng(3).integers(-9, 10, tokens) * (not sigmoid)
    c.load()
    o, (_, _, loss, z) = c.forward(), c.want()
    assert np.array_equal(o["loss"].numpy(), ref.f32(loss))
    if experts == 1:
        assert np.array_equal(o["zloss"].numpy(), ref.f32(z))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("experts", [12, 200, 300])
def test_infinite_logits(zc, experts, sigmoid):
    """The logarithm of a sum that is infinite: infinite.  A sigmoid score of +inf is 1, a softmax has no value; NaN stays NaN, and
    all of it in its sequence."""
    c = Case(zc, 100, experts, 2, sigmoid, offsets=[0, 20, 40, 60, 80, 100])
    clean = {k: v.numpy().copy() for k, v in c.forward().items()}
    c.d["x"][25, 3] = float("inf")
    c.d["x"][45, [1, 11]] = float("inf")
    c.d["x"][45, 2] = float("-inf")
    c.d["x"][65, 3], c.d["x"][65, 7] = float("inf"), float("nan")
    o = c.forward()
    z, loss = o["zloss"].numpy(), o["loss"].numpy()
    assert np.isposinf(z[[1, 2]]).all() and np.isnan(z[3])
    assert np.array_equal(z[[0, 4]], clean["zloss"][[0, 4]]) and np.array_equal(loss[[0, 4]], clean["loss"][[0, 4]])
    assert np.array_equal(o["counts"].numpy(), clean["counts"])
    assert np.isnan(loss[3]) and (np.isfinite(loss[[1, 2]]).all() if sigmoid else np.isnan(loss[[1, 2]]).all())
    if sigmoid:
        x = c.x.copy()
        x[25, 3] = x[45, 1] = x[45, 11] = 200.0  # whose sigmoid is 1 too
        x[45, 2] = -np.inf
        want = ref.balance(x, c.ids, c.mask, c.offsets, experts, 2, True)[2]
        assert (np.abs(loss - want)[[1, 2]] <= 500 * ref.EPS32 * want[[1, 2]]).all()
