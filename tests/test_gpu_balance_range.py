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
