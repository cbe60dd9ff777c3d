"""Routing by groups of experts whose scores are negative, of both signs, or cancel:
balance biases of any sign and size, and numbers of groups from 2 to 16.  Ids are
those of the 64-bit scores, exactly."""
import numpy as np
import pytest

import moe_ref as ref
from moe_gpu import close, moe
from test_gpu_moe_route import run, weight_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


def check(zc, x, bias, cfg, bf16=False):
    """x, bias: 64-bit values that the 32-bit arrays hold exactly."""
    ids, w, _ = run(zc, x, cfg, bias, bf16)
    want_ids, want_w, _ = ref.route(x, bias, cfg)
    wrong = int((ids != want_ids).any(axis=1).sum())
    assert wrong == 0, "%d of %d tokens have other experts" % (wrong, len(ids))
    close(w, want_w, weight_tolerance(want_w, cfg.top_k), "weights")


def f32(x):
    return np.asarray(x).astype(np.float32).astype(np.float64)


# biases around a value: group scores all positive, all negative, or of both signs (a sigmoid lies between 0 and 1)
@pytest.mark.parametrize("middle,spread", [(0.5, 0.05), (-0.9, 0.05), (-1.0, 0.1), (-2.0, 0.05), (-100.0, 0.5), (0.0, 3.0)])
@pytest.mark.parametrize("group_score", [1, 2])
@pytest.mark.parametrize("groups,group_top,per", [(2, 1, 24), (4, 2, 16), (5, 3, 13), (8, 4, 32), (12, 3, 8), (16, 5, 16),
                                                  (11, 10, 3), (3, 2, 1)])
def test_biases_of_either_sign(zc, groups, group_top, per, group_score, middle, spread):
    g = np.random.default_rng([groups, per, group_score, int(100 * abs(middle))])
    e = groups * per
    x, bias = f32(g.standard_normal((400, e))), f32(middle + spread * g.standard_normal(e))
    cfg = zc.route_config(e, min(8, group_top * per), "sigmoid", groups=groups, group_top=group_top,
                          group_score=group_score, scale=2.5)
    check(zc, x, bias, cfg)


@pytest.mark.parametrize("bf16", [False, True])
def test_negative_bias_bf16_logits(zc, bf16):
    g = np.random.default_rng(5)
    x = f32(g.standard_normal((500, 256)))
    x = ref.bf16(x) if bf16 else x
    cfg = zc.route_config(256, 8, "sigmoid", groups=8, group_top=4, group_score=2)
    check(zc, x, f32(-0.95 + 0.05 * g.standard_normal(256)), cfg, bf16)


# One expert of a group is lifted and the others are pushed down by as much: a group's two best scores cancel, and what is left
# has the roundings of the large ones.
@pytest.mark.parametrize("size", [1.0, 16.0, 64.0, 1e3, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("groups,group_top,per", [(2, 1, 4), (8, 3, 4), (16, 5, 2), (16, 8, 16)])
def test_scores_that_cancel(zc, groups, group_top, per, size):
    g = np.random.default_rng([groups, per, int(size)])
    bias = np.full((groups, per), -size)
    bias[np.arange(groups), g.integers(0, per, groups)] = size
    cfg = zc.route_config(groups * per, min(3, group_top * per), "sigmoid", groups=groups, group_top=group_top,
                          group_score=2)
    check(zc, f32(g.standard_normal((6000, groups * per))), f32(bias.reshape(-1)), cfg)


def test_two_groups_that_cancel(zc):
    """64-bit group scores 1.02975 and 1.02953; 32-bit sums come out the other way round."""
    x = f32([[0.24, -0.73, -0.12, -0.62, 0.31, -1.11, -0.24, -0.19]])
    bias = f32([1e4, -1e4, -1e4, -1e4] * 2)
    check(zc, x, bias, zc.route_config(8, 2, "sigmoid", groups=2, group_top=1, group_score=2))


@pytest.mark.parametrize("groups,group_top", [(4, 2), (8, 3), (16, 4)])
def test_masks_that_leave_one_expert(zc, groups, group_top):
    """A mask of -1e9 leaves one expert in some groups, none in others: their scores stand far below those of the rest, and
    still in the order of the 64-bit sums."""
    g = np.random.default_rng(groups)
    per = 8
    bias = np.zeros((groups, per))
    bias[0, 1:] = bias[1, :] = -1e9
    bias[2, :5] = -1e9
    bias = bias + 0.01 * g.standard_normal((groups, per))
    cfg = zc.route_config(groups * per, 6, "sigmoid", groups=groups, group_top=group_top, group_score=2)
    check(zc, f32(g.standard_normal((300, groups * per))), f32(bias.reshape(-1)), cfg)


def test_near_tied_groups_of_negative_scores(zc):
    """Group scores below zero that 32 bits cannot tell apart, fewer groups than a token has lanes."""
    g = np.random.default_rng(17)
    groups, per = 6, 16
    x = np.empty((40, groups, per), dtype=np.float32)
    for r in range(40):
        x[r] = g.standard_normal((groups, per)) * 0.25 - 2
        x[r, :, 3] = np.float32(1.5) + g.permutation(groups).astype(np.float32) * np.float32(2.0 ** -23)
        x[r, :, 9] = np.float32(1.0)
    cfg = zc.route_config(groups * per, 5, "sigmoid", groups=groups, group_top=2, group_score=2)
    check(zc, x.reshape(40, -1).astype(np.float64), np.full(groups * per, -1.5), cfg)
