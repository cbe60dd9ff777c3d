"""Routing by groups of experts whose scores are negative or of both signs: balance
biases of any sign, and numbers of groups from 2 to 16.  Ids are
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
