"""Routing and its gradient against the formulas in 64 bits: ids exactly, weights
and gradients to the roundings that the 32-bit results make."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from moe_gpu import Out, close, device, moe, to_numpy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


def logits_on_device(x, bf16, stride):
    t, e = x.shape
    buf = torch.full((t, stride), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    buf[:, :e] = torch.from_numpy(x).to(torch.float32).to(buf.dtype).cuda()
    return buf


def run(zc, x, cfg, bias=None, bf16=False, stride=None):
    t, e = x.shape
    stride = stride or e
    logits = logits_on_device(x, bf16, stride)
    ids, w = Out((t, cfg.top_k), torch.int32), Out((t, cfg.top_k), torch.float32)
    b = None if bias is None else device(bias.astype(np.float32))
    zc.zc_route(logits, zc.ZC_BF16 if bf16 else zc.ZC_F32, t, stride, b, cfg, ids, w)
    return ids.numpy(), w.numpy(), logits


# softmax or sigmoid, a sum of at most 32 scores, a quotient, a product, and each 32-bit score's own rounding
def weight_tolerance(w, k):
    return (k + 6) * ref.F32_HALF_STEP * np.abs(w) + 2.0 ** -140


CASES = [
    dict(t=1, experts=256, top_k=8, score="sigmoid", groups=8, group_top=4, group_score=2),
    dict(t=5, experts=1, top_k=1, score="softmax"),
    dict(t=67, experts=64, top_k=1, score="sigmoid"),
    dict(t=130, experts=65, top_k=7, score="softmax", groups=5, group_top=3, group_score=1),
    dict(t=33, experts=160, top_k=6, score="softmax", groups=8, group_top=3, group_score=2, renormalise=False, scale=2.5),
    dict(t=300, experts=384, top_k=8, score="sigmoid", renormalise=True, scale=2.446),
    dict(t=19, experts=1024, top_k=32, score="sigmoid", groups=64, group_top=5, group_score=2),
    dict(t=9, experts=1000, top_k=31, score="softmax", groups=4, group_top=4, group_score=2),
    dict(t=40, experts=64, top_k=9, score="sigmoid", groups=64, group_top=9, group_score=2),
    dict(t=40, experts=12, top_k=12, score="softmax", groups=2, group_top=2, group_score=2),
    dict(t=2049, experts=128, top_k=8, score="softmax"),
]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d-%s" % (c["t"], c["experts"], c["score"]))
def test_route(zc, case, bf16, bias):
    kw = dict(case)
    t = kw.pop("t")
    cfg = zc.route_config(**kw)
    g = np.random.default_rng([t, cfg.experts, int(bf16), int(bias)])
    x = g.standard_normal((t, cfg.experts)).astype(np.float32).astype(np.float64)
    if bf16:
        x = ref.bf16(x)  # eight bits of mantissa: ties between experts are common
    b = g.standard_normal(cfg.experts).astype(np.float32).astype(np.float64) * 0.05 if bias else None
    b = None if b is None else b.astype(np.float32).astype(np.float64)
    ids, w, _ = run(zc, x, cfg, b, bf16, stride=cfg.experts + 3)
    want_ids, want_w, _ = ref.route(x, b, cfg)
    assert np.array_equal(ids, want_ids)
    close(w, want_w, weight_tolerance(want_w, cfg.top_k), "weights")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_masks_and_special_values(zc, score, groups):
    e, k = 64, 8
    cfg = zc.route_config(e, k, score, groups=groups, group_top=min(groups, 2), group_score=2 if groups > 1 else 1)
    inf, nan = np.inf, np.nan
    x = np.random.default_rng(7).standard_normal((12, e)).astype(np.float32).astype(np.float64)
    x[0] = 1.5                      # every expert ties
    x[1] = -inf                     # nothing is left
    x[2] = -inf
    x[2, 40:43] = (0.0, 2.0, 1.0)   # three are left, fewer than top_k
    x[3] = np.finfo(np.float32).min  # masked with the type's lowest value
    x[4] = np.finfo(np.float32).min
    x[4, 63] = 0.0
    x[5, ::2] = x[5, 1::2]          # ties in pairs
    x[6, 10] = nan
    x[7, 10] = inf
    x[8] = nan
    x[9] = -80.0 - np.arange(e)     # sigmoid scores far below 1
    x[10] = 100.0                   # sigmoid scores that round to 1 alike
    x[11] = np.where(np.arange(e) % 2 == 0, 0.0, -0.0)
    ids, w, _ = run(zc, x, cfg)
    want_ids, want_w, _ = ref.route(x, None, cfg)
    assert np.array_equal(ids, want_ids)
    close(w, want_w, weight_tolerance(want_w, k) + 2.0 ** -126, "weights")
    assert not w[1].any() and np.array_equal(np.sort(ids[1]), np.unique(ids[1]))


def test_bias_masks_experts(zc):
    """A bias of -inf takes experts out of the choice, and leaves the weights alone."""
    cfg = zc.route_config(48, 4, "sigmoid", scale=1.5)
    g = np.random.default_rng(9)
    x = g.standard_normal((50, 48)).astype(np.float32).astype(np.float64)
    b = np.where(np.arange(48) % 3 == 0, 0.0, -np.inf)
    ids, w, _ = run(zc, x, cfg, b)
    want_ids, want_w, _ = ref.route(x, b, cfg)
    assert np.array_equal(ids, want_ids) and not (ids % 3).any()
    close(w, want_w, weight_tolerance(want_w, 4))


def test_near_ties_are_decided_in_64_bits(zc):
    """Scores that a 32-bit sigmoid cannot tell apart."""
    e = 256
    cfg = zc.route_config(e, 8, "sigmoid")
    base = np.float32(3.0)
    steps = np.random.default_rng(3).permutation(e)
    x = np.empty((4, e), dtype=np.float32)
    for r in range(4):
        x[r] = base + np.roll(steps, r).astype(np.float32) * np.float32(2.0 ** -22)
    ids, w, _ = run(zc, x.astype(np.float64), cfg)
    want_ids, _, _ = ref.route(x.astype(np.float64), None, cfg)
    assert np.array_equal(ids, want_ids)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", [1, 2])
def test_near_tied_groups_are_decided_in_64_bits(zc, score, group_score):
    """Groups whose scores differ by less than 32 bits show; in the last rows their second and third experts do too."""
    g = np.random.default_rng(31)
    groups, per = 8, 32
    cfg = zc.route_config(groups * per, 6, score, groups=groups, group_top=3, group_score=group_score)
    x = np.empty((24, groups, per), dtype=np.float32)
    for r in range(24):
        x[r] = g.standard_normal((groups, per)).astype(np.float32) * 0.25 - 2
        x[r, :, 5] = np.float32(1.5) + g.permutation(groups).astype(np.float32) * np.float32(2.0 ** -23)
        x[r, :, 9] = np.float32(1.0)
        if r >= 16:
            x[r, :, 20] = np.float32(1.0) + g.integers(-1, 2, groups).astype(np.float32) * np.float32(2.0 ** -23)
    x = x.reshape(24, -1).astype(np.float64)
    ids, w, _ = run(zc, x, cfg)
    want_ids, want_w, _ = ref.route(x, None, cfg)
    assert np.array_equal(ids, want_ids)
    close(w, want_w, weight_tolerance(want_w, 6), "weights")


def backward(zc, x, cfg, ids, dw, bf16, logits):
    t, e = x.shape
    out = Out((t, e + 5), torch.bfloat16 if bf16 else torch.float32)
    zc.zc_route_backward(logits, zc.ZC_BF16 if bf16 else zc.ZC_F32, t, logits.shape[1], cfg, device(ids.astype(np.int32)),
                         device(dw.astype(np.float32)), out, e + 5)
    full = out.numpy()
    raw = out.t.contiguous().view(torch.uint8).view(t, e + 5, -1)[:, e:]
    assert bool((raw == 0xA5).all()), "written between the rows"
    return full[:, :e]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d-%s" % (c["t"], c["experts"], c["score"]))
def test_route_backward(zc, case, bf16):
    kw = dict(case)
    t = kw.pop("t")
    cfg = zc.route_config(**kw)
    g = np.random.default_rng([t, cfg.experts, 5])
    x = g.standard_normal((t, cfg.experts)).astype(np.float32).astype(np.float64)
    if bf16:
        x = ref.bf16(x)
    ids, _, logits = run(zc, x, cfg, None, bf16, stride=cfg.experts + 1)
    dw = g.standard_normal((t, cfg.top_k)).astype(np.float32).astype(np.float64)
    got = backward(zc, x, cfg, ids, dw, bf16, logits)
    want, size = ref.route_backward(x, cfg, ids, dw)
    # 32-bit exponentials (2 ulp each), sums over the experts in trees, and about ten more operations
    tol = 48 * ref.F32_HALF_STEP * size + (ref.BF16_HALF_STEP * np.abs(want) if bf16 else 0.0) + 2.0 ** -133
    close(got, want, tol, "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_backward_against_differences(zc, score, renormalise):
    """The kernel's gradient against central differences of the 64-bit weights (the choice held fixed)."""
    cfg = zc.route_config(32, 4, score, groups=4, group_top=2, group_score=2, renormalise=renormalise, scale=1.7)
    g = np.random.default_rng(11)
    x = g.standard_normal((6, 32)).astype(np.float32).astype(np.float64)
    ids, _, logits = run(zc, x, cfg)
    dw = g.standard_normal((6, 4)).astype(np.float32).astype(np.float64)
    got = backward(zc, x, cfg, ids, dw, False, logits)

    def loss(v):
        _, _, s = ref.route(v, None, cfg)
        p = np.take_along_axis(s, ids, axis=1)
        w = p / (p.sum(axis=1, keepdims=True) + 1e-20) if renormalise else p
        return (w * float(np.float32(1.7)) * dw).sum(axis=1)

    h = 1e-5
    for j in range(32):
        d = np.zeros_like(x)
        d[:, j] = h
        diff = (loss(x + d) - loss(x - d)) / (2 * h)
        # differences: h^2 times a third derivative (below 10 here) and 64-bit roundings over h; the kernel's 32 bits
        close(got[:, j], diff, 1e-8 + 1e-5 * np.abs(dw).max(axis=1), "logit %d" % j)


def test_route_backward_ids_out_of_range_and_masked_rows(zc):
    cfg = zc.route_config(40, 3, "softmax")
    x = np.random.default_rng(2).standard_normal((4, 40)).astype(np.float32).astype(np.float64)
    x[3] = -np.inf
    ids, _, logits = run(zc, x, cfg)
    dw = np.full((4, 3), 1e30)
    dw[:3] = 1.0
    bad = ids.copy()
    bad[1, 1], bad[2] = -1, (40, -5, 1 << 30)
    got = backward(zc, x, cfg, bad, dw, False, logits)
    want, size = ref.route_backward(x[:1], cfg, ids[:1], dw[:1])
    close(got[:1], want, 48 * ref.F32_HALF_STEP * size + 2.0 ** -133)
    p = to_numpy(torch.softmax(logits[1].double(), 0))
    d = np.zeros(40)
    on = [int(ids[1, 0]), int(ids[1, 2])]
    total = p[on].sum() + 1e-20
    d[on] = (1.0 - p[on].sum() / total) / total
    close(got[1], p * (d - (d * p).sum()), 48 * ref.F32_HALF_STEP * 4 * p / total)
    assert not got[2].any() and not got[3].any()


def test_route_on_another_stream(zc):
    cfg = zc.route_config(128, 8, "softmax")
    x = np.random.default_rng(8).standard_normal((4096, 128)).astype(np.float32).astype(np.float64)
    logits = logits_on_device(x, False, 128)
    ids, w = Out((4096, 8), torch.int32), Out((4096, 8), torch.float32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    zc.zc_route(logits, zc.ZC_F32, 4096, 128, None, cfg, ids, w, stream=st)
    st.synchronize()
    assert np.array_equal(ids.numpy(), ref.route(x, None, cfg)[0])


def test_route_more_tokens_than_a_launch_takes(zc):
    t, period = 16 * 2 ** 20 + 21, 1009
    x = np.random.default_rng(3).standard_normal((period, 4)).astype(np.float32)
    cfg = zc.route_config(4, 1, score="sigmoid", renormalise=False)
    logits = torch.from_numpy(x).cuda().repeat(t // period + 1, 1)[:t].contiguous()
    ids, w = Out((t, 1), torch.int32), Out((t, 1), torch.float32)
    zc.zc_route(logits, zc.ZC_F32, t, 4, None, cfg, ids, w)
    ids.numpy(), w.numpy()
    best = x.argmax(axis=1)
    value = 1 / (1 + np.exp(-x.astype(np.float64).max(axis=1)))
    at = torch.arange(t, device="cuda") % period
    assert torch.equal(ids.t[:, 0].long(), torch.from_numpy(best).cuda()[at])
    want = torch.from_numpy(value).cuda()[at]
    assert bool(((w.t[:, 0].double() - want).abs() <= torch.from_numpy(weight_tolerance(value, 1)).cuda()[at]).all())
