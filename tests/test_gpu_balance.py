"""Copies of every expert, balance and z losses and the logits' gradient against 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from moe_gpu import Out, close, device, moe

pytestmark = pytest.mark.gpu
EPS = ref.EPS32


@pytest.fixture(scope="module")
def zc():
    return moe()


class Case:
    def __init__(self, zc, tokens, experts, top_k, sigmoid=False, offsets=None, mask=False, bf16=False, gap=0, spread=1.0, seed=0):
        g = np.random.default_rng([tokens, experts, top_k, seed])
        self.zc, self.tokens, self.experts, self.top_k, self.sigmoid, self.gap = zc, tokens, experts, top_k, sigmoid, gap
        self.x = (ref.bf16 if bf16 else ref.f32)(spread * g.standard_normal((tokens, experts)))
        self.ids = g.integers(-1, experts + 1, (tokens, top_k)).astype(np.int32)
        self.mask = (g.random(tokens) < 0.7).astype(np.uint8) if mask else None
        self.given = offsets
        self.offsets = np.array([0, tokens] if offsets is None else offsets, dtype=np.int32)
        self.s = len(self.offsets) - 1
        self.bf16, self.kind = bf16, zc.ZC_BF16 if bf16 else zc.ZC_F32
        self.t = torch.bfloat16 if bf16 else torch.float32
        self.cfg = zc.route_config(experts, top_k, "sigmoid" if sigmoid else "softmax")
        self.dloss, self.dz = ref.f32(g.standard_normal(self.s)), ref.f32(0.1 * g.standard_normal(self.s))
        self.add = (ref.bf16 if bf16 else ref.f32)(0.01 * g.standard_normal((tokens, experts)))
        self.load()

    def load(self):
        def rows(v, fill=float("nan")):
            b = torch.full((max(self.tokens, 1), self.experts + self.gap), fill, dtype=self.t, device="cuda")
            b[:self.tokens, :self.experts] = device(v).to(self.t)
            return b
        self.d = dict(x=rows(self.x), add=rows(self.add), ids=device(self.ids),
                      mask=None if self.mask is None else device(self.mask),
                      off=None if self.given is None else device(self.offsets), dloss=device(self.dloss).float(),
                      dz=device(self.dz).float())

    def forward(self, loss=True, z=True):
        zc, s, e = self.zc, self.s, self.experts
        o = dict(counts=Out((s, e), torch.int32), used=Out((s,), torch.int32), loss=Out((s,), torch.float32),
                 zloss=Out((s,), torch.float32))
        ws = torch.full((zc.zc_balance_workspace_bytes(self.tokens, e, s),), 0xFF, dtype=torch.uint8, device="cuda")
        zc.zc_balance(self.d["x"] if loss or z else None, self.kind, self.tokens, e + self.gap, self.cfg, self.d["ids"],
                      self.d["mask"], s, self.d["off"], ws, ws.numel(), o["counts"], o["used"], o["loss"] if loss else None,
                      o["zloss"] if z else None)
        return o

    def argument(self):
        """The largest argument of an exponential that is not 0."""
        return 2 * np.abs(np.where(np.abs(self.x) < 1e30, self.x, 0)).max(initial=0)

    def want(self):
        return ref.balance(self.x, self.ids, self.mask, self.offsets, self.experts, self.top_k, self.sigmoid)

    def check_forward(self):
        """A score: exponential and its argument, the sum over the experts and its inverse, some 24 + |argument| half steps
        (sums of positive numbers, a hundred additions deep at most); the losses' sums over tokens and tiles a few
        hundred more, all of positive terms (the squares of the z loss: twice the logarithm's error, whose absolute part is that
        of the sum)."""
        o, (counts, used, loss, z) = self.forward(), self.want()
        assert np.array_equal(o["counts"].numpy(), counts) and np.array_equal(o["used"].numpy(), used)
        deep = 400 + self.tokens / 256
        arg = self.argument()
        close(o["loss"].numpy(), loss, EPS * (deep + arg) * np.abs(loss), "loss")
        _, _, lse, _ = ref.scores(self.x, self.sigmoid)
        lse = np.abs(lse).max(initial=0)
        close(o["zloss"].numpy(), z, EPS * (deep * np.abs(z) + 2 * (lse + 1) * (100 + arg)), "z")
        return o

    def backward(self, loss=True, z=True, add=True, in_place=False):
        zc, e = self.zc, self.experts
        o = self.forward()
        out = Out((max(self.tokens, 1), e + self.gap), self.t)
        given = self.d["add"] if add else None
        if in_place:
            out.t.copy_(given)
            given = out
        zc.zc_balance_backward(self.d["x"], self.kind, self.tokens, e + self.gap, self.cfg, self.d["mask"], self.s,
                               self.d["off"], o["counts"], o["used"], self.d["dloss"] if loss else None,
                               self.d["dz"] if z else None, given, e + self.gap, out, e + self.gap)
        return out

    def check_backward(self, loss=True, z=True, add=True, in_place=False):
        counts, used, _, _ = self.want()
        want, size = ref.balance_backward(self.x, self.mask, self.offsets, self.experts, self.top_k, self.sigmoid, counts,
                                          used, self.dloss if loss else None, self.dz if z else None,
                                          self.add if add else None)
        out = self.backward(loss, z, add, in_place)
        arg = self.argument()
        half = ref.BF16_HALF_STEP if self.bf16 else ref.F32_HALF_STEP
        # the scores' error enters each term once or twice, the sum over the experts another hundred half steps
        close(out.numpy()[:self.tokens, :self.experts], want, half * np.abs(want) + EPS * (400 + 4 * arg) * size + 2.0 ** -125,
              "dlogits")
        if self.gap:
            rest = out.t[:, self.experts:].contiguous().view(torch.uint8)
            if not in_place:
                assert bool((rest == 0xA5).all())


CASES = [dict(tokens=1, experts=1, top_k=1), dict(tokens=1, experts=8, top_k=2), dict(tokens=48, experts=8, top_k=2, gap=3),
         dict(tokens=700, experts=64, top_k=6), dict(tokens=333, experts=65, top_k=4, mask=True),
         dict(tokens=900, experts=160, top_k=6, offsets=[0, 1, 1, 300, 301, 880], mask=True),
         dict(tokens=5000, experts=256, top_k=8, offsets=[10, 2000, 2000, 4500]),
         dict(tokens=300, experts=257, top_k=3), dict(tokens=260, experts=1000, top_k=32, gap=1),
         dict(tokens=130, experts=1024, top_k=8, offsets=[0, 130]),
         dict(tokens=4200, experts=32, top_k=2, offsets=list(range(0, 4200, 41)), mask=True),
         dict(tokens=20000, experts=128, top_k=8, offsets=[0, 19999])]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kw", CASES)
def test_against_64_bits(zc, kw, sigmoid, bf16):
    c = Case(zc, sigmoid=sigmoid, bf16=bf16, **kw)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_parts_left_out(zc, sigmoid):
    c = Case(zc, 500, 96, 4, sigmoid, offsets=[3, 200, 470], mask=True)
    full = {k: v.numpy().copy() for k, v in c.forward().items()}
    for loss, z in ((True, False), (False, True), (False, False)):
        o = c.forward(loss, z)
        for k in ("counts", "used", *(("loss",) if loss else ()), *(("zloss",) if z else ())):
            assert np.array_equal(o[k].numpy(), full[k]), k
        for k in (*(() if loss else ("loss",)), *(() if z else ("zloss",))):
            assert bool((o[k].raw == 0xA5).all()), k
        c.check_backward(loss, z, add=True)
        c.check_backward(loss, z, add=False)
    c.check_backward(in_place=True)


def test_offsets_that_lead_nowhere(zc):
    """Offsets outside 0..tokens or not ascending are clamped; 1024 sequences, most of them empty."""
    for offsets in ([-5, 40, 30, 1 << 30], [200, 100, 100], [5, 5, 5, 5], [-(1 << 31), (1 << 31) - 1]):
        c = Case(zc, 150, 16, 2, offsets=offsets)
        c.check_forward()
        c.check_backward()
    g = np.random.default_rng(4)
    c = Case(zc, 3000, 24, 3, offsets=[0, *np.sort(g.integers(0, 3001, 1023)), 3000], mask=True)
    c.check_forward()
    c.check_backward()


def test_sequences_without_tokens(zc):
    """A mask that leaves nothing: no losses, no gradient, the other sequences as they are."""
    c = Case(zc, 90, 12, 2, offsets=[0, 30, 60, 90], mask=True)
    c.mask[30:60] = 0
    c.load()
    o = c.check_forward()
    assert o["used"].numpy()[1] == 0 and o["loss"].numpy()[1] == 0 and o["zloss"].numpy()[1] == 0
    c.check_backward()


def test_no_tokens(zc):
    for s in (1, 70):
        o = dict(counts=Out((s, 9), torch.int32), used=Out((s,), torch.int32), loss=Out((s,), torch.float32),
                 zloss=Out((s,), torch.float32))
        off = torch.zeros(s + 1, dtype=torch.int32, device="cuda")
        zc.zc_balance(None, zc.ZC_F32, 0, 9, zc.route_config(9, 2), None, None, s, off, None, 0, *o.values())
        for v in o.values():
            assert not v.numpy().any()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_special_logits(zc, sigmoid):
    """-inf and the type's lowest value as masks, rows of nothing else, and NaN where the mask hides it."""
    c = Case(zc, 40, 20, 3, sigmoid, mask=True, spread=3.0)
    c.x[::3, 4:9] = -np.inf
    c.x[1::3, 4:9] = float(torch.finfo(torch.float32).min)
    c.x[7] = -np.inf
    c.x[11] = -60.0
    c.x[12] = 100.0
    c.mask[[7, 11, 12]] = 1
    c.mask[[20, 21]] = 0
    c.load()
    c.d["x"][20], c.d["x"][21] = float("nan"), float("inf")
    c.check_forward()
    c.check_backward()


def test_nan_stays_in_its_sequence(zc):
    c = Case(zc, 60, 10, 2, offsets=[0, 20, 40, 60])
    clean = {k: v.numpy().copy() for k, v in c.forward().items()}
    c.d["x"][25, 3] = float("nan")
    o = c.forward()
    assert np.array_equal(o["counts"].numpy(), clean["counts"])
    for k in ("loss", "zloss"):
        got = o[k].numpy()
        assert np.isnan(got[1]) and np.array_equal(got[[0, 2]], clean[k][[0, 2]])


@pytest.mark.parametrize("sigmoid", [False, True])
def test_backward_against_differences(zc, sigmoid):
    """Central differences of the 64-bit losses along a random direction (the counts do not move)."""
    c = Case(zc, 30, 12, 3, sigmoid, offsets=[0, 11, 30])
    got = c.backward(add=False).numpy()[:30, :12]
    u = np.random.default_rng(8).standard_normal(c.x.shape)

    def total(s):
        _, _, loss, z = ref.balance(c.x + s * u, c.ids, c.mask, c.offsets, 12, 3, sigmoid)
        return (loss * c.dloss).sum() + (z * c.dz).sum()

    slope = (total(1e-5) - total(-1e-5)) / 2e-5
    counts, used, _, _ = c.want()
    want, size = ref.balance_backward(c.x, c.mask, c.offsets, 12, 3, sigmoid, counts, used, c.dloss, c.dz, None)
    # e^2 times a third derivative, and 64-bit roundings over e: below 1e-7 of the terms
    off = 1e-7 * (1 + (size * np.abs(u)).sum())
    assert abs((want * u).sum() - slope) <= off
    assert abs((got * u).sum() - slope) <= off + EPS * (400 + 4 * c.argument()) * (size * np.abs(u)).sum()


def test_repeats_itself(zc):
    c = Case(zc, 9000, 256, 8, True, offsets=[0, 8000, 9000])
    first = {k: v.numpy().copy() for k, v in c.forward().items()}
    grad = c.backward().numpy()
    for _ in range(3):
        for k, v in c.forward().items():
            assert np.array_equal(v.numpy(), first[k]), k
        assert np.array_equal(c.backward().numpy(), grad)
