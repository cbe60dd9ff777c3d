"""Norms with gate and residual sum, and their gradients, against 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from moe_gpu import Out, bf16_device, close, device, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


def half_step(f32):
    return ref.F32_HALF_STEP if f32 else ref.BF16_HALF_STEP


def stream_device(x, f32, stride, offset=0):
    """Rows `stride` apart, the gaps NaN, starting `offset` elements into their buffer."""
    if not f32:
        return bf16_device(x, stride, offset)
    buf = torch.full((offset + x.shape[0] * stride,), float("nan"), dtype=torch.float32, device="cuda")
    view = buf[offset:].view(x.shape[0], stride)
    view[:, :x.shape[1]] = device(x).float()
    return view


class Case:
    """Inputs of one call; every array on its own stride."""

    def __init__(self, zc, rows, cols, after=ref.RMS, before=ref.RMS, f32=False, params_f32=False, weights=True, bias=False,
                 gate=True, row_gate=False, z=True, scale=0.5, eps=1e-6, gap=0, offset=0, seed=0, mean=0.2):
        self.zc, self.rows, self.cols, self.f32, self.gap = zc, rows, cols, f32, gap
        g = np.random.default_rng([rows, cols, seed])
        rnd = ref.f32 if f32 else ref.bf16
        prm = ref.f32 if params_f32 else ref.bf16
        self.x = rnd(3 * g.standard_normal((rows, cols)) + mean)
        self.z = ref.bf16(1.5 * g.standard_normal((rows, cols)) - mean) if z else None
        self.dr = rnd(g.standard_normal((rows, cols)))
        self.dy = ref.bf16(g.standard_normal((rows, cols)))

        def param(on, mean):
            return prm(0.3 * g.standard_normal(cols) + mean) if on else None

        self.after = ref.Side(after, param(weights, 1.0), param(bias, 0.1), eps)
        self.before = ref.Side(before, param(weights, 1.0), param(bias, -0.1), eps)
        self.gate, self.scale = param(gate, 0.5), scale
        self.row_gate = ref.f32(g.standard_normal(rows)) if row_gate else None
        self.pt = torch.float32 if params_f32 else torch.bfloat16
        self.stride = cols + gap
        self.offset = offset

        def dev(p):
            if p is None:
                return None
            buf = torch.zeros(offset + cols, dtype=self.pt, device="cuda")
            buf[offset:] = device(p).to(self.pt)
            return buf[offset:]

        self.d = {k: dev(v) for k, v in (("w1", self.after.w), ("b1", self.after.b), ("w2", self.before.w),
                                         ("b2", self.before.b), ("gate", self.gate))}
        self.cfg = zc.norm_config(zc.norm_params(after, self.d["w1"], self.d["b1"], eps),
                                  zc.norm_params(before, self.d["w2"], self.d["b2"], eps), self.d["gate"],
                                  None if self.row_gate is None else device(self.row_gate).float(), scale)
        self.dx, self.dz = stream_device(self.x, f32, self.stride, offset), None
        if z:
            self.dz = bf16_device(self.z, self.stride, offset)
        self.kind = zc.ZC_F32 if f32 else zc.ZC_BF16
        self.st = torch.float32 if f32 else torch.bfloat16

    def forward(self, r=True, y=True, q=False):
        zc, m, n, s = self.zc, self.rows, self.cols, self.stride
        size = 4 if self.f32 else 2
        o = {"r": Out((m, s), self.st, size * self.offset), "y": Out((m, s), torch.bfloat16, 2 * self.offset),
             "q": Out((m, zc.zc_fp8_stride(n)), torch.uint8), "s": Out((m, zc.zc_fp8_scale_stride(n)), torch.uint8)}
        zc.zc_norm(self.dx, self.kind, m, n, s, self.dz, s, self.cfg, o["r"] if r else None, s, o["y"] if y else None, s,
                   o["q"] if q else None, o["s"] if q else None)
        return o

    def check_forward(self):
        o = self.forward(q=True)
        r, er, y, ey = ref.norm(self.x, self.z, self.after, self.before, self.gate, self.row_gate, self.scale)
        close(o["r"].numpy()[:, :self.cols], r, half_step(self.f32) * np.abs(r) + 2 * er, "r")
        got = o["y"].numpy()
        close(got[:, :self.cols], y, ref.BF16_HALF_STEP * np.abs(y) + 2 * ey, "y")
        # the 8-bit y is the blocks of the BF16 y
        zc, m, n = self.zc, self.rows, self.cols
        q, s = Out((m, zc.zc_fp8_stride(n)), torch.uint8), Out((m, zc.zc_fp8_scale_stride(n)), torch.uint8)
        zc.zc_fp8_quantize(o["y"], m, n, self.stride, zc.ZC_FP8_E4M3, 1, q, s)
        assert np.array_equal(o["q"].numpy(), q.numpy()) and np.array_equal(o["s"].numpy(), s.numpy())
        if self.gap:  # what lies between the rows is left as it was
            for v, t in ((o["y"], torch.bfloat16), (o["r"], self.st)):
                sent = torch.full((1, 1), 0, dtype=t).view(torch.uint8).fill_(0xA5).view(t)
                rest = v.t[:, self.cols:]
                assert bool((rest.contiguous().view(torch.uint8) == 0xA5).all()), sent

    def backward(self, dr=True, dy=True, dx=True, dz=True, grads=("w1", "b1", "gate", "w2", "b2", "row"), in_place=False):
        zc, m, n, s = self.zc, self.rows, self.cols, self.stride
        size = 4 if self.f32 else 2
        o = {"dx": Out((m, s), self.st, size * self.offset), "dz": Out((m, s), torch.bfloat16, 2 * self.offset)}
        for k in ("w1", "b1", "gate", "w2", "b2"):
            o["d" + k] = Out((n,), torch.float32)
        o["drow_gate"] = Out((m,), torch.float32)
        gr = zc.norm_grads(*[o["d" + k] if k in grads else None for k in ("w1", "b1", "gate", "w2", "b2")],
                           o["drow_gate"] if "row" in grads else None)
        ws = torch.full((max(16, zc.zc_norm_backward_workspace_bytes(m, n)),), 0xFF, dtype=torch.uint8, device="cuda")
        d = stream_device(self.dr, self.f32, s, self.offset) if dr else None
        if in_place:
            o["dx"].t.copy_(d)
            d = o["dx"]
        zc.zc_norm_backward(self.dx, self.kind, m, n, s, self.dz, s, self.cfg, d, s,
                            bf16_device(self.dy, s, self.offset) if dy else None, s, o["dx"] if dx else None, s,
                            o["dz"] if dz and self.dz is not None else None, s, gr, ws, ws.numel())
        return o

    def check_backward(self, dr=True, dy=True, **kw):
        o = self.backward(dr=dr, dy=dy, **kw)
        want = ref.norm_backward(self.x, self.z, self.after, self.before, self.gate, self.row_gate, self.scale,
                                 self.dr if dr else None, self.dy if dy else None)
        for name in ("dx", "dw1", "db1", "dgate", "dw2", "db2", "drow_gate"):
            v, e = want[name]
            got = o[name].numpy()
            close(got[:, :self.cols] if got.ndim == 2 else got, v,
                  (half_step(self.f32) if name == "dx" else ref.F32_HALF_STEP) * np.abs(v) + 2 * e, name)
        if self.z is not None:
            v, e = want["dz"]
            close(o["dz"].numpy()[:, :self.cols], v, ref.BF16_HALF_STEP * np.abs(v) + 2 * e, "dz")


# every team and number of chunks, ragged last chunks, single columns and rows, rows more than the blocks
SHAPES = [(1, 1, 0, 0), (3, 7, 2, 1), (2, 8, 0, 0), (9, 130, 0, 0), (5, 512, 8, 0), (6, 513, 0, 0), (4, 1000, 8, 8),
          (3, 1025, 1, 3), (2, 2048, 0, 0), (3, 2056, 0, 0), (2, 4100, 4, 0), (3, 5125, 0, 1), (2, 7168, 0, 0),
          (2, 8193, 0, 0), (2, 12288, 0, 0), (1, 16384, 0, 0), (2100, 64, 0, 0), (600, 2049, 0, 0)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,gap,offset", SHAPES)
def test_forward(zc, m, n, gap, offset, f32):
    Case(zc, m, n, gap=gap, offset=offset, f32=f32, params_f32=f32, row_gate=True).check_forward()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,gap,offset", SHAPES)
def test_backward(zc, m, n, gap, offset, f32):
    Case(zc, m, n, gap=gap, offset=offset, f32=f32, params_f32=f32, row_gate=True).check_backward()


KINDS = [dict(after=a, before=b, bias=bias) for a in range(3) for b in range(3) for bias in (False, True)]


@pytest.mark.parametrize("kw", KINDS + [dict(weights=False), dict(gate=False), dict(z=False), dict(z=False, before=ref.LAYER),
                                        dict(gate=False, row_gate=True, bias=True), dict(scale=0.0), dict(scale=-3.0),
                                        dict(params_f32=True, bias=True), dict(f32=True, bias=True, after=ref.LAYER)])
def test_kinds(zc, kw):
    for m, n in ((5, 200), (3, 2500)):
        c = Case(zc, m, n, **kw)
        c.check_forward()
        c.check_backward()
        c.check_backward(dr=False)
        c.check_backward(dy=False)
        c.check_backward(in_place=True)


def test_results_left_out(zc):
    c = Case(zc, 7, 300, bias=True, row_gate=True)
    full = {k: v.numpy().copy() for k, v in c.forward(q=True).items()}
    for kw, names in ((dict(y=False), ("r",)), (dict(r=False), ("y",)), (dict(r=False, y=False, q=True), ("q", "s")),
                      (dict(r=False, y=False), ())):
        part = c.forward(**kw)
        for k, v in part.items():
            if k in names:
                assert np.array_equal(v.numpy(), full[k]), k
            else:
                assert bool((v.raw == 0xA5).all()), k
    full = {k: v.numpy().copy() for k, v in c.backward().items()}
    for kw, names in ((dict(dx=False, dz=False), ("dw1", "db1", "dgate", "dw2", "db2", "drow_gate")),
                      (dict(grads=()), ("dx", "dz")), (dict(dz=False, grads=("w2",)), ("dx", "dw2")),
                      (dict(dx=False, grads=("b1", "row")), ("dz", "db1", "drow_gate")),
                      (dict(dx=False, dz=False, grads=()), ())):
        part = c.backward(**kw)
        for k, v in part.items():
            if k in names:
                assert np.array_equal(v.numpy(), full[k]), k
            else:
                assert bool((v.raw == 0xA5).all()), k


def test_sum_in_place(zc):
    """r over x."""
    c = Case(zc, 40, 1300)
    want = c.forward()["r"].numpy()
    o = Out((40, 1300), torch.bfloat16)
    o.t.copy_(c.dx)
    zc.zc_norm(o, c.kind, 40, 1300, 1300, c.dz, 1300, c.cfg, o, 1300)
    assert np.array_equal(o.numpy(), want)


def test_no_rows(zc):
    """Without rows the gradients of the parameters are zeros, and nothing else is written."""
    c = Case(zc, 1, 100, bias=True)
    out = {k: Out((100,), torch.float32) for k in ("w1", "b1", "gate", "w2", "b2")}
    zc.zc_norm_backward(None, c.kind, 0, 100, 100, None, 100, c.cfg, None, 100, None, 100, None, 100, None, 100,
                        zc.norm_grads(*out.values()), None, 0)
    for v in out.values():
        assert not v.numpy().any()


def differences(f, v, e=1e-5):
    return (f(v + e) - f(v - e)) / (2 * e)


@pytest.mark.parametrize("kind", [ref.RMS, ref.LAYER])
def test_backward_against_differences(zc, kind):
    """Central differences of the 64-bit forward pass along random directions: the error of a difference is e^2 times a
    third derivative and 64-bit roundings over e, below 1e-7 of the sum of the terms' sizes."""
    c = Case(zc, 3, 40, after=kind, before=kind, bias=True, row_gate=True)
    o = c.backward()
    g = np.random.default_rng(5)

    def total(x, z, p):
        after, before = ref.Side(kind, p["w1"], p["b1"]), ref.Side(kind, p["w2"], p["b2"])
        r, _, y, _ = ref.norm(x, z, after, before, p["gate"], p["rg"], c.scale)
        return (r * c.dr).sum() + (y * c.dy).sum()

    # the gradient is evaluated at the stored sum: x such that the sum is the stored one
    h = c.after.apply(c.z)[1]
    x = c.x - c.scale * c.gate * c.row_gate[:, None] * h
    p = dict(w1=c.after.w, b1=c.after.b, w2=c.before.w, b2=c.before.b, gate=c.gate, rg=c.row_gate)
    want = ref.norm_backward(c.x, c.z, c.after, c.before, c.gate, c.row_gate, c.scale, c.dr, c.dy)
    names = dict(w1="dw1", b1="db1", w2="dw2", b2="db2", gate="dgate", rg="drow_gate")
    for key in ("x", "z", *names):
        base = x if key == "x" else c.z if key == "z" else p[key]
        u = g.standard_normal(base.shape)

        def f(s):
            if key == "x":
                return total(x + s * u, c.z, p)
            if key == "z":
                return total(x, c.z + s * u, p)
            return total(x, c.z, {**p, key: p[key] + s * u})

        name = {"x": "dx", "z": "dz"}.get(key) or names[key]
        v, e = want[name]
        got = o[name].numpy()
        slope = differences(f, 0.0)
        assert abs((v * u).sum() - slope) <= 1e-6 * (1 + np.abs(v * u).sum()), key
        tol = (np.abs(u) * (ref.BF16_HALF_STEP * np.abs(v) + 2 * e)).sum() + 1e-6 * (1 + np.abs(v * u).sum())
        assert abs((got * u).sum() - slope) <= tol, key


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", [ref.RMS, ref.LAYER])
@pytest.mark.parametrize("power", [100, 70, 30, -30, -60, -100])
def test_rows_of_any_size(zc, kind, power, f32):
    """Squares far outside the range of a float: the statistics are those of the row, whatever its size."""
    for eps in (1e-6, 1e-30):
        c = Case(zc, 4, 700, after=kind, before=kind, eps=eps, f32=f32)
        for name in ("x", "z"):
            setattr(c, name, getattr(c, name) * 2.0 ** power)
        c.dx, c.dz = stream_device(c.x, f32, 700), bf16_device(c.z, 700)
        c.check_forward()
        c.check_backward()


def test_layer_norm_of_rows_far_from_zero(zc):
    """A mean a thousand times the deviation."""
    g = np.random.default_rng(3)
    c = Case(zc, 6, 900, after=ref.LAYER, before=ref.LAYER, f32=True)
    c.z = ref.bf16(g.integers(0, 2, (6, 900)) * 2.0 + 510.0)  # 510 or 512, both BF16 values
    c.x = ref.f32(1000 + g.standard_normal((6, 900)))
    c.dx, c.dz = stream_device(c.x, True, 900), bf16_device(c.z, 900)
    c.check_forward()
    c.check_backward()


def test_special_rows(zc):
    """Rows of zeros, and rows that hold NaN or an infinity: what the formula gives, and nothing to the rows beside them."""
    n = 600
    c = Case(zc, 6, n, after=ref.NONE, gate=False, scale=1.0, z=False)
    clean = c.forward()["y"].numpy().copy()
    x = c.x.copy()
    x[0] = 0.0
    x[2, 5] = np.nan
    x[4, 7] = np.inf
    c.dx = bf16_device(x, n)
    y = c.forward()["y"].numpy()
    assert not y[0].any()
    assert np.isnan(y[2]).all()
    assert np.isnan(y[4, 7]) and not np.delete(y[4], 7).any()  # finite / infinite
    for i in (1, 3, 5):
        assert np.array_equal(y[i], clean[i])
    o = c.backward(grads=())
    dx = o["dx"].numpy()
    assert np.isnan(dx[2]).all() and np.isfinite(dx[[0, 1, 3, 5]]).all()


def test_repeats_itself(zc):
    c = Case(zc, 700, 3000, bias=True, row_gate=True)
    first = {k: v.numpy().copy() for k, v in c.backward().items()}
    for _ in range(3):
        for k, v in c.backward().items():
            assert np.array_equal(v.numpy(), first[k]), k
