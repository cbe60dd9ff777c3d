"""Every array on a stride and an alignment of its own: sentinels between the rows of results, NaN between those of inputs."""
import numpy as np
import pytest
import torch

import block_ref as ref
from moe_gpu import Out, bf16_device, close, device, moe
from test_gpu_balance import Case as Balance
from test_gpu_norm import Case as Norm, half_step, stream_device
from test_gpu_product import EPS, exact, sum_error, whole_numbers, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


class Rows(Out):
    """A result of m rows of n values, `gap` apart, `offset` values into its buffer."""

    def __init__(self, m, n, f32, gap, offset):
        self.cols, self.gap = n, gap
        super().__init__((m, n + gap), torch.float32 if f32 else torch.bfloat16, offset * (4 if f32 else 2))

    def values(self):
        v = self.numpy()
        if self.gap:
            assert bool((self.t[:, self.cols:].contiguous().view(torch.uint8) == 0xA5).all()), "written between the rows"
        return v[:, :self.cols]


# gaps and offsets of up to eight arrays: rows anywhere, rows on 16 bytes (as BF16 and floats), and one array off them
PLACES = {"anywhere": [(1, 1), (2, 3), (3, 0), (5, 2), (7, 5), (11, 7), (13, 4), (17, 6)],
          "wide": [(0, 0), (8, 8), (16, 8), (24, 16), (32, 0), (40, 8), (48, 24), (56, 8)]}
PLACES["all but one"] = [(3, 1)] + PLACES["wide"][1:]
PLACES["all but another"] = PLACES["wide"][:3] + [(5, 3)] + PLACES["wide"][4:]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("places", PLACES)
@pytest.mark.parametrize("n", [200, 205, 2504, 5125])
def test_norm(zc, n, places, f32):
    m, p = 5, PLACES[places]
    c = Norm(zc, m, n, after=ref.LAYER, bias=True, row_gate=True, f32=f32)

    def st(i):
        return n + p[i][0]

    x, z = stream_device(c.x, f32, st(0), p[0][1]), bf16_device(c.z, st(1), p[1][1])
    r, y = Rows(m, n, f32, *p[2]), Rows(m, n, False, *p[3])
    zc.zc_norm(x, c.kind, m, n, st(0), z, st(1), c.cfg, r, st(2), y, st(3))
    want, er, wy, ey = ref.norm(c.x, c.z, c.after, c.before, c.gate, c.row_gate, c.scale)
    close(r.values(), want, half_step(f32) * np.abs(want) + 2 * er, "r")
    close(y.values(), wy, ref.BF16_HALF_STEP * np.abs(wy) + 2 * ey, "y")
    dr, dy = stream_device(c.dr, f32, st(4), p[4][1]), bf16_device(c.dy, st(5), p[5][1])
    dx, dz = Rows(m, n, f32, *p[6]), Rows(m, n, False, *p[7])
    sums = [Out((n,), torch.float32) for _ in range(5)]
    row = Out((m,), torch.float32)
    ws = workspace(zc, zc.zc_norm_backward_workspace_bytes(m, n))
    zc.zc_norm_backward(x, c.kind, m, n, st(0), z, st(1), c.cfg, dr, st(4), dy, st(5), dx, st(6), dz, st(7),
                        zc.norm_grads(*sums, row), ws, ws.numel())
    want = ref.norm_backward(c.x, c.z, c.after, c.before, c.gate, c.row_gate, c.scale, c.dr, c.dy)
    for name, got in (("dx", dx.values()), ("dz", dz.values()), ("drow_gate", row.numpy()),
                      *zip(("dw1", "db1", "dgate", "dw2", "db2"), (s.numpy() for s in sums))):
        v, e = want[name]
        half = ref.BF16_HALF_STEP if name == "dz" or (name == "dx" and not f32) else ref.F32_HALF_STEP
        close(got, v, half * np.abs(v) + 2 * e, name)


# few rows, tiles, ragged tiles, whole tiles, split contractions (the last three), of whole numbers: results are exact
PRODUCTS = [(2, 40, 70), (20, 33, 256), (200, 264, 130), (256, 256, 128), (130, 128, 8192), (128, 256, 8192), (300, 264, 8200)]


@pytest.mark.parametrize("types", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("places", PLACES)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(zc, m, n, k, places, types):
    out_f32, res_f32 = types
    p = PLACES[places]
    g = np.random.default_rng([m, n, k])
    a, w, res, bias = whole_numbers(g, m, k), whole_numbers(g, n, k), whole_numbers(g, m, n), whole_numbers(g, n)
    da, dw = bf16_device(a, k + p[0][0], p[0][1]), bf16_device(w, k + p[1][0], p[1][1])
    dres = stream_device(res, res_f32, n + p[2][0], p[2][1])
    ws = workspace(zc, zc.zc_matmul_workspace_bytes(m, n, k))
    v = exact(0, a, w) + bias
    for act in (zc.ZC_ACT_NONE, zc.ZC_ACT_RELU):
        for keep in (True, False):
            pre, out = Rows(m, n, False, *p[3]), Rows(m, n, out_f32, *p[4])
            e = zc.epilogue(device(bias).float(), act, dres, n + p[2][0], pre if keep else None, n + p[3][0], -2.0)
            zc.zc_matmul(da, m, k + p[0][0], dw, n, k, k + p[1][0], e, out, zc.ZC_F32 if out_f32 else zc.ZC_BF16, n + p[4][0], ws,
                         0 if ws is None else ws.numel())
            want = res - 2 * (np.maximum(v, 0) if act else v)
            assert np.array_equal(out.values(), want if out_f32 else ref.bf16(want)), (act, keep)
            if keep:
                assert np.array_equal(pre.values(), ref.bf16(v)), act


@pytest.mark.parametrize("types", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("places", PLACES)
@pytest.mark.parametrize("m,n,k", [(20, 33, 250), (200, 264, 130), (256, 256, 128), (128, 136, 8192)])
def test_gradients_of_operands(zc, m, n, k, places, types):
    out_f32, add_f32 = types
    p = PLACES[places]
    for which, call in ((1, zc.zc_matmul_dgrad), (2, zc.zc_matmul_wgrad)):
        g = np.random.default_rng([m, n, k, which])
        a, b, add = whole_numbers(g, *((k, m) if which == 2 else (m, k))), whole_numbers(g, k, n), whole_numbers(g, m, n)
        da, db = bf16_device(a, a.shape[1] + p[0][0], p[0][1]), bf16_device(b, n + p[1][0], p[1][1])
        dadd = stream_device(add, add_f32, n + p[2][0], p[2][1])
        out = Rows(m, n, out_f32, *p[3])
        ws = workspace(zc, zc.zc_matmul_workspace_bytes(m, n, k))
        call(da, a.shape[0], a.shape[1], a.shape[1] + p[0][0], db, n, n + p[1][0], dadd, zc.ZC_F32 if add_f32 else zc.ZC_BF16, n + p[2][0],
             out, zc.ZC_F32 if out_f32 else zc.ZC_BF16, n + p[3][0], ws, 0 if ws is None else ws.numel())
        want = exact(which, a, b) + add
        assert np.array_equal(out.values(), want if out_f32 else ref.bf16(want)), which


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("places", PLACES)
@pytest.mark.parametrize("m,n", [(3, 9), (40, 513), (300, 520)])
def test_gradient_of_the_pre_activation(zc, m, n, places, f32):
    p = PLACES[places]
    g = np.random.default_rng([m, n])
    d, v = (ref.f32 if f32 else ref.bf16)(g.standard_normal((m, n))), ref.bf16(2 * g.standard_normal((m, n)))
    dd, pre = stream_device(d, f32, n + p[0][0], p[0][1]), bf16_device(v, n + p[1][0], p[1][1])
    dpre, dbias = Rows(m, n, False, *p[2]), Out((n,), torch.float32)
    ws = workspace(zc, zc.zc_activation_backward_workspace_bytes(m, n))
    zc.zc_activation_backward(dd, zc.ZC_F32 if f32 else zc.ZC_BF16, m, n, n + p[0][0], pre, n + p[1][0], zc.ZC_ACT_SILU, 0.75, dpre,
                              n + p[2][0], dbias, ws, ws.numel())
    want = 0.75 * d * ref.activation(v, 2)[1]
    one = 0.75 * np.abs(d) * ref.activation_error(v, 2)[1] + 3 * EPS * np.abs(want)
    close(dpre.values(), want, ref.BF16_HALF_STEP * np.abs(want) + one, "dpre")
    close(dbias.numpy(), want.sum(0), one.sum(0) + EPS * (m + 64) * np.abs(want).sum(0), "dbias")


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("places", PLACES)
def test_balance(zc, places, sigmoid, bf16):
    p, t, e = PLACES[places], 150, 40
    c = Balance(zc, t, e, 4, sigmoid, offsets=[0, 60, 140], mask=True, bf16=bf16)
    counts, used, _, _ = c.want()
    x, add = stream_device(c.x, not bf16, e + p[0][0], p[0][1]), stream_device(c.add, not bf16, e + p[1][0], p[1][1])
    out = Rows(t, e, not bf16, *p[2])
    dc, du = device(counts.astype(np.int32)), device(used.astype(np.int32))
    zc.zc_balance_backward(x, c.kind, t, e + p[0][0], c.cfg, c.d["mask"], c.s, c.d["off"], dc, du, c.d["dloss"], c.d["dz"], add,
                           e + p[1][0], out, e + p[2][0])
    want, size = ref.balance_backward(c.x, c.mask, c.offsets, e, 4, sigmoid, counts, used, c.dloss, c.dz, c.add)
    half = ref.BF16_HALF_STEP if bf16 else ref.F32_HALF_STEP
    close(out.values(), want, half * np.abs(want) + EPS * (400 + 4 * c.argument()) * size + 2.0 ** -125, "dlogits")
