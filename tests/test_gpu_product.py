"""BF16 products with their epilogue, and the gradients of their operands, against 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from moe_gpu import Out, bf16_device, close, device, moe

pytestmark = pytest.mark.gpu
EPS = ref.EPS32


@pytest.fixture(scope="module")
def zc():
    return moe()


def whole_numbers(g, *shape):
    """Small whole numbers: products and sums of up to 2^16 of them are exact in 32 bits in any order."""
    return g.integers(-8, 9, shape).astype(np.float64)


def stride(width, gap):
    """Rows `gap` apart, or, for a gap below 0, on the next multiple of 8 and 8 more (ragged rows on the wide path)."""
    return width + gap if gap >= 0 else (width + 7) // 8 * 8 + 8


def placed(x, gap, offset):
    """Rows a stride apart, the gaps NaN, `offset` values into their buffer."""
    return bf16_device(x, stride(x.shape[1], gap), offset)


def workspace(zc, n):
    return None if not n else torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def product(zc, which, a, b, m, n, k, out_f32=True, add=None, add_f32=False, gap=0, offset=0, room=True, epilogue=None):
    """which 0: a (m x k) b (n x k); 1: a (m x k) b (k x n); 2: a (k x m) b (k x n); the results as an Out."""
    da, db = placed(a, gap, offset), placed(b, gap, offset)
    size = 4 if out_f32 else 2
    sm, sn, sk = (stride(v, gap) for v in (m, n, k))
    out = Out((m, sn), torch.float32 if out_f32 else torch.bfloat16, size * offset)
    kind = zc.ZC_F32 if out_f32 else zc.ZC_BF16
    ws = workspace(zc, zc.zc_matmul_workspace_bytes(m, n, k)) if room else None
    nb = 0 if ws is None else ws.numel()
    at = zc.ZC_F32 if add_f32 else zc.ZC_BF16
    dadd = None if add is None else (device(add).float() if add_f32 else device(add).bfloat16())
    if which == 0:
        zc.zc_matmul(da, m, sk, db, n, k, sk, epilogue, out, kind, sn, ws, nb)
    elif which == 1:
        zc.zc_matmul_dgrad(da, m, k, sk, db, n, sn, dadd, at, n, out, kind, sn, ws, nb)
    else:
        zc.zc_matmul_wgrad(da, k, m, sm, db, n, sn, dadd, at, n, out, kind, sn, ws, nb)
    return out


def operands(which, m, n, k, draw):
    a = draw(k, m) if which == 2 else draw(m, k)
    b = draw(n, k) if which == 0 else draw(k, n)
    return a, b


def exact(which, a, b):
    ta, tb = device(a).double(), device(b).double()
    ta = ta.t().contiguous() if which == 2 else ta
    tb = tb.t().contiguous() if which == 0 else tb
    return torch.mm(ta, tb).cpu().numpy()


# single rows and columns, contractions of nothing, of less than a block, ragged and whole; every shape of tile, with
# and without a split; (gap, offset) off the wide path
SIZES = [(1, 1, 1), (1, 16, 0), (3, 5, 7), (1, 300, 64), (16, 257, 129), (17, 31, 500), (32, 1000, 1024), (33, 64, 63), (33, 130, 65),
         (64, 512, 2048), (100, 200, 8), (129, 127, 192), (130, 260, 2056), (255, 257, 1000), (256, 256, 64), (300, 300, 72),
         (512, 520, 4096), (1000, 1032, 136), (1024, 1024, 256), (2048, 2000, 192), (4096, 4096, 200), (5000, 2100, 64),
         (129, 8200, 640), (8200, 129, 640), (600, 6400, 1200)]


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_whole_numbers_are_exact(zc, m, n, k, which):
    """Sums of whole numbers have no rounding, whatever the order: any difference is a wrong element."""
    g = np.random.default_rng([m, n, k, which])
    a, b = operands(which, m, n, k, lambda *s: whole_numbers(g, *s))
    want = exact(which, a, b)
    for gap, offset in ((0, 0), (-1, 8), (3, 1)):
        for room in (True, False):
            got = product(zc, which, a, b, m, n, k, gap=gap, offset=offset, room=room)
            assert np.array_equal(got.numpy()[:, :n], want), (gap, offset, room)
            if gap:
                assert bool((got.t[:, n:].contiguous().view(torch.uint8) == 0xA5).all())
    got = product(zc, which, a, b, m, n, k, out_f32=False)
    assert np.array_equal(got.numpy(), ref.bf16(want))


# every shape of tile with all of its tiles whole, with all split and with those past the last whole turn of the CUs
# split, on the wide path and off it
LARGER = [(1000, 2056, 264), (1000, 4100, 520), (1000, 4100, 1032), (1000, 4100, 2056), (1000, 8200, 520), (1000, 8200, 2056),
          (100, 8200, 1032), (130, 6000, 640), (130, 6000, 1032), (260, 4100, 2056), (2000, 4100, 640), (2000, 8200, 1032),
          (1032, 2900, 136), (2056, 260, 7168), (777, 1104, 7168), (3, 200, 4200), (20, 200, 4200), (16, 4100, 2200), (2, 162, 10889)]


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("m,n,k", LARGER)
def test_larger_whole_numbers_are_exact(zc, m, n, k, which):
    g = np.random.default_rng([m, n, k, which])
    a, b = operands(which, m, n, k, lambda *s: whole_numbers(g, *s))
    add = whole_numbers(g, m, n)
    want = exact(which, a, b)
    for gap, offset in ((-1, 8), (3, 1)):
        for room in (True, False):
            got = product(zc, which, a, b, m, n, k, gap=gap, offset=offset, room=room)
            assert np.array_equal(got.numpy()[:, :n], want), (gap, offset, room)
            assert bool((got.t[:, n:].contiguous().view(torch.uint8) == 0xA5).all())
    if which:
        got = product(zc, which, a, b, m, n, k, out_f32=False, add=add, gap=-1, offset=8)
        assert np.array_equal(got.numpy()[:, :n], ref.bf16(want + add))


def sum_error(k, size):
    """Every addition of a 32-bit sum may be off by half a step of what is summed so far (a whole one where an instruction
    cuts): at most all k of them in a row."""
    return 2 * EPS * (k + 16) * size


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("m,n,k", [(5, 40, 333), (64, 96, 4096), (300, 520, 1000), (1030, 1100, 260), (2050, 2060, 136)])
def test_against_64_bits(zc, m, n, k, which):
    g = np.random.default_rng([m, n, k])
    a, b = operands(which, m, n, k, lambda *s: ref.bf16(g.standard_normal(s)))
    want, size = exact(which, a, b), exact(which, np.abs(a), np.abs(b))
    add = ref.bf16(10 * g.standard_normal((m, n)))
    for f32 in (True, False):
        got = product(zc, which, a, b, m, n, k, out_f32=f32).numpy()
        half = EPS if f32 else ref.BF16_HALF_STEP
        close(got, want, half * np.abs(want) + sum_error(k, size), "product")
        if which:
            for add_f32 in (False, True):
                got = product(zc, which, a, b, m, n, k, out_f32=f32, add=add, add_f32=add_f32).numpy()
                close(got, want + add, half * np.abs(want + add) + EPS * np.abs(add) + sum_error(k, size), "with add")


@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("m,n,k", [(40, 60, 50), (128, 128, 8192)])
def test_sum_onto_itself(zc, m, n, k, which):
    """add and the result in one array, over two calls; the second size splits its contraction."""
    g = np.random.default_rng([m, k])
    a, b = operands(which, m, n, k, lambda *s: whole_numbers(g, *s))
    want = exact(which, a, b)
    da, db = device(a).bfloat16(), device(b).bfloat16()
    out = Out((m, n), torch.float32)
    out.t.fill_(5.0)
    ws = workspace(zc, zc.zc_matmul_workspace_bytes(m, n, k))
    for _ in range(2):
        if which == 1:
            zc.zc_matmul_dgrad(da, m, k, k, db, n, n, out, zc.ZC_F32, n, out, zc.ZC_F32, n, ws, 0 if ws is None else ws.numel())
        else:
            zc.zc_matmul_wgrad(da, k, m, m, db, n, n, out, zc.ZC_F32, n, out, zc.ZC_F32, n, ws, 0 if ws is None else ws.numel())
    assert np.array_equal(out.numpy(), 2 * want + 5)


def run_epilogue(zc, m, n, k, act, bias_f32=True, res_f32=False, out_f32=False, scale=1.0, res=True, bias=True, in_place=False, seed=0):
    g = np.random.default_rng([m, n, k, seed])
    a, w = ref.bf16(g.standard_normal((m, k))), ref.bf16(g.standard_normal((n, k)) * 2 / max(k, 1) ** 0.5)
    bv = (ref.f32 if bias_f32 else ref.bf16)(g.standard_normal(n)) if bias else None
    if in_place:
        res_f32 = out_f32
    rv = (ref.f32 if res_f32 else ref.bf16)(g.standard_normal((m, n))) if res else None
    ft = {True: torch.float32, False: torch.bfloat16}
    pre, out = Out((m, n), torch.bfloat16), Out((m, n), ft[out_f32])
    dres = device(rv).to(ft[res_f32]) if res else None
    if in_place:
        out.t.copy_(dres)
        dres = out.t
    e = zc.epilogue(device(bv).to(ft[bias_f32]) if bias else None, act, dres, n, pre, n, scale)
    ws = workspace(zc, zc.zc_matmul_workspace_bytes(m, n, k))
    zc.zc_matmul(device(a).bfloat16(), m, k, device(w).bfloat16(), n, k, k, e, out, zc.ZC_F32 if out_f32 else zc.ZC_BF16, n, ws,
                 0 if ws is None else ws.numel())
    v = exact(0, a, w) + (0 if bv is None else bv)
    ev = sum_error(k, exact(0, np.abs(a), np.abs(w))) + EPS * np.abs(v)
    close(pre.numpy(), v, ref.BF16_HALF_STEP * np.abs(v) + ev, "pre")
    y, slope = ref.activation(v, act)
    # no slope is above 1.2
    ey = ref.activation_error(v, act)[0] + 1.2 * ev
    want = scale * y + (0 if rv is None else rv)
    tol = (EPS if out_f32 else ref.BF16_HALF_STEP) * np.abs(want) + EPS * (2 * np.abs(scale * y) + np.abs(want)) + abs(scale) * ey
    close(out.numpy(), want, tol, "out")
    return pre, out


@pytest.mark.parametrize("act", range(6))
@pytest.mark.parametrize("m,n,k", [(3, 50, 70), (20, 33, 256), (200, 264, 130), (128, 256, 8192)])
def test_epilogue(zc, m, n, k, act):
    """Few rows, tiles, ragged tiles and a split contraction."""
    run_epilogue(zc, m, n, k, act)
    run_epilogue(zc, m, n, k, act, bias_f32=False, res_f32=True, out_f32=True, scale=-1.5)


@pytest.mark.parametrize("kw", [dict(res=False), dict(bias=False), dict(res=False, bias=False, scale=0.5), dict(in_place=True),
                                dict(in_place=True, out_f32=True), dict(res_f32=True)])
def test_epilogue_parts(zc, kw):
    for m, n, k in ((2, 40, 64), (150, 136, 72), (128, 128, 8192), (40, 60, 0)):
        run_epilogue(zc, m, n, k, 2, **kw)


def activation_inputs():
    """BF16 values over the whole range of an activation, both signs, and around its bends."""
    v = np.concatenate([np.linspace(-12, 12, 4001), np.linspace(-120, 120, 400), np.geomspace(1e-30, 3e38, 300), [0.0]])
    return np.unique(ref.bf16(np.concatenate([v, -v])))


@pytest.mark.parametrize("act", range(1, 6))
def test_activation_values(zc, act):
    """The activation itself: the contraction is one value times 1, the result has 32 bits."""
    v = activation_inputs()
    n = v.size
    out = Out((1, n), torch.float32)
    e = zc.epilogue(activation=act)
    zc.zc_matmul(torch.ones(1, 1, dtype=torch.bfloat16, device="cuda"), 1, 1, device(v).bfloat16(), n, 1, 1, e, out, zc.ZC_F32, n)
    with np.errstate(over="ignore", invalid="ignore"):
        want = ref.activation(v, act)[0]
        if act == 4:
            want = np.where(np.abs(v) > 1e10, np.maximum(v, 0), want)
    close(out.numpy()[0], want, EPS * np.abs(want) + ref.activation_error(v, act)[0], "activation %d" % act)


@pytest.mark.parametrize("act", range(1, 6))
def test_activation_slopes(zc, act):
    """dpre in BF16, and through a bias sum of a single row in 32 bits."""
    v = activation_inputs()
    n = v.size
    dpre, dbias = Out((1, n), torch.bfloat16), Out((n,), torch.float32)
    ws = workspace(zc, zc.zc_activation_backward_workspace_bytes(1, n))
    zc.zc_activation_backward(torch.ones(1, n, dtype=torch.float32, device="cuda"), zc.ZC_F32, 1, n, n, device(v).bfloat16(), n,
                              act, 1.0, dpre, n, dbias, ws, ws.numel())
    with np.errstate(over="ignore", invalid="ignore"):
        want, tol = ref.activation(v, act)[1], ref.activation_error(v, act)[1]
        if act in (2, 3, 4):
            far = np.abs(v) > 1000
            want, tol = np.where(far, (v > 0) * 1.0, want), np.where(far, EPS, tol)
    close(dbias.numpy(), want, EPS * np.abs(want) + tol, "slope %d" % act)
    close(dpre.numpy()[0], want, ref.BF16_HALF_STEP * np.abs(want) + tol, "slope %d" % act)


@pytest.mark.parametrize("act", range(2, 6))
def test_slopes_against_differences(zc, act):
    """Central differences of the 64-bit activation: e^2 times a third derivative, and 64-bit roundings over e."""
    v = ref.bf16(np.linspace(-8, 8, 999))
    dbias = Out((999,), torch.float32)
    ws = workspace(zc, zc.zc_activation_backward_workspace_bytes(1, 999))
    zc.zc_activation_backward(torch.ones(1, 999, device="cuda"), zc.ZC_F32, 1, 999, 999, device(v).bfloat16(), 999, act, 1.0, None,
                              0, dbias, ws, ws.numel())
    slope = (ref.activation(v + 1e-5, act)[0] - ref.activation(v - 1e-5, act)[0]) / 2e-5
    close(dbias.numpy(), slope, 1e-9 + 1e-9 * np.abs(v) + EPS * np.abs(slope) + ref.activation_error(v, act)[1], "slope")


def test_far_tails_keep_their_digits(zc):
    """Where the exponential is below the normal numbers, its product with a large gradient is not."""
    v = ref.bf16(np.linspace(-104.0, -88.0, 65))
    d = np.full(65, 2.0 ** 80)
    for act in (2, 5):
        dbias = Out((65,), torch.float32)
        ws = workspace(zc, zc.zc_activation_backward_workspace_bytes(1, 65))
        zc.zc_activation_backward(device(d[None]).float(), zc.ZC_F32, 1, 65, 65, device(v).bfloat16(), 65, act, 1.0, None, 0, dbias, ws,
                                  ws.numel())
        want = d * ref.activation(v, act)[1]
        close(dbias.numpy(), want, 2.0 ** 80 * (ref.activation_error(v, act)[1] - 2.0 ** -125) + EPS * np.abs(want), "act %d" % act)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("act", [0, 2])
@pytest.mark.parametrize("m,n,gap,offset", [(1, 1, 0, 0), (7, 9, 0, 0), (300, 513, 3, 1), (1000, 136, 8, 8), (70, 2000, 0, 0)])
def test_activation_backward(zc, m, n, gap, offset, act, f32):
    g = np.random.default_rng([m, n])
    d = (ref.f32 if f32 else ref.bf16)(g.standard_normal((m, n)))
    v = ref.bf16(2 * g.standard_normal((m, n)))
    s = n + gap
    buf = torch.zeros(offset + m * s, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    dd = buf[offset:].view(m, s)
    dd[:, :n] = device(d).to(dd.dtype)
    dpre, dbias = Out((m, s), torch.bfloat16, 2 * offset), Out((n,), torch.float32)
    ws = workspace(zc, zc.zc_activation_backward_workspace_bytes(m, n))
    pre = placed(v, gap, offset)

    def call(dout, out, bias, kind=zc.ZC_F32 if f32 else zc.ZC_BF16):
        zc.zc_activation_backward(dout, kind, m, n, s, pre if act else None, s, act, 0.75, out, s, bias, ws, ws.numel())

    call(dd, dpre, dbias)
    slope, es = ref.activation(v, act)[1], ref.activation_error(v, act)[1]
    want = 0.75 * d * slope
    one = 0.75 * np.abs(d) * es + 3 * EPS * np.abs(want)
    close(dpre.numpy()[:, :n], want, ref.BF16_HALF_STEP * np.abs(want) + one, "dpre")
    close(dbias.numpy(), want.sum(0), one.sum(0) + EPS * (m + 64) * np.abs(want).sum(0), "dbias")
    if gap:
        assert bool((dpre.t[:, n:].contiguous().view(torch.uint8) == 0xA5).all())
    first = dpre.numpy().copy(), dbias.numpy().copy()
    other = Out((m, s), torch.bfloat16, 2 * offset)
    call(dd, other, None)
    assert np.array_equal(other.numpy()[:, :n], first[0][:, :n])
    again = Out((n,), torch.float32)
    call(dd, None, again)
    assert np.array_equal(again.numpy(), first[1])
    if not f32:  # over the gradient itself
        other.t.copy_(dd)
        call(other, other, None)
        assert np.array_equal(other.numpy()[:, :n], first[0][:, :n])


def test_no_rows(zc):
    dbias = Out((50,), torch.float32)
    zc.zc_activation_backward(None, zc.ZC_BF16, 0, 50, 50, None, 50, 2, 1.0, None, 0, dbias, None, 0)
    assert not dbias.numpy().any()


@pytest.mark.parametrize("which", [0, 1, 2])
def test_special_values(zc, which):
    """An infinity or NaN in one row (column) reaches that row (column) of the results and no other, also where tiles
    and blocks of the contraction are ragged."""
    for m, n, k in ((10, 20, 100), (140, 150, 90), (300, 270, 2100)):
        g = np.random.default_rng(m)
        a, b = operands(which, m, n, k, lambda *s: whole_numbers(g, *s) + 0.5)
        want = exact(which, a, b)
        a2 = a.copy()
        a2[(k - 1, m - 1) if which == 2 else (m - 1, k - 1)] = np.nan
        got = product(zc, which, a2, b, m, n, k).numpy()
        assert np.isnan(got[m - 1]).all() and np.isfinite(got[:m - 1]).all()
        close(got[:m - 1], want[:m - 1], sum_error(k, exact(which, np.abs(a), np.abs(b)))[:m - 1], "beside NaN")
        b2 = b.copy()
        b2[(n - 1, 0) if which == 0 else (0, n - 1)] = np.inf
        got = product(zc, which, a, b2, m, n, k).numpy()
        assert not np.isfinite(got[:, n - 1]).any() and np.isfinite(got[:, :n - 1]).all()


def test_rows_far_apart(zc):
    """Offsets past 32 bits: two rows 2^31 + 8 values apart, as either operand and as the result."""
    far, k = (1 << 31) + 8, 96
    g = np.random.default_rng(1)
    a, b = whole_numbers(g, 2, k), whole_numbers(g, 40, k)
    buf = torch.zeros(far + k, dtype=torch.bfloat16, device="cuda")
    buf[:k], buf[far:] = device(a[0]).bfloat16(), device(a[1]).bfloat16()
    db = device(b).bfloat16()
    want = a @ b.T
    out = Out((2, 40), torch.float32)
    zc.zc_matmul(buf, 2, far, db, 40, k, k, None, out, zc.ZC_F32, 40)
    assert np.array_equal(out.numpy(), want)
    out = Out((40, 2), torch.float32)
    zc.zc_matmul(db, 40, k, buf, 2, k, far, None, out, zc.ZC_F32, 2)
    assert np.array_equal(out.numpy(), want.T)
    # across the contraction: 2 values of it
    out = Out((k, 40), torch.float32)
    c = whole_numbers(g, 2, 40)
    zc.zc_matmul_wgrad(buf, 2, k, far, device(c).bfloat16(), 40, 40, None, zc.ZC_F32, 40, out, zc.ZC_F32, 40)
    assert np.array_equal(out.numpy(), a.T @ c)
    rows = torch.zeros(far + 40, dtype=torch.bfloat16, device="cuda")
    small = whole_numbers(g, 2, 4)
    zc.zc_matmul(device(small).bfloat16(), 2, 4, device(b[:, :4]).bfloat16(), 40, 4, 4, None, rows, zc.ZC_BF16, far)
    want = small @ b[:, :4].T
    assert np.array_equal(rows[:40].double().cpu().numpy(), want[0]) and np.array_equal(rows[far:].double().cpu().numpy(), want[1])


def test_repeats_itself(zc):
    g = np.random.default_rng(2)
    for which, (m, n, k) in ((0, (300, 512, 8192)), (1, (700, 900, 2000)), (2, (512, 512, 9000)), (0, (8, 4096, 4096))):
        a, b = operands(which, m, n, k, lambda *s: ref.bf16(g.standard_normal(s)))
        first = product(zc, which, a, b, m, n, k).numpy()
        for _ in range(3):
            assert np.array_equal(product(zc, which, a, b, m, n, k).numpy(), first)


def test_more_rows_than_small_tiles_fit_a_launch(zc):
    """A product by 1: every row has to come out as it went in."""
    m = (1 << 30) + 5
    a = (torch.arange(m, device="cuda", dtype=torch.int32) % 251 - 125).bfloat16()
    out = torch.full((m,), -1.0, dtype=torch.bfloat16, device="cuda")
    zc.zc_matmul(a, m, 1, torch.ones(1, dtype=torch.bfloat16, device="cuda"), 1, 1, 1, None, out, zc.ZC_BF16, 1)
    assert torch.equal(out.view(torch.int16), a.view(torch.int16))
