"""8-bit blocks: bytes and scales against the definition, exactly, in every layout
(rows, squares, transposed by groups); products against 64 bits."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from moe_gpu import Out, bf16_device, close, device, moe

pytestmark = pytest.mark.gpu

TYPES = [ref.E4M3, ref.E5M2]


@pytest.fixture(scope="module")
def zc():
    return moe()


def matrix(g, m, k):
    """BF16 values whose blocks differ in size by many powers of two."""
    x = g.standard_normal((m, k)) * 2.0 ** g.integers(-12, 13, (m, 1)) * 2.0 ** g.integers(-3, 4, (1, k))
    return ref.bf16(x)


def same_bytes(got, want, kind, what):
    """Equal bytes, or both NaN."""
    nan = np.isnan(ref.VALUES[kind])
    bad = (got != want) & ~(nan[got] & nan[want])
    assert not bad.any(), "%s: %d bytes differ, first at %s" % (what, int(bad.sum()), np.argwhere(bad)[:3].tolist())


def quantize(zc, x, kind, block_rows=1, stride=None, offset=0):
    m, k = x.shape
    q = Out((m, zc.zc_fp8_stride(k)), torch.uint8)
    s = Out((ref.up(m, block_rows) // block_rows, zc.zc_fp8_scale_stride(k)), torch.uint8)
    xd = bf16_device(x, stride, offset)
    zc.zc_fp8_quantize(xd, m, k, stride or k, kind, block_rows, q, s)
    return q, s


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,k,stride,offset", [(1, 1, None, 0), (1, 128, None, 0), (3, 130, None, 0), (129, 7, 9, 1),
                                               (128, 640, None, 0), (200, 1000, 1008, 0), (257, 384, 391, 3),
                                               (70, 520, 520, 8)])
def test_quantize(zc, kind, block_rows, m, k, stride, offset):
    x = matrix(np.random.default_rng([m, k]), m, k)
    q, s = quantize(zc, x, kind, block_rows, stride, offset)
    want_q, want_s = ref.quantize(x, kind, block_rows)
    assert np.array_equal(s.numpy(), want_s)
    same_bytes(q.numpy(), want_q, kind, "values")


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_every_bf16_pattern(zc, kind):
    """All 65,536 patterns, sorted so that a block holds one octave: every scale, subnormals, NaN and infinities."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(512, 128)
    xd = torch.from_numpy(bits.view(np.int16)).cuda().view(512, 128)
    q, s = Out((512, 128), torch.uint8), Out((512, 4), torch.uint8)
    zc.zc_fp8_quantize(xd, 512, 128, 128, kind, 1, q, s)
    want_q, want_s = ref.quantize(x, kind)
    assert np.array_equal(s.numpy(), want_s)
    same_bytes(q.numpy(), want_q, kind, "values")


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_ties_and_limits(zc, kind):
    """Blocks whose largest value is at, just below and just above 1.75 times a power of two; NaN and infinities
    beside finite values, which keep the scale that they have alone."""
    g = np.random.default_rng(6)
    x = ref.bf16(g.uniform(-1, 1, (8, 128)))
    for r, top in enumerate((1.75, 1.7421875, 1.7578125, 1.0, 1.9921875)):
        x[r, 17] = top * 2.0 ** (r - 3)
    x[5, 3], x[5, 4] = np.nan, np.inf
    x[6] = np.inf
    x[7] = 0.0
    q, s = quantize(zc, x, kind)
    want_q, want_s = ref.quantize(x, kind)
    assert np.array_equal(s.numpy(), want_s)
    same_bytes(q.numpy(), want_q, kind, "values")


GROUPS = [(1, None, 300), (1, None, 1), (4, [0, 0, 130, 130, 300], 300), (3, [5, 128, 256, 290], 300),
          (70, None, 500), (4, [-9, 200, 100, 9000, 250], 300)]


def offsets_of(groups, offsets, rows):
    if offsets is None and groups > 1:
        offsets = np.sort(np.random.default_rng(groups).integers(0, rows + 1, groups + 1))
    return offsets


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("source", ["bf16", "kept"])
@pytest.mark.parametrize("cols,gap", [(1, 0), (64, 0), (200, 0), (333, 2)])
@pytest.mark.parametrize("groups,offsets,rows", GROUPS)
def test_quantize_t(zc, groups, offsets, rows, cols, gap, source, kind):
    offsets = offsets_of(groups, offsets, rows)
    x = matrix(np.random.default_rng([rows, cols]), rows, cols)
    padded = zc.zc_fp8_padded_rows(rows, groups) + 128
    od = None if offsets is None else device(np.asarray(offsets, dtype=np.int32))
    q, s = Out((cols, padded), torch.uint8), Out((cols, zc.zc_fp8_scale_stride(padded)), torch.uint8)
    if source == "bf16":
        zc.zc_fp8_quantize_t(bf16_device(x, cols + gap), None, zc.ZC_BF16, rows, cols, cols + gap, groups, od, kind, q,
                             s, padded)
    else:  # the checkpoint of a forward pass, e4m3
        kq, ks = quantize(zc, x, ref.E4M3)
        zc.zc_fp8_quantize_t(kq, ks, ref.E4M3, rows, cols, zc.zc_fp8_stride(cols), groups, od, kind, q, s, padded)
        x = ref.values(kq.numpy(), ks.numpy(), ref.E4M3, cols)
    want_q, want_s, used = ref.quantize_t(x, kind, groups, offsets, padded)
    got_q, got_s = q.numpy(), s.numpy()
    assert np.array_equal(got_s[:, :used // 128], want_s[:, :used // 128])
    same_bytes(got_q[:, :used], want_q[:, :used], kind, "values")
    assert (got_q[:, used:] == 0xA5).all(), "columns of no group were written"


@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (2, 128, 256), (3, 200, 130), (1, 513, 640)])
def test_transpose(zc, batch, rows, cols):
    g = np.random.default_rng([rows, cols])
    qs, ss = zc.zc_fp8_stride(cols), zc.zc_fp8_scale_stride(cols)
    qts, sts = zc.zc_fp8_stride(rows), zc.zc_fp8_scale_stride(rows)
    rb, cb = ref.up(rows, 128) // 128, ref.up(cols, 128) // 128
    q = np.zeros((batch, rows, qs), dtype=np.uint8)
    q[:, :, :cols] = g.integers(0, 256, (batch, rows, cols))
    s = np.zeros((batch, rb, ss), dtype=np.uint8)
    s[:, :, :cb] = g.integers(0, 248, (batch, rb, cb))
    qt, st = Out((batch, cols, qts), torch.uint8), Out((batch, cb, sts), torch.uint8)
    zc.zc_fp8_transpose(device(q), device(s), batch, rows, cols, qt, st)
    want_q, want_s = np.zeros((batch, cols, qts), dtype=np.uint8), np.zeros((batch, cb, sts), dtype=np.uint8)
    want_q[:, :, :rows] = q[:, :, :cols].transpose(0, 2, 1)
    want_s[:, :, :rb] = s[:, :, :cb].transpose(0, 2, 1)
    assert np.array_equal(qt.numpy(), want_q)
    assert np.array_equal(st.numpy(), want_s)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def product_tolerance(want, size, terms, f32):
    """Each of the terms' additions rounds (or truncates) to 24 bits; then the result's own rounding."""
    return (0 if f32 else ref.BF16_HALF_STEP) * np.abs(want) + (terms + 8) * 2 * ref.F32_HALF_STEP * size + 2.0 ** -126


def weights(g, groups, n, k, kind):
    qs, ss, vs = [], [], []
    for _ in range(groups):
        w = ref.bf16(g.standard_normal((n, k)) * 2.0 ** g.integers(-8, 3))
        q, s = ref.quantize(w, kind, 128)
        qs.append(q)
        ss.append(s)
        vs.append(ref.values(q, s, kind, k, 128))
    return np.stack(qs), np.stack(ss), vs


def matmul(zc, g, m, n, k, groups, offsets, ta=ref.E4M3, tb=ref.E4M3, f32=False, gap=0, workspace=False):
    x = matrix(g, m, k)
    aq, as_ = ref.quantize(x, ta)
    bq, bs, bv = weights(g, groups, n, k, tb)
    out = Out((m, n + gap), torch.float32 if f32 else torch.bfloat16)
    od = None if offsets is None else device(np.asarray(offsets, dtype=np.int32))
    nb = zc.zc_fp8_matmul_workspace_bytes(m, n, k, groups) if workspace else 0
    ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda") if workspace else None  # NaN, if read unwritten
    aqd, asd, bqd, bsd = device(aq), device(as_), device(bq), device(bs)
    zc.zc_fp8_matmul(aqd, asd, ta, m, bqd, bsd, tb, n, k, groups, od, out, zc.ZC_F32 if f32 else zc.ZC_BF16, n + gap,
                     zc.ZC_FP8_SUM_FULL, ws, nb)
    got = out.numpy()
    a = ref.values(aq, as_, ta, k)
    fill = np.float64(np.uint32(0xA5A5A5A5).view(np.float32)) if f32 else float(
        torch.tensor([0xA5A5 - 65536], dtype=torch.int16).view(torch.bfloat16).double())
    want, tol = np.full((m, n + gap), fill), np.zeros((m, n + gap))
    for i, (r0, r1) in enumerate(ref.spans(offsets, groups, m)):
        want[r0:r1, :n] = a[r0:r1] @ bv[i].T
        size = np.abs(a[r0:r1]) @ np.abs(bv[i]).T
        tol[r0:r1, :n] = product_tolerance(want[r0:r1, :n], size, k, f32)
    close(got, want, tol, "product %s" % ((m, n, k, groups),))


@pytest.mark.parametrize("ta", TYPES)
@pytest.mark.parametrize("tb", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (130, 140, 300), (40, 70, 520)])
def test_matmul_types(zc, ta, tb, f32, m, n, k):
    matmul(zc, np.random.default_rng([m, n, k]), m, n, k, 1, None, ta, tb, f32)


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 128, 128), (1, 516, 1030), (2, 64, 4096), (7, 300, 640), (16, 256, 1152), (17, 129, 129),
                                   (32, 1000, 2000), (33, 96, 2049), (48, 260, 896), (64, 512, 1536), (65, 132, 768),
                                   (100, 1028, 384), (128, 256, 1280), (200, 250, 257), (256, 512, 512), (257, 513, 1025),
                                   (500, 300, 700), (700, 1100, 640)])
def test_matmul_sizes(zc, m, n, k, workspace):
    matmul(zc, np.random.default_rng([m, n, k]), m, n, k, 1, None, gap=n % 5, workspace=workspace)


@pytest.mark.parametrize("groups,offsets,rows", [
    (1, [0, 40], 40), (3, [0, 0, 40, 40], 40), (4, [0, 100, 100, 400, 700], 700), (3, [10, 20, 300, 310], 330),
    (8, [0, 1, 2, 3, 4, 5, 6, 7, 8], 8), (8, [0, 1, 1, 3, 4, 4, 4, 7, 8], 8), (5, [-3, 50, 20, 90, 4000, 60], 100),
    (70, None, 300), (130, None, 64), (2, [0, 257, 257 + 511], 768)])
@pytest.mark.parametrize("n,k", [(200, 300), (516, 1024)])
def test_matmul_groups(zc, groups, offsets, rows, n, k):
    offsets = offsets_of(groups, offsets, rows)
    for workspace in (False, True):
        matmul(zc, np.random.default_rng([groups, n]), rows, n, k, groups, offsets, workspace=workspace)


def fast_tolerance(a, b, want, f32):
    """ZC_FP8_SUM_FAST: the 8-bit instructions lose, in 64 neighbouring products, up to 2^-11.4 of the largest of them
    (their arithmetic, measured on 4,096 sums of single instructions); 2^-10 of it is allowed here, for every 64, on top of the
    tolerance of full sums."""
    k = ref.up(a.shape[1], 64)
    a = np.pad(np.abs(a), ((0, 0), (0, k - a.shape[1])))
    b = np.pad(np.abs(b), ((0, 0), (0, k - b.shape[1])))
    lost = np.zeros((a.shape[0], b.shape[0]))
    for c in range(0, k, 64):
        largest = np.zeros_like(lost)
        for i in range(c, c + 64):
            np.maximum(largest, np.outer(a[:, i], b[:, i]), out=largest)
        lost += largest
    return product_tolerance(want, a @ b.T, k, f32) + 2.0 ** -10 * lost


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ta,tb", [(ref.E4M3, ref.E4M3), (ref.E5M2, ref.E4M3), (ref.E4M3, ref.E5M2), (ref.E5M2, ref.E5M2)])
@pytest.mark.parametrize("m,n,k,groups,offsets", [
    (1, 5, 3, 1, None), (70, 90, 200, 1, None), (200, 260, 640, 1, None), (300, 516, 1100, 3, [0, 7, 290, 300]),
    (600, 270, 384, 2, [0, 300, 600])])
def test_matmul_fast(zc, m, n, k, groups, offsets, ta, tb, f32):
    g = np.random.default_rng([m, n, k, 9])
    aq, as_ = ref.quantize(matrix(g, m, k), ta)
    bq, bs, bv = weights(g, groups, n, k, tb)
    a = ref.values(aq, as_, ta, k)
    od = None if offsets is None else device(np.asarray(offsets, dtype=np.int32))
    out = Out((m, n), torch.float32 if f32 else torch.bfloat16)
    ops = [device(v) for v in (aq, as_, bq, bs)]
    zc.zc_fp8_matmul(ops[0], ops[1], ta, m, ops[2], ops[3], tb, n, k, groups, od, out, zc.ZC_F32 if f32 else zc.ZC_BF16, n,
                     zc.ZC_FP8_SUM_FAST)
    got = out.numpy()
    for i, (r0, r1) in enumerate(ref.spans(offsets, groups, m)):
        want = a[r0:r1] @ bv[i].T
        close(got[r0:r1], want, fast_tolerance(a[r0:r1], bv[i], want, f32), "group %d" % i)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ta,tb", [(ref.E4M3, ref.E4M3), (ref.E5M2, ref.E4M3)])
@pytest.mark.parametrize("n,k", [(90, 70), (516, 260)])
def test_wgrad_fast(zc, n, k, ta, tb, f32):
    g = np.random.default_rng([n, k, 4])
    rows, groups, offsets = 700, 4, [0, 3, 400, 400, 700]
    dy, x = matrix(g, rows, n), matrix(g, rows, k)
    padded = zc.zc_fp8_padded_rows(rows, groups)
    od = device(np.asarray(offsets, dtype=np.int32))
    ops = []
    for v, cols, kind in ((dy, n, ta), (x, k, tb)):
        q = Out((cols, padded), torch.uint8)
        s = Out((cols, zc.zc_fp8_scale_stride(padded)), torch.uint8)
        zc.zc_fp8_quantize_t(bf16_device(v), None, zc.ZC_BF16, rows, cols, cols, groups, od, kind, q, s, padded)
        ops.append((q, s))
    out = Out((groups, n, k), torch.float32 if f32 else torch.bfloat16)
    zc.zc_fp8_matmul_wgrad(*ops[0], ta, n, *ops[1], tb, k, padded, rows, groups, od, out,
                           zc.ZC_F32 if f32 else zc.ZC_BF16, zc.ZC_FP8_SUM_FAST)
    got = out.numpy()
    for i, (r0, r1) in enumerate(ref.spans(offsets, groups, rows)):
        if r0 == r1:
            assert not got[i].any()
            continue
        a = ref.values(*ref.quantize(np.ascontiguousarray(dy[r0:r1].T), ta), ta, r1 - r0)
        b = ref.values(*ref.quantize(np.ascontiguousarray(x[r0:r1].T), tb), tb, r1 - r0)
        want = a @ b.T
        close(got[i], want, fast_tolerance(a, b, want, f32), "group %d" % i)


def test_matmul_without_contraction(zc):
    out = Out((5, 9), torch.float32)
    zc.zc_fp8_matmul(None, None, ref.E4M3, 5, None, None, ref.E4M3, 9, 0, 1, None, out, zc.ZC_F32, 9)
    assert not out.numpy().any()


def test_matmul_special_values(zc):
    """NaN of one row or column stays in it; an infinity of the other type spreads as it does in a sum."""
    g = np.random.default_rng(12)
    m, n, k = 70, 90, 260
    x, w = ref.bf16(g.standard_normal((m, k))), ref.bf16(g.standard_normal((n, k)))
    x[3, 7], w[5, 200] = np.nan, np.inf
    aq, as_ = ref.quantize(x, ref.E4M3)
    bq, bs = ref.quantize(w, ref.E5M2, 128)
    out = Out((m, n), torch.float32)
    aqd, asd, bqd, bsd = device(aq), device(as_), device(bq), device(bs)
    zc.zc_fp8_matmul(aqd, asd, ref.E4M3, m, bqd, bsd, ref.E5M2, n, k, 1, None, out, zc.ZC_F32, n)
    got = out.numpy()
    assert np.isnan(got[3]).all()
    assert not np.isfinite(got[:, 5]).any()
    rest = np.delete(np.delete(got, 3, axis=0), 5, axis=1)
    assert np.isfinite(rest).all()


@pytest.mark.parametrize("groups,offsets,rows", GROUPS)
@pytest.mark.parametrize("n,k,ta,f32", [(1, 1, ref.E4M3, True), (200, 300, ref.E5M2, False), (516, 256, ref.E4M3, True)])
def test_wgrad(zc, groups, offsets, rows, n, k, ta, f32):
    """dW = dY^T X over every group's tokens, from the transposed blocks that the library makes."""
    offsets = offsets_of(groups, offsets, rows)
    g = np.random.default_rng([rows, n])
    dy, x = matrix(g, rows, n), matrix(g, rows, k)
    padded = zc.zc_fp8_padded_rows(rows, groups)
    od = None if offsets is None else device(np.asarray(offsets, dtype=np.int32))
    ops = []
    for v, cols, kind in ((dy, n, ta), (x, k, ref.E4M3)):
        q = torch.full((cols, padded), 0x7F, dtype=torch.uint8, device="cuda")  # NaN in columns of no group
        s = torch.full((cols, zc.zc_fp8_scale_stride(padded)), 0xFF, dtype=torch.uint8, device="cuda")
        zc.zc_fp8_quantize_t(bf16_device(v), None, zc.ZC_BF16, rows, cols, cols, groups, od, kind, q, s, padded)
        ops.append((q, s))
    out = Out((groups, n, k), torch.float32 if f32 else torch.bfloat16)
    zc.zc_fp8_matmul_wgrad(*ops[0], ta, n, *ops[1], ref.E4M3, k, padded, rows, groups, od, out,
                           zc.ZC_F32 if f32 else zc.ZC_BF16, zc.ZC_FP8_SUM_FULL)
    got = out.numpy()
    for i, (r0, r1) in enumerate(ref.spans(offsets, groups, rows)):
        if r0 == r1:
            assert not got[i].any()
            continue
        a = ref.values(*ref.quantize(np.ascontiguousarray(dy[r0:r1].T), ta), ta, r1 - r0)
        b = ref.values(*ref.quantize(np.ascontiguousarray(x[r0:r1].T), ref.E4M3), ref.E4M3, r1 - r0)
        want = a @ b.T
        close(got[i], want, product_tolerance(want, np.abs(a) @ np.abs(b).T, r1 - r0, f32), "group %d" % i)


def test_wgrad_without_rows(zc):
    out = Out((2, 6, 10), torch.bfloat16)
    off = device(np.zeros(3, dtype=np.int32))
    zc.zc_fp8_matmul_wgrad(None, None, ref.E4M3, 6, None, None, ref.E4M3, 10, 0, 0, 2, off, out, zc.ZC_BF16)
    assert not out.numpy().any()


def test_product_gradients_against_differences(zc):
    """dX and dW of L = <Y, D> where Y is the product of what the 8-bit inputs stand for: L is linear in each, so a
    difference of any length is exact, and only the gradients' own 8-bit inputs differ (D is chosen to be exact)."""
    g = np.random.default_rng(21)
    m, n, k = 96, 130, 200
    x = matrix(g, m, k)
    xq, xs = ref.quantize(x, ref.E4M3)
    xv = ref.values(xq, xs, ref.E4M3, k)
    wq, ws, wv = weights(g, 1, n, k, ref.E4M3)
    d = ref.bf16(g.integers(-8, 9, (m, n)).astype(np.float64))  # whole numbers to 8: exact in e4m3 under any scale
    dq, ds = ref.quantize(d, ref.E4M3)
    wt, wts = Out((k, zc.zc_fp8_stride(n)), torch.uint8), Out((ref.up(k, 128) // 128, zc.zc_fp8_scale_stride(n)), torch.uint8)
    zc.zc_fp8_transpose(device(wq), device(ws), 1, n, k, wt, wts)
    dx = Out((m, k), torch.float32)
    zc.zc_fp8_matmul(device(dq), device(ds), ref.E4M3, m, wt, wts, ref.E4M3, k, n, 1, None, dx, zc.ZC_F32, k, zc.ZC_FP8_SUM_FULL)
    got_dx = dx.numpy()
    for i, j in ((0, 0), (5, 199), (95, 100), (50, 64)):
        e = np.zeros_like(xv)
        e[i, j] = 1.0
        diff = (((xv + e) @ wv[0].T * d).sum() - ((xv - e) @ wv[0].T * d).sum()) / 2
        size = np.abs(d[i]) @ np.abs(wv[0][:, j])
        assert abs(got_dx[i, j] - diff) <= 2 * (n + 8) * ref.F32_HALF_STEP * size + 1e-9 * np.abs(xv @ wv[0].T * d).sum()
    padded = zc.zc_fp8_padded_rows(m, 1)
    ops = []
    for src, sc, kind, cols, stride in ((bf16_device(d), None, zc.ZC_BF16, n, n),
                                        (device(xq), device(xs), ref.E4M3, k, zc.zc_fp8_stride(k))):
        q = Out((cols, padded), torch.uint8)
        s = Out((cols, zc.zc_fp8_scale_stride(padded)), torch.uint8)
        zc.zc_fp8_quantize_t(src, sc, kind, m, cols, stride, 1, None, ref.E4M3, q, s, padded)
        ops.append((q, s))
    dw = Out((n, k), torch.float32)
    zc.zc_fp8_matmul_wgrad(*ops[0], ref.E4M3, n, *ops[1], ref.E4M3, k, padded, m, 1, None, dw, zc.ZC_F32,
                           zc.ZC_FP8_SUM_FULL)
    got_dw = dw.numpy()
    xt = ref.values(ops[1][0].numpy(), ops[1][1].numpy(), ref.E4M3, m).T  # the checkpoint, re-blocked along the tokens
    for i, j in ((0, 0), (129, 199), (64, 3)):
        diff = (d[:, i] * xt[:, j]).sum()
        size = (np.abs(d[:, i]) * np.abs(xt[:, j])).sum()
        assert abs(got_dw[i, j] - diff) <= 2 * (m + 8) * ref.F32_HALF_STEP * size + 1e-12


# ---------------------------------------------------------------------------
# more tiles than the device holds at once
# ---------------------------------------------------------------------------

def close_on_device(got, a, b, f32, what):
    """got against a b^T in 64 bits on the device, within fast_tolerance's bound with the largest product of 64 taken as
    the product of the largest factors."""
    a, b = a.double(), b.double()
    want = a @ b.T
    k = ref.up(a.shape[1], 64)

    def largest(v):
        return torch.nn.functional.pad(v.abs(), (0, k - v.shape[1])).view(v.shape[0], -1, 64).amax(dim=2)

    tol = (0 if f32 else ref.BF16_HALF_STEP) * want.abs() + (a.shape[1] + 8) * 2 * ref.F32_HALF_STEP * (a.abs() @ b.abs().T)
    tol += 2.0 ** -10 * (largest(a) @ largest(b).T) + 2.0 ** -126
    over = (got.double() - want).abs() > tol
    assert not bool(over.any()), "%s: %d of %d off" % (what, int(over.sum()), over.numel())


def stood_for(q, s, cols, block_rows=1):
    """What e4m3 blocks on the device stand for, in 64 bits."""
    t = torch.tensor(ref.VALUES[ref.E4M3], device="cuda")[q.long()]
    e = torch.exp2(s.double() - 127).round(decimals=60)[:, :t.shape[1] // 128].repeat_interleave(128, dim=1)
    return (t * e.repeat_interleave(block_rows, dim=0)[:t.shape[0]])[:, :cols]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k,groups", [(4400, 4500, 128, 1), (4352, 4352, 256, 1), (4400, 4353, 300, 1), (4500, 4609, 640, 1),
                                          (9000, 2100, 1100, 5), (4800, 8200, 384, 9)])
def test_matmul_many_tiles(zc, m, n, k, groups, f32):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    x = (torch.randn(m, k, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 7, (m, 1), generator=g, device="cuda"))).bfloat16()
    w = (torch.randn(groups, n, k, generator=g, device="cuda") * 0.1).bfloat16()
    xq, xs = Out((m, zc.zc_fp8_stride(k)), torch.uint8), Out((m, zc.zc_fp8_scale_stride(k)), torch.uint8)
    zc.zc_fp8_quantize(x, m, k, k, ref.E4M3, 1, xq, xs)
    wq = Out((groups, n, zc.zc_fp8_stride(k)), torch.uint8)
    ws = Out((groups, ref.up(n, 128) // 128, zc.zc_fp8_scale_stride(k)), torch.uint8)
    for i in range(groups):
        zc.zc_fp8_quantize(w[i], n, k, k, ref.E4M3, 128, wq.t[i], ws.t[i])
    cuts = np.sort(np.random.default_rng(m).integers(0, m + 1, groups - 1))
    offsets = np.concatenate([[0], cuts, [m]])
    out = Out((m, n + 3), torch.float32 if f32 else torch.bfloat16)
    for _ in range(2):  # the second time over the first one's results
        zc.zc_fp8_matmul(xq, xs, ref.E4M3, m, wq, ws, ref.E4M3, n, k, groups, device(offsets.astype(np.int32)), out,
                         zc.ZC_F32 if f32 else zc.ZC_BF16, n + 3)
    out.numpy()
    a = stood_for(xq.t, xs.t, k)
    for i, (r0, r1) in enumerate(zip(offsets, offsets[1:])):
        if r0 < r1:
            close_on_device(out.t[r0:r1, :n], a[r0:r1], stood_for(wq.t[i], ws.t[i], k, 128), f32, "group %d" % i)


@pytest.mark.parametrize("f32", [False, True])
def test_wgrad_many_tiles(zc, f32):
    """Groups of no, one, two and more blocks of tokens, next to each other."""
    n, k = 1100, 1300
    counts = [300, 0, 1, 700, 128, 129, 0, 256, 5, 1000, 385, 64]
    rows, groups = sum(counts), len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dy, x = torch.randn(rows, n, generator=g, device="cuda").bfloat16(), torch.randn(rows, k, generator=g, device="cuda").bfloat16()
    padded = zc.zc_fp8_padded_rows(rows, groups)
    od = device(offsets.astype(np.int32))
    ops = []
    for v, cols in ((dy, n), (x, k)):
        q = torch.full((cols, padded), 0x7F, dtype=torch.uint8, device="cuda")
        s = torch.full((cols, zc.zc_fp8_scale_stride(padded)), 0xFF, dtype=torch.uint8, device="cuda")
        zc.zc_fp8_quantize_t(v, None, zc.ZC_BF16, rows, cols, cols, groups, od, ref.E4M3, q, s, padded)
        ops.append((q, s))
    out = Out((groups, n, k), torch.float32 if f32 else torch.bfloat16)
    for _ in range(2):
        zc.zc_fp8_matmul_wgrad(*ops[0], ref.E4M3, n, *ops[1], ref.E4M3, k, padded, rows, groups, od, out,
                               zc.ZC_F32 if f32 else zc.ZC_BF16)
    out.numpy()
    at = 0
    for i, c in enumerate(counts):
        if not c:
            assert not bool(out.t[i].any())
            continue
        b0, b1 = at // 128, at // 128 + ref.up(c, 128) // 128
        pair = [stood_for(q[:, 128 * b0:128 * b1], s[:, b0:b1], c) for q, s in ops]
        close_on_device(out.t[i], *pair, f32, "group %d" % i)
        at = 128 * b1
