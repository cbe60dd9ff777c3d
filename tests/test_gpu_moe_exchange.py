"""The order of token copies, the payload, the weighted sum and its gradients
against plain implementations: integers and moved values exactly, sums to the
roundings of 32 bits."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from moe_gpu import Out, bf16_device, close, device, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zc():
    return moe()


def plan_ref(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    on = (flat >= 0) & (flat < experts)
    order = np.lexsort((np.arange(flat.size), np.where(on, flat, experts)))
    position = np.empty(flat.size, dtype=np.int64)
    position[order] = np.arange(flat.size)
    counts = np.bincount(flat[on], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    source = np.where(np.arange(flat.size) < offsets[-1], order, -1)
    return offsets, np.where(on, position, -1).reshape(ids.shape), source


def plan(zc, ids, experts, with_source=True):
    t, k = ids.shape
    n = zc.zc_dispatch_workspace_bytes(t, k, experts)
    ws = Out((n,), torch.uint8)
    off, pos, src = Out((experts + 1,), torch.int32), Out((t, k), torch.int32), Out((t * k,), torch.int32)
    zc.zc_dispatch_plan(device(ids.astype(np.int32)), t, k, experts, ws, n, off, pos, src if with_source else None)
    ws.numpy()
    return off.numpy(), pos.numpy(), src.numpy()


@pytest.mark.parametrize("t,k,experts", [(1, 1, 1), (1, 8, 256), (3, 7, 5), (64, 1, 2), (255, 8, 256), (257, 8, 100),
                                         (700, 3, 1024), (8192, 8, 256), (33333, 2, 999)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "dropped", "one"])
def test_plan(zc, t, k, experts, kind):
    g = np.random.default_rng([t, k, experts])
    if kind == "uniform":
        ids = g.integers(0, experts, (t, k))
    elif kind == "skewed":
        ids = np.minimum((g.random((t, k)) ** 6 * experts).astype(np.int64), experts - 1)
    elif kind == "dropped":  # out of range on both sides
        ids = g.integers(-experts, 2 * experts, (t, k))
        ids[0, 0] = np.iinfo(np.int32).min
        ids[-1, -1] = np.iinfo(np.int32).max
    else:
        ids = np.full((t, k), experts - 1)
    off, pos, src = plan(zc, ids, experts)
    w_off, w_pos, w_src = plan_ref(ids, experts)
    assert np.array_equal(off, w_off)
    assert np.array_equal(pos, w_pos)
    assert np.array_equal(src, w_src)


def test_plan_without_source_and_without_tokens(zc):
    ids = np.random.default_rng(1).integers(0, 9, (100, 2))
    off, pos, src = plan(zc, ids, 9, with_source=False)
    assert np.array_equal(pos, plan_ref(ids, 9)[1])
    assert (src == np.array(0xA5A5A5A5, dtype=np.uint32).view(np.int32)).all()
    off = Out((10,), torch.int32)
    zc.zc_dispatch_plan(None, 0, 2, 9, None, 0, off, None, None)
    assert not off.numpy().any()


def positions(g, t, k, rows, drop):
    """Distinct rows of 0..rows-1 for the copies, some dropped (-1, or past the rows)."""
    pos = g.permutation(rows)[:t * k].reshape(t, k).astype(np.int64)
    if drop:
        pos[g.random((t, k)) < 0.3] = -1
        pos[g.random((t, k)) < 0.1] = rows + 3
        pos[0] = -1  # a token that went nowhere
    return pos


SHAPES = [(1, 1, 1, 1), (1, 8, 64, 0), (5, 2, 7, 1), (16, 8, 7168, 0), (33, 3, 1000, 0), (40, 6, 1001, 5),
          (130, 4, 2056, 8), (9, 32, 24, 0), (300, 8, 136, 8)]


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("t,k,hidden,gap", SHAPES)
def test_dispatch(zc, t, k, hidden, gap, drop):
    g = np.random.default_rng([t, k, hidden])
    rows = t * k + 5
    pos = positions(g, t, k, rows, drop)
    x = g.integers(0, 1 << 16, (t, hidden)).astype(np.uint16)  # every bit pattern moves unchanged
    xd = torch.zeros(t, hidden + gap, dtype=torch.int16, device="cuda")
    xd[:, :hidden] = torch.from_numpy(x.view(np.int16)).cuda()
    out = Out((rows, hidden + 2 * gap), torch.int16)
    zc.zc_dispatch(xd, t, hidden, hidden + gap, device(pos.astype(np.int32)), k, out, rows, hidden + 2 * gap)
    got = out.numpy().view(np.uint16)
    want = np.full((rows, hidden + 2 * gap), 0xA5A5, dtype=np.uint16)
    for i in range(t):
        for j in range(k):
            if 0 <= pos[i, j] < rows:
                want[pos[i, j], :hidden] = x[i]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("t,k,hidden,gap", SHAPES)
def test_combine_and_its_gradients(zc, t, k, hidden, gap, drop, weighted):
    g = np.random.default_rng([t, k, hidden, 1])
    rows = t * k + 5
    pos = positions(g, t, k, rows, drop)
    on = (pos >= 0) & (pos < rows)
    at = np.where(on, pos, 0)
    z = ref.bf16(g.standard_normal((rows, hidden)))
    w = g.random((t, k)).astype(np.float32).astype(np.float64) if weighted else np.ones((t, k))
    w_eff = np.where(on, w, 0.0)
    posd, wd = device(pos.astype(np.int32)), device(w.astype(np.float32)) if weighted else None
    zd = bf16_device(z, hidden + gap)
    y = Out((t, hidden + gap), torch.bfloat16)
    zc.zc_combine(zd, rows, hidden, hidden + gap, posd, wd, t, k, y, hidden + gap)
    got = y.numpy()[:, :hidden]
    want = (w_eff[:, :, None] * z[at]).sum(axis=1)
    size = (w_eff[:, :, None] * np.abs(z[at])).sum(axis=1)
    close(got, want, ref.BF16_HALF_STEP * np.abs(want) + (k + 1) * ref.F32_HALF_STEP * 2 * size + 2.0 ** -133, "y")

    dy = ref.bf16(g.standard_normal((t, hidden)))
    dyd = bf16_device(dy, hidden + gap)
    dz, dw = Out((rows, hidden + gap), torch.bfloat16), Out((t, k), torch.float32)
    zc.zc_combine_backward(dyd, hidden + gap, zd, rows, hidden, hidden + gap, posd, wd, t, k, dz, hidden + gap, dw)
    got_dz, got_dw = dz.numpy()[:, :hidden], dw.numpy()
    fill = float(torch.tensor([0xA5A5 - 65536], dtype=torch.int16).view(torch.bfloat16).double())
    want_dz, tol = np.full((rows, hidden), fill), np.zeros((rows, hidden))
    want_dz[pos[on]] = (w[:, :, None] * dy[:, None, :])[on]
    tol[pos[on]] = ref.BF16_HALF_STEP * np.abs(want_dz[pos[on]]) + 2.0 ** -133
    tol[pos[on]] *= 1 + 2.0 ** -15  # the 32-bit product's rounding, before BF16's
    close(got_dz, want_dz, tol, "dz")
    want_dw = np.where(on, (dy[:, None, :] * z[at]).sum(axis=2), 0.0)
    size = np.where(on, np.abs(dy[:, None, :] * z[at]).sum(axis=2), 0.0)
    # a sum of hidden terms: at most hidden / 256 in a row and a tree on top; hidden roundings bound it
    close(got_dw, want_dw, (hidden + 2) * ref.F32_HALF_STEP * size, "dw")

    # each gradient alone is the same
    dz2, dw2 = Out((rows, hidden + gap), torch.bfloat16), Out((t, k), torch.float32)
    zc.zc_combine_backward(dyd, hidden + gap, None, rows, hidden, 0, posd, wd, t, k, dz2, hidden + gap, None)
    zc.zc_combine_backward(dyd, hidden + gap, zd, rows, hidden, hidden + gap, posd, None, t, k, None, 0, dw2)
    assert np.array_equal(dz2.numpy()[:, :hidden], got_dz)
    assert np.array_equal(dw2.numpy(), got_dw)


def test_gradient_of_dispatch_is_the_plain_sum(zc):
    """<dispatch(x), d> = <x, combine(d)>: against differences of a linear map, its own product."""
    g = np.random.default_rng(4)
    t, k, h, rows = 50, 4, 96, 200
    pos = positions(g, t, k, rows, True)
    x, d = ref.bf16(g.standard_normal((t, h))), ref.bf16(g.standard_normal((rows, h)))
    out, dx = Out((rows, h), torch.bfloat16), Out((t, h), torch.bfloat16)
    out.t.zero_()
    posd = device(pos.astype(np.int32))
    zc.zc_dispatch(bf16_device(x), t, h, h, posd, k, out, rows, h)
    zc.zc_combine(bf16_device(d), rows, h, h, posd, None, t, k, dx, h)
    a, b = (out.numpy() * d).sum(), (x * dx.numpy()).sum()
    assert abs(a - b) <= ref.BF16_HALF_STEP * np.abs(x * dx.numpy()).sum() * 1.01


def test_combine_skips_what_is_masked(zc):
    """Infinities and NaN in rows that no copy names, and weights of dropped copies, take no part."""
    z = np.full((4, 16), np.nan)
    z[2] = 3.0
    w = np.array([[2.0, np.nan], [np.inf, np.nan]])
    pos = np.array([[2, -1], [-1, 4]])
    y = Out((2, 16), torch.bfloat16)
    zc.zc_combine(bf16_device(z), 4, 16, 16, device(pos.astype(np.int32)), device(w.astype(np.float32)), 2, 2, y, 16)
    got = y.numpy()
    assert (got[0] == 6.0).all() and not got[1].any()


def test_rows_past_32_bit_offsets(zc):
    """Rows whose byte offset passes 2^32 (the payload lies in a 4.4 GB buffer)."""
    rows, h = 300_000, 7168
    z = torch.empty(rows, h, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, h, device="cuda").bfloat16()
    pos = torch.tensor([[rows - 1, 5], [rows - 2, 299_593], [149_797, 0]], dtype=torch.int32, device="cuda")
    zc.zc_dispatch(x, 3, h, h, pos, 2, z, rows, h)
    y = torch.empty(3, h, dtype=torch.bfloat16, device="cuda")
    zc.zc_combine(z, rows, h, h, pos, None, 3, 2, y, h)
    torch.cuda.synchronize()
    assert torch.equal(z[pos.reshape(-1).long()], x.repeat_interleave(2, dim=0))
    assert torch.equal(y, (2 * x.float()).bfloat16())
