"""Products at sizes that reach every tile shape with the 8-bit instructions: 256 x
128 tiles, split contractions whose parts start inside four blocks of scales, and
256 x 256 tiles with either type in either place."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from moe_gpu import Out, close, device, moe
from test_gpu_moe_fp8 import close_on_device, fast_tolerance, product_tolerance

pytestmark = pytest.mark.gpu
TYPES = [(ref.E4M3, ref.E4M3), (ref.E5M2, ref.E4M3), (ref.E4M3, ref.E5M2), (ref.E5M2, ref.E5M2)]


@pytest.fixture(scope="module")
def zc():
    return moe()


def stood_for(q, s, kind, cols, block_rows=1):
    """What the blocks on the device stand for, in 64 bits."""
    t = torch.tensor(ref.VALUES[kind], device="cuda")[q.long()]
    e = (s.int()[:, :q.shape[1] // 128] - 127).repeat_interleave(128, dim=1).repeat_interleave(block_rows, dim=0)
    return torch.ldexp(t, e[:t.shape[0]])[:, :cols]


def values(g, rows, cols):
    """Gaussian rows of very different sizes."""
    size = torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda"))
    return (torch.randn(rows, cols, generator=g, device="cuda") * size).bfloat16()


def product(zc, m, n, k, groups, ta, tb, f32, workspace=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    xq, xs = Out((m, zc.zc_fp8_stride(k)), torch.uint8), Out((m, zc.zc_fp8_scale_stride(k)), torch.uint8)
    zc.zc_fp8_quantize(values(g, m, k), m, k, k, ta, 1, xq, xs)
    wq = Out((groups, n, zc.zc_fp8_stride(k)), torch.uint8)
    ws = Out((groups, ref.up(n, 128) // 128, zc.zc_fp8_scale_stride(k)), torch.uint8)
    for i in range(groups):
        zc.zc_fp8_quantize(values(g, n, k), n, k, k, tb, 128, wq.t[i], ws.t[i])
    offsets = np.linspace(0, m, groups + 1).astype(np.int32) + np.array([0] + [i % 7 for i in range(1, groups)] + [0], dtype=np.int32)
    od = device(offsets)
    out = Out((m, n + 3), torch.float32 if f32 else torch.bfloat16)
    nb = zc.zc_fp8_matmul_workspace_bytes(m, n, k, groups) if workspace else 0
    assert bool(nb) == workspace, "the contraction is not split"
    room = Out((nb,), torch.uint8) if workspace else None
    zc.zc_fp8_matmul(xq, xs, ta, m, wq, ws, tb, n, k, groups, od, out, zc.ZC_F32 if f32 else zc.ZC_BF16, n + 3,
                     zc.ZC_FP8_SUM_FAST, room, nb)
    out.numpy()
    assert bool((out.t.contiguous().view(torch.uint8).view(m, n + 3, -1)[:, n:] == 0xA5).all()), "written between the rows"
    if workspace:
        room.numpy()
    a = stood_for(xq.t, xs.t, ta, k)
    for i, (r0, r1) in enumerate(zip(offsets, offsets[1:])):
        close_on_device(out.t[r0:r1, :n], a[r0:r1], stood_for(wq.t[i], ws.t[i], tb, k, 128), f32, "group %d" % i)


# 256 x 128 tiles: more than 256 tiles of 128 x 128, at most 256 of 256 x 128, a contraction of more than 8 blocks
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ta,tb", TYPES)
@pytest.mark.parametrize("m,n,k,groups", [(1100, 4001, 1500, 1), (1153, 4100, 2310, 1), (1285, 3000, 1300, 4)])
def test_tiles_of_256_by_128(zc, m, n, k, groups, ta, tb, f32):
    product(zc, m, n, k, groups, ta, tb, f32)


# parts of 18 blocks in 4 start at blocks 0, 4, 9, 13; of 15 in 2 at 0 and 7; of 41 in 8 at 0, 5, 10, 15, 20, 25, 30, 35
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ta,tb", TYPES)
@pytest.mark.parametrize("m,n,k,groups", [(300, 200, 2200, 1), (100, 300, 1920, 1), (130, 261, 5131, 1), (600, 300, 2304, 3),
                                          (70, 129, 2816, 2), (333, 514, 3000, 1)])
def test_split_contractions(zc, m, n, k, groups, ta, tb, f32):
    product(zc, m, n, k, groups, ta, tb, f32, workspace=True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ta,tb", TYPES)
@pytest.mark.parametrize("m,n,k,groups", [(2001, 4100, 1100, 1), (5000, 2100, 650, 3), (4400, 4500, 128, 1), (4352, 4352, 256, 1),
                                          (4500, 4609, 640, 1), (9000, 2100, 1100, 5), (4800, 8200, 384, 9)])
def test_tiles_of_256_by_256(zc, m, n, k, groups, ta, tb, f32):
    product(zc, m, n, k, groups, ta, tb, f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ta,tb", TYPES)
@pytest.mark.parametrize("counts", [[300, 1, 700, 0, 129, 1000, 385], [300, 0, 1, 700, 128, 129, 0, 256, 5, 1000, 385, 64]],
                         ids=["7groups", "12groups"])
def test_weight_gradients_of_256_by_256(zc, counts, ta, tb, f32):
    n, k = 1100, 1300  # 5 x 6 tiles a group
    rows, groups = sum(counts), len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    padded = zc.zc_fp8_padded_rows(rows, groups)
    od = device(offsets.astype(np.int32))
    ops = []
    for cols, kind in ((n, ta), (k, tb)):
        q = torch.full((cols, padded), 0x7F, dtype=torch.uint8, device="cuda")
        s = torch.full((cols, zc.zc_fp8_scale_stride(padded)), 0xFF, dtype=torch.uint8, device="cuda")
        zc.zc_fp8_quantize_t(values(g, rows, cols), None, zc.ZC_BF16, rows, cols, cols, groups, od, kind, q, s, padded)
        ops.append((q, s, kind))
    out = Out((groups, n, k), torch.float32 if f32 else torch.bfloat16)
    zc.zc_fp8_matmul_wgrad(*ops[0][:2], ta, n, *ops[1][:2], tb, k, padded, rows, groups, od, out,
                           zc.ZC_F32 if f32 else zc.ZC_BF16, zc.ZC_FP8_SUM_FAST)
    out.numpy()
    at = 0
    for i, c in enumerate(counts):
        if not c:
            assert not bool(out.t[i].any())
            continue
        b0, b1 = at // 128, at // 128 + ref.up(c, 128) // 128
        pair = [stood_for(q[:, 128 * b0:128 * b1], s[:, b0:b1], kind, c) for q, s, kind in ops]
        close_on_device(out.t[i], *pair, f32, "group %d" % i)
        at = 128 * b1


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("m", [3, 70])
@pytest.mark.parametrize("ta,tb", TYPES)
def test_smallest_and_largest_scales(zc, ta, tb, m, fast):
    """Blocks next to the smallest numbers (scale bytes 0 to 3) times blocks next to the largest, and the other way round."""
    n, k = 66, 256
    r = np.random.default_rng([m, ta, tb])
    for low, high in ((-126, 100), (-117, 110), (-130, 115)):
        small, large = [ref.bf16(r.uniform(-2, 2, (rows, k)) * 2.0 ** e) for rows, e in ((m, low), (n, high))]
        for swap in (False, True):
            x, w = (ref.bf16(large[:1] * r.uniform(0.5, 1.0, (m, 1))), ref.bf16(small[:1] * r.uniform(0.5, 1.0, (n, 1)))) if swap else (small, large)
            aq, as_ = ref.quantize(x, ta)
            bq, bs = ref.quantize(w, tb, 128)
            a, b = ref.values(aq, as_, ta, k), ref.values(bq, bs, tb, k, 128)
            out = Out((m, n), torch.float32)
            ops = [device(v) for v in (aq, as_, bq, bs)]
            zc.zc_fp8_matmul(ops[0], ops[1], ta, m, ops[2], ops[3], tb, n, k, 1, None, out, zc.ZC_F32, n,
                             zc.ZC_FP8_SUM_FAST if fast else zc.ZC_FP8_SUM_FULL)
            want = a @ b.T
            tol = fast_tolerance(a, b, want, True) if fast else product_tolerance(want, np.abs(a) @ np.abs(b).T, k, True)
            close(out.numpy(), want, tol, "scales %s" % ((low, high, swap),))


@pytest.mark.parametrize("kind", [ref.E4M3, ref.E5M2])
@pytest.mark.parametrize("exponent", [-133, -130, -126, -118, 100, 120])
def test_reblocking_keeps_the_smallest_values(zc, kind, exponent):
    """The transposed form of an 8-bit checkpoint whose values are next to the smallest or the largest numbers."""
    rows, cols = 150, 200
    r = np.random.default_rng([kind, exponent + 200])
    x = ref.bf16(r.uniform(-4, 4, (rows, cols)) * 2.0 ** exponent)
    q, s = ref.quantize(x, kind)
    padded = zc.zc_fp8_padded_rows(rows, 1)
    qt, st = Out((cols, padded), torch.uint8), Out((cols, zc.zc_fp8_scale_stride(padded)), torch.uint8)
    zc.zc_fp8_quantize_t(device(q), device(s), kind, rows, cols, zc.zc_fp8_stride(cols), 1, None, ref.E4M3, qt, st, padded)
    want_q, want_s, n = ref.quantize_t(ref.values(q, s, kind, cols), ref.E4M3, 1, None, padded)
    assert n == padded and np.array_equal(qt.numpy(), want_q)
    assert np.array_equal(st.numpy()[:, :padded // 128], want_s[:, :padded // 128])
