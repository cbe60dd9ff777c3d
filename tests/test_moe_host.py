"""Host-side checks of the mixture-of-experts operators that need no GPU: the
library exports every entry point of include/zc_moe.h, the sizes it reports, and
every argument it refuses, before anything is enqueued."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from lossless_bf16_exponent_amd import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that passes the alignment checks and is never read


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(_build.LIB):
        _build.build()
    from lossless_bf16_exponent_amd import zc_moe
    return zc_moe


@pytest.fixture(scope="module")
def zc():
    from lossless_bf16_exponent_amd import zc as mod
    return mod


def test_exports_every_declared_entry_point(moe):
    text = open(os.path.join(ROOT, "include", "zc_moe.h")).read()
    names = set(re.findall(r"^(?:zc_status|uint64_t)\s+(zc_[a-z_0-9]+)\s*\(", text, re.M))
    assert names == set(moe.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", _build.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (zc_\w+)", out))
    for name in ("ZC_MAX_EXPERTS", "ZC_MAX_TOP_K", "ZC_MAX_EXPERT_GROUPS", "ZC_FP8_BLOCK", "ZC_MOE_ROW_SLACK", "ZC_F32",
                 "ZC_BF16", "ZC_FP8_E4M3", "ZC_FP8_E5M2", "ZC_SCORE_SOFTMAX", "ZC_SCORE_SIGMOID", "ZC_FP8_SUM_FAST",
                 "ZC_FP8_SUM_FULL"):
        assert int(re.search(r"#define %s (\d+)u" % name, text).group(1)) == getattr(moe, name)


def test_header_compiles_as_c_and_cpp(tmp_path):
    for comp, std, ext in (("gcc", "-std=c11", "c"), ("g++", "-std=c++17", "cpp")):
        src = tmp_path / ("h." + ext)
        src.write_text('#include "zc_moe.h"\nint main(void) { return (int)sizeof(zc_route_config) - 32; }\n')
        subprocess.run([comp, std, "-Wall", "-Wextra", "-Werror", "-I", _build.INCLUDE, "-fsyntax-only", str(src)],
                       check=True)


def test_sizes(moe):
    assert [moe.zc_fp8_stride(c) for c in (0, 1, 128, 129, 7168)] == [0, 128, 128, 256, 7168]
    assert [moe.zc_fp8_scale_stride(c) for c in (0, 1, 512, 513, 7168)] == [0, 4, 4, 8, 56]
    g = np.random.default_rng(1)
    for _ in range(300):
        groups = int(g.integers(1, 70))
        counts = g.integers(0, 400, groups) * (g.random(groups) < 0.6)
        rows = int(counts.sum())
        assert sum((int(c) + 127) // 128 * 128 for c in counts) <= moe.zc_fp8_padded_rows(rows, groups)
        assert moe.zc_fp8_padded_rows(rows, groups) <= rows + 127 * groups
    assert moe.zc_fp8_padded_rows(1, 0) == 0
    assert moe.zc_dispatch_workspace_bytes(8192, 8, 256) % 256 == 0
    assert moe.zc_dispatch_workspace_bytes(8192, 8, 256) >= 4 * 257
    assert moe.zc_dispatch_workspace_bytes(8192, 0, 256) == 0
    assert moe.zc_dispatch_workspace_bytes(1 << 31, 1, 256) == 0
    for m, n, k, groups in ((1, 4096, 7168, 1), (64, 4096, 14336, 1), (65536, 4096, 7168, 32), (0, 0, 0, 1)):
        assert moe.zc_fp8_matmul_workspace_bytes(m, n, k, groups) <= moe.ZC_FP8_MATMUL_WORKSPACE_MAX


# (entry point, good arguments, [(argument index, bad value, status)]); the good arguments have no work to do or
# would be launched, so only the bad ones are called.
INVALID, CAPACITY, MISALIGNED = 1, 2, 3


def config(moe, **kw):
    base = dict(experts=64, top_k=4, score="sigmoid", groups=8, group_top=4, group_score=2)
    base.update(kw)
    return moe.route_config(**base)


def call(zc, moe, fn, args):
    conv = [ctypes.byref(a) if isinstance(a, moe.zc_route_config) else a for a in args]
    return zc.raw_status(fn, *conv)


def refusals(moe):
    cfg = config(moe)
    e4, bf = moe.ZC_FP8_E4M3, moe.ZC_BF16
    yield "zc_route", [P, 0, 4, 64, P, cfg, P, P, None], [
        (0, None, INVALID), (0, P + 2, MISALIGNED), (1, 2, INVALID), (2, 1 << 31, INVALID), (3, 63, INVALID),
        (4, P + 2, MISALIGNED), (6, None, INVALID), (6, P + 1, MISALIGNED), (7, None, INVALID), (7, P + 2, MISALIGNED)]
    yield "zc_route_backward", [P, 1, 4, 64, cfg, P, P, P, 64, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 3, INVALID), (5, None, INVALID), (6, None, INVALID),
        (7, None, INVALID), (7, P + 1, MISALIGNED), (8, 63, INVALID)]
    yield "zc_dispatch_plan", [P, 100, 8, 64, P, 1 << 20, P, P, P, None], [
        (0, None, INVALID), (0, P + 2, MISALIGNED), (1, 1 << 30, INVALID), (2, 0, INVALID), (2, 33, INVALID),
        (3, 0, INVALID), (3, 1025, INVALID), (4, None, INVALID), (4, P + 8, MISALIGNED), (5, 8, CAPACITY),
        (6, None, INVALID), (7, None, INVALID), (7, P + 1, MISALIGNED), (8, P + 2, MISALIGNED)]
    yield "zc_dispatch", [P, 10, 64, 64, P, 2, P, 20, 64, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 1 << 31, INVALID), (3, 63, INVALID), (4, None, INVALID),
        (4, P + 2, MISALIGNED), (5, 0, INVALID), (6, None, INVALID), (7, 1 << 31, INVALID), (8, 63, INVALID)]
    yield "zc_combine", [P, 20, 64, 64, P, P, 10, 2, P, 64, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 1 << 31, INVALID), (3, 63, INVALID), (4, None, INVALID),
        (5, P + 2, MISALIGNED), (6, 1 << 31, INVALID), (7, 0, INVALID), (7, 33, INVALID), (8, None, INVALID),
        (9, 63, INVALID)]
    yield "zc_combine_backward", [P, 64, P, 20, 64, 64, P, P, 10, 2, P, 64, P, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 63, INVALID), (2, None, INVALID), (5, 63, INVALID),
        (6, None, INVALID), (6, P + 2, MISALIGNED), (9, 0, INVALID), (10, P + 1, MISALIGNED), (11, 63, INVALID),
        (12, P + 2, MISALIGNED)]
    yield "zc_fp8_quantize", [P, 4, 200, 200, e4, 1, P, P, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 1 << 31, INVALID), (3, 199, INVALID), (4, bf, INVALID),
        (4, 4, INVALID), (5, 2, INVALID), (6, None, INVALID), (6, P + 8, MISALIGNED), (7, None, INVALID),
        (7, P + 2, MISALIGNED)]
    yield "zc_fp8_quantize_t", [P, P, e4, 300, 200, 256, 2, P, e4, P, P, 512, None], [
        (0, None, INVALID), (0, P + 2, MISALIGNED), (1, None, INVALID), (2, 0, INVALID), (5, 200, INVALID),
        (6, 0, INVALID), (6, 1025, INVALID), (7, None, INVALID), (7, P + 1, MISALIGNED), (8, 1, INVALID),
        (9, None, INVALID), (9, P + 8, MISALIGNED), (10, P + 2, MISALIGNED), (11, 384, CAPACITY), (11, 513, INVALID)]
    yield "zc_fp8_transpose", [P, P, 2, 200, 300, P, P, None], [
        (0, None, INVALID), (0, P + 8, MISALIGNED), (1, None, INVALID), (2, 1025, INVALID), (3, 1 << 29, INVALID),
        (5, None, INVALID), (6, P + 1, MISALIGNED)]
    yield "zc_fp8_matmul", [P, P, e4, 16, P, P, e4, 64, 128, 2, P, P, bf, 64, 0, None, 0, None], [
        (0, None, INVALID), (0, P + 8, MISALIGNED), (1, None, INVALID), (2, bf, INVALID), (3, 1 << 31, INVALID),
        (4, None, INVALID), (5, P + 2, MISALIGNED), (6, 0, INVALID), (7, 1 << 29, INVALID), (8, 1 << 29, INVALID),
        (9, 0, INVALID), (10, None, INVALID), (10, P + 2, MISALIGNED), (11, None, INVALID), (11, P + 1, MISALIGNED),
        (12, e4, INVALID), (13, 63, INVALID), (14, 2, INVALID), (15, P + 8, MISALIGNED)]
    yield "zc_fp8_matmul_wgrad", [P, P, e4, 64, P, P, e4, 64, 512, 300, 2, P, P, 0, 1, None], [
        (0, None, INVALID), (0, P + 8, MISALIGNED), (2, 0, INVALID), (6, 1, INVALID), (8, 384, CAPACITY),
        (8, 500, INVALID), (9, 1 << 31, INVALID), (10, 0, INVALID), (11, None, INVALID), (12, None, INVALID),
        (12, P + 2, MISALIGNED), (13, 2, INVALID), (14, 2, INVALID)]
    yield "zc_swiglu", [P, 4, 64, 128, P, 64, P, P, P, P, None], [
        (0, None, INVALID), (0, P + 1, MISALIGNED), (1, 1 << 31, INVALID), (3, 127, INVALID), (4, P + 1, MISALIGNED),
        (5, 63, INVALID), (6, None, INVALID), (7, None, INVALID), (8, P + 8, MISALIGNED), (9, None, INVALID)]
    yield "zc_swiglu_backward", [P, P, 4, 64, P, 64, P, 128, None], [
        (0, None, INVALID), (1, None, INVALID), (1, P + 2, MISALIGNED), (4, None, INVALID), (5, 63, INVALID),
        (6, P + 1, MISALIGNED), (7, 127, INVALID)]


def test_refusals(zc, moe):
    for fn, good, bad in refusals(moe):
        for index, value, status in bad:
            args = list(good)
            args[index] = value
            assert call(zc, moe, fn, args) == status, (fn, index, value)


@pytest.mark.parametrize("kw", [dict(experts=0), dict(experts=1025, groups=1, group_top=1), dict(groups=7), dict(groups=0),
                                dict(experts=128, groups=128, group_top=1), dict(group_top=0), dict(group_top=9),
                                dict(group_score=0), dict(group_score=3), dict(top_k=0), dict(top_k=33),
                                dict(group_top=1, top_k=9), dict(score=2), dict(renormalise=2),
                                dict(scale=float("nan")), dict(scale=float("inf"))])
def test_refused_configurations(zc, moe, kw):
    assert call(zc, moe, "zc_route", [P, 0, 4, 1024 + 1, None, config(moe, **kw), P, P, None]) == INVALID


def test_null_configuration(zc):
    assert zc.raw_status("zc_route", P, 0, 4, 64, None, None, P, P, None) == INVALID


def test_nothing_to_do_is_ok(zc, moe):
    """Counts of zero return ZC_OK without a launch (there is no GPU to launch on here)."""
    cfg = config(moe)
    e4 = moe.ZC_FP8_E4M3
    for fn, args in (("zc_route", [None, 0, 0, 64, None, cfg, None, None, None]),
                     ("zc_route_backward", [None, 0, 0, 64, cfg, None, None, None, 64, None]),
                     ("zc_dispatch", [None, 0, 64, 64, None, 2, None, 0, 64, None]),
                     ("zc_combine", [None, 0, 64, 64, None, None, 0, 2, None, 64, None]),
                     ("zc_combine_backward", [None, 64, None, 0, 64, 64, None, None, 0, 2, None, 64, None, None]),
                     ("zc_fp8_quantize", [None, 0, 64, 64, e4, 1, None, None, None]),
                     ("zc_fp8_quantize_t", [None, None, 1, 0, 64, 64, 1, None, e4, None, None, 0, None]),
                     ("zc_fp8_transpose", [None, None, 0, 64, 64, None, None, None]),
                     ("zc_fp8_matmul", [None, None, e4, 0, None, None, e4, 64, 64, 1, None, None, 1, 64, 0, None, 0, None]),
                     ("zc_fp8_matmul_wgrad", [None, None, e4, 0, None, None, e4, 64, 0, 0, 1, None, None, 1, 0, None]),
                     ("zc_swiglu", [None, 0, 64, 128, None, 64, None, None, None, None, None]),
                     ("zc_swiglu_backward", [None, None, 0, 64, None, 64, None, 128, None])):
        assert call(zc, moe, fn, args) == 0, fn


def test_products_are_summed_in_full_unless_told_otherwise(moe):
    """A caller who does not say how a product is summed gets the sums that lose nothing."""
    import inspect
    for f in (moe.zc_fp8_matmul, moe.zc_fp8_matmul_wgrad):
        assert inspect.signature(f).parameters["sum_mode"].default == moe.ZC_FP8_SUM_FULL
