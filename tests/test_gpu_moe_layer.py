"""The example's whole layer (routing, exchange through the codec, 8-bit products,
gated activation, and every gradient) against 64 bits, and the operators under HIP
graph replay and on other streams."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_ref as ref
from moe_gpu import moe, to_numpy

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def zc():
    return moe()


@pytest.fixture(scope="module")
def example(zc):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rows8(x):
    return ref.values(*ref.quantize(x, ref.E4M3), ref.E4M3, x.shape[1])


def squares8(w):
    return ref.values(*ref.quantize(w, ref.E4M3, 128), ref.E4M3, w.shape[1], 128)


def oracle(cfg, x, logits, w1, w2, dy):
    """The layer in 64 bits with the roundings that its definition has: BF16 results of every call, 8-bit blocks of every
    product's operands, the kept gates and ups."""
    t, h = x.shape
    f, k = w2.shape[2], cfg.top_k
    ids, weights, _ = ref.route(logits, None, cfg)
    y, dx, dweights = np.zeros((t, h)), np.zeros((t, h)), np.zeros((t, k))
    dw1, dw2 = np.zeros(w1.shape), np.zeros(w2.shape)
    for e in range(cfg.experts):
        r, c = np.nonzero(ids == e)
        if not r.size:
            continue
        w1q, w2q = squares8(w1[e]), squares8(w2[e])
        x8 = rows8(x[r])
        gu = ref.bf16(x8 @ w1q.T)
        h8 = rows8(ref.bf16(ref.swiglu(gu[:, :f], gu[:, f:])))
        z = ref.bf16(h8 @ w2q.T)
        np.add.at(y, r, weights[r, c, None] * z)
        dweights[r, c] = (dy[r] * z).sum(axis=1)
        dz = ref.bf16(weights[r, c, None] * dy[r])
        dh = ref.bf16(rows8(dz) @ w2q)
        dw2[e] = rows8(dz.T) @ rows8(h8.T).T
        dg, du, _ = ref.swiglu_backward(rows8(gu[:, :f]), rows8(gu[:, f:]), dh)
        dgu = ref.bf16(np.concatenate([dg, du], axis=1))
        np.add.at(dx, r, ref.bf16(rows8(dgu) @ w1q))
        dw1[e] = rows8(dgu.T) @ rows8(x8.T).T
    return y, dx, ref.route_backward(logits, cfg, ids, dweights)[0], dw1, dw2


# A value in front of a rounding differs by 2^-16 or so of itself (8-bit instructions, 32-bit sums): one in some hundred
# rounds to the other BF16 neighbour (2^-8), and one in some thousand then to the other 8-bit one (2^-3.5).  The mean square
# of that over a result is about 0.1 %, and BF16 results add 0.2 % of their own.
LIMIT = 0.01


@pytest.mark.parametrize("kw,score,top_k,destinations", [
    (dict(tokens=300, hidden=256, inner=192, experts=16), "sigmoid", 4, 4),
    (dict(tokens=1, hidden=512, inner=128, experts=8), "sigmoid", 8, 8),
    (dict(tokens=1000, hidden=648, inner=200, experts=8), "softmax", 2, 2)])
def test_layer_against_64_bits(zc, example, kw, score, top_k, destinations):
    x, dy, logits, w1, w2 = example.inputs(**kw)
    cfg = zc.route_config(kw["experts"], top_k, score, scale=2.0)
    layer = example.Layer(cfg, w1, w2, destinations)
    y = layer.forward(x, logits)
    got = y, *layer.backward(dy)
    torch.cuda.synchronize()
    want = oracle(cfg, *(to_numpy(v) for v in (x, logits, w1, w2, dy)))
    for name, a, b in zip(("y", "dx", "dlogits", "dw1", "dw2"), got, want):
        off = np.linalg.norm(to_numpy(a) - b) / np.linalg.norm(b)
        assert off <= LIMIT, (name, off)
    assert layer.compressed < 0.8 * 2 * kw["tokens"] * top_k * kw["hidden"] + 4096 * destinations


class Step:
    """Every call on buffers of its own, from inputs that can be refilled; `outputs` lists the results."""

    def __init__(self, zc, tokens=700, hidden=256, inner=192, experts=12, top_k=3, seed=0):
        self.zc, self.shape = zc, (tokens, hidden, inner, experts, top_k)
        rows, f = tokens * top_k, inner

        def e(*shape, dtype=torch.bfloat16):
            return torch.zeros(*shape, dtype=dtype, device="cuda")

        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        S, SS = zc.zc_fp8_stride, zc.zc_fp8_scale_stride
        self.x, self.dy, self.logits = e(tokens, hidden), e(tokens, hidden), e(tokens, experts, dtype=f32)
        self.cfg = zc.route_config(experts, top_k, "sigmoid", groups=4, group_top=2, group_score=2, scale=1.5)
        self.bias = torch.linspace(-0.05, 0.05, experts, device="cuda")
        self.ids, self.w = e(tokens, top_k, dtype=i32), e(tokens, top_k, dtype=f32)
        self.off, self.pos = e(experts + 1, dtype=i32), e(tokens, top_k, dtype=i32)
        self.src = e(rows, dtype=i32)
        self.ws = e(zc.zc_dispatch_workspace_bytes(tokens, top_k, experts), dtype=u8)
        self.mws = e(64 << 20, dtype=u8)
        self.pay, self.xq, self.xs = e(rows, hidden), e(rows, S(hidden), dtype=u8), e(rows, SS(hidden), dtype=u8)
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        w1 = (torch.randn(experts, 2 * f, hidden, generator=g, device="cuda") * 0.06).bfloat16()
        self.w1, self.w1s = e(experts, 2 * f, S(hidden), dtype=u8), e(experts, (2 * f + 127) // 128, SS(hidden), dtype=u8)
        for i in range(experts):
            zc.zc_fp8_quantize(w1[i], 2 * f, hidden, hidden, zc.ZC_FP8_E4M3, 128, self.w1[i], self.w1s[i])
        self.w1t, self.w1ts = e(experts, hidden, S(2 * f), dtype=u8), e(experts, (hidden + 127) // 128, SS(2 * f), dtype=u8)
        zc.zc_fp8_transpose(self.w1, self.w1s, experts, 2 * f, hidden, self.w1t, self.w1ts)
        self.gu, self.h = e(rows, 2 * f), e(rows, f)
        self.hq, self.hs = e(rows, S(f), dtype=u8), e(rows, SS(f), dtype=u8)
        self.kq, self.ks = e(rows, 2 * S(f), dtype=u8), e(rows, SS(2 * S(f)), dtype=u8)
        self.dgu, self.dq, self.ds = e(rows, 2 * f), e(rows, S(2 * f), dtype=u8), e(rows, SS(2 * f), dtype=u8)
        self.dpay = e(rows, hidden)
        self.padded = zc.zc_fp8_padded_rows(rows, experts)
        self.at, self.ats = e(2 * f, self.padded, dtype=u8), e(2 * f, SS(self.padded), dtype=u8)
        self.bt, self.bts = e(hidden, self.padded, dtype=u8), e(hidden, SS(self.padded), dtype=u8)
        self.dw = e(experts, 2 * f, hidden, dtype=f32)
        self.y, self.dpay2, self.dweights = e(tokens, hidden), e(rows, hidden), e(tokens, top_k, dtype=f32)
        self.dlogits = e(tokens, experts, dtype=f32)
        self.outputs = ["ids", "w", "off", "pos", "src", "pay", "xq", "xs", "gu", "h", "hq", "hs", "kq", "ks", "dgu", "dq",
                        "ds", "dpay", "dw", "y", "dpay2", "dweights", "dlogits"]
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + seed)
        for t in (self.x, self.dy, self.logits):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    def run(self, stream=None):
        zc, (t, hd, f, e, k) = self.zc, self.shape
        rows, e4 = t * k, zc.ZC_FP8_E4M3
        kw = {"stream": stream}
        zc.zc_route(self.logits, zc.ZC_F32, t, e, self.bias, self.cfg, self.ids, self.w, **kw)
        zc.zc_dispatch_plan(self.ids, t, k, e, self.ws, self.ws.numel(), self.off, self.pos, self.src, **kw)
        zc.zc_dispatch(self.x, t, hd, hd, self.pos, k, self.pay, rows, hd, **kw)
        zc.zc_fp8_quantize(self.pay, rows, hd, hd, e4, 1, self.xq, self.xs, **kw)
        zc.zc_fp8_matmul(self.xq, self.xs, e4, rows, self.w1, self.w1s, e4, 2 * f, hd, e, self.off, self.gu, zc.ZC_BF16, 2 * f,
                         zc.ZC_FP8_SUM_FAST, self.mws, self.mws.numel(), **kw)
        zc.zc_swiglu(self.gu, rows, f, 2 * f, self.h, f, self.hq, self.hs, self.kq, self.ks, **kw)
        zc.zc_swiglu_backward(self.kq, self.ks, rows, f, self.h, f, self.dgu, 2 * f, **kw)
        zc.zc_fp8_quantize(self.dgu, rows, 2 * f, 2 * f, e4, 1, self.dq, self.ds, **kw)
        zc.zc_fp8_matmul(self.dq, self.ds, e4, rows, self.w1t, self.w1ts, e4, hd, 2 * f, e, self.off, self.dpay, zc.ZC_BF16,
                         hd, zc.ZC_FP8_SUM_FULL, self.mws, self.mws.numel(), **kw)
        zc.zc_fp8_quantize_t(self.dgu, None, zc.ZC_BF16, rows, 2 * f, 2 * f, e, self.off, e4, self.at, self.ats, self.padded,
                             **kw)
        zc.zc_fp8_quantize_t(self.xq, self.xs, e4, rows, hd, zc.zc_fp8_stride(hd), e, self.off, e4, self.bt, self.bts,
                             self.padded, **kw)
        zc.zc_fp8_matmul_wgrad(self.at, self.ats, e4, 2 * f, self.bt, self.bts, e4, hd, self.padded, rows, e, self.off,
                               self.dw, zc.ZC_F32, zc.ZC_FP8_SUM_FAST, **kw)
        zc.zc_combine(self.dpay, rows, hd, hd, self.pos, self.w, t, k, self.y, hd, **kw)
        zc.zc_combine_backward(self.dy, hd, self.dpay, rows, hd, hd, self.pos, self.w, t, k, self.dpay2, hd, self.dweights,
                               **kw)
        zc.zc_route_backward(self.logits, zc.ZC_F32, t, e, self.cfg, self.ids, self.dweights, self.dlogits, e, **kw)

    def results(self):
        torch.cuda.synchronize()
        return {n: getattr(self, n).clone() for n in self.outputs}


def same(got, want, what):
    for name in want:
        a, b = got[name].contiguous().view(torch.uint8), want[name].contiguous().view(torch.uint8)
        assert torch.equal(a, b), "%s: %s differs in %d bytes" % (what, name, int((a != b).sum()))


def test_results_are_reproducible(zc):
    s = Step(zc)
    s.run()
    first = s.results()
    for _ in range(3):
        s.run()
        same(s.results(), first, "the same inputs again")


def test_graph_replays_with_new_inputs(zc):
    """One captured graph of all calls, replayed with new inputs between eager work: every replay equals the eager
    results."""
    s = Step(zc)
    s.run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        s.run()
    eager = Step(zc)
    for seed in (1, 2, 3, 4):
        eager.fill(seed)
        eager.run()
        want = eager.results()
        s.fill(seed)
        graph.replay()
        same(s.results(), want, "replay %d" % seed)


def test_other_stream_with_work_before_it(zc):
    """The inputs are made on the stream that the calls are given, while other work runs on the default one."""
    a, b = Step(zc), Step(zc)
    a.fill(9)
    a.run()
    want = a.results()
    st = torch.cuda.Stream()
    noise = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        b.fill(9)
    for _ in range(5):
        noise = noise @ noise * 1e-3
    b.run(stream=st)
    st.synchronize()
    same(b.results(), want, "another stream")
