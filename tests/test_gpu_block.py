"""The example's whole block (norms, router, experts, shared expert, losses, and every gradient) against 64 bits, and the
norms, products and balance losses under HIP graph replay, on other streams and after another call's error."""
import ctypes
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import block_ref as ref
import moe_ref
import test_gpu_moe_layer as layer_test
from moe_gpu import Out, moe, to_numpy

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def zc():
    return moe()


@pytest.fixture(scope="module")
def example(zc):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def oracle(cfg, x, p, dr, loss_weight=0.01, z_weight=0.001):
    """The block in 64 bits with the roundings that its definition has: BF16 results of every call, and those of
    the experts' layer."""
    none, sigmoid = ref.Side(), cfg.score == 1
    before, after = ref.Side(ref.RMS, p["before"]), ref.Side(ref.RMS, p["after"])
    t = x.shape[0]
    y = ref.bf16(ref.norm(x, None, none, before, None, None, 1.0)[2])
    logits = y @ p["router"].T
    routed = layer_test.oracle(cfg, y, logits, p["w1"], p["w2"], np.zeros_like(x))[0]
    v = y @ p["s1"].T + p["b1"]
    pre, hs = ref.bf16(v), ref.bf16(ref.activation(v, 2)[0])
    z = ref.bf16(hs @ p["s2"].T + ref.bf16(routed))
    r = ref.bf16(ref.norm(x, z, after, none, p["gate"], None, 1.0)[0])
    ids = moe_ref.route(logits, None, cfg)[0]
    whole = [0, t]
    counts, used, loss, zl = ref.balance(logits, ids, None, whole, cfg.experts, cfg.top_k, sigmoid)
    o = ref.norm_backward(r, z, after, none, p["gate"], None, 1.0, dr, None)
    g = {"after": o["dw1"][0], "gate": o["dgate"][0]}
    dz = ref.bf16(o["dz"][0])
    _, dy, dlogits, g["w1"], g["w2"] = layer_test.oracle(cfg, y, logits, p["w1"], p["w2"], dz)
    g["s2"] = dz.T @ hs
    d = ref.bf16(dz @ p["s2"]) * ref.activation(pre, 2)[1]
    g["b1"] = d.sum(axis=0)
    g["s1"] = ref.bf16(d).T @ y
    dy = ref.bf16(ref.bf16(dy) + ref.bf16(d) @ p["s1"])
    dl = ref.bf16(ref.balance_backward(logits, None, whole, cfg.experts, cfg.top_k, sigmoid, counts, used, np.array([loss_weight]),
                                       np.array([z_weight]), dlogits)[0])
    g["router"] = dl.T @ y
    dy = ref.bf16(dy + dl @ p["router"])
    o = ref.norm_backward(x, None, none, before, None, None, 1.0, ref.bf16(dr), dy)
    g["before"] = o["dw2"][0]
    return r, loss[0], zl[0], o["dx"][0], g


@pytest.mark.parametrize("kw,score,top_k,destinations", [
    (dict(tokens=300, hidden=256, inner=192, shared=128, experts=16), "sigmoid", 4, 4),
    (dict(tokens=1, hidden=512, inner=128, shared=256, experts=8), "sigmoid", 8, 8),
    (dict(tokens=700, hidden=648, inner=200, shared=136, experts=8), "softmax", 2, 2)])
def test_block_against_64_bits(zc, example, kw, score, top_k, destinations):
    x, dr, params = example.inputs(**kw)
    cfg = zc.route_config(kw["experts"], top_k, score, scale=2.0)
    block = example.Block(cfg, params, destinations)
    r, loss, z_loss = block.forward(x)
    dx, g = block.backward(dr)
    torch.cuda.synchronize()
    want = oracle(cfg, to_numpy(x), {n: to_numpy(v) for n, v in params.items()}, to_numpy(dr))
    branch = to_numpy(x)
    pairs = [("branch", to_numpy(r) - branch, want[0] - branch), ("dx", to_numpy(dx), want[3]),
             *((n, to_numpy(g[n]), want[4][n]) for n in example.NAMES)]
    for name, a, b in pairs:
        off = np.linalg.norm(a - b) / np.linalg.norm(b)
        # the branch is the difference of BF16 sums: half a step of the sum, beside the branch itself
        slack = ref.BF16_HALF_STEP * np.linalg.norm(branch) / np.linalg.norm(b) if name == "branch" else 0.0
        assert off <= layer_test.LIMIT + slack, (name, off)
    assert abs(float(loss) - want[1]) <= 1e-4 * want[1] and abs(float(z_loss) - want[2]) <= 1e-4 * want[2]


class Step:
    """Every call on buffers of its own, from inputs that can be refilled; `outputs` lists the results."""

    def __init__(self, zc, tokens=600, hidden=520, inner=392, experts=24, top_k=3, seed=0, workspace=None):
        self.zc, self.shape = zc, (tokens, hidden, inner, experts, top_k)
        t, h, f, e = tokens, hidden, inner, experts
        bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

        def z(*shape, dtype=bf):
            return torch.zeros(*shape, dtype=dtype, device="cuda")

        g = torch.Generator(device="cuda")
        g.manual_seed(11)

        def weight(*shape, scale=0.05, mean=0.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).bfloat16()

        self.x, self.z, self.dr, self.dy = z(t, h), z(t, h), z(t, h), z(t, h)
        self.dout, self.add = z(t, f), z(t, h)
        self.w, self.router, self.bias = weight(f, h), weight(e, h), weight(f).float()
        self.cfg = zc.norm_config(zc.norm_params(zc.ZC_NORM_LAYER, weight(h, mean=1.0), weight(h)),
                                  zc.norm_params(zc.ZC_NORM_RMS, weight(h, mean=1.0)), weight(h, mean=0.5), weight(t).float(), 0.5)
        self.rc = zc.route_config(e, top_k, "sigmoid")
        self.offsets = torch.tensor([0, 100, 100, t - 20], dtype=i32, device="cuda")
        self.mask = (torch.arange(t, device="cuda") % 7 != 3).to(u8)
        self.dloss, self.dzl = torch.tensor([0.1, 0.2, 0.3], device="cuda"), torch.tensor([0.01, 0.02, 0.03], device="cuda")
        self.r, self.y, self.yq, self.ys = z(t, h), z(t, h), z(t, zc.zc_fp8_stride(h), dtype=u8), z(t, zc.zc_fp8_scale_stride(h), dtype=u8)
        self.dx, self.dz = z(t, h), z(t, h)
        self.g = [z(h, dtype=f32) for _ in range(5)] + [z(t, dtype=f32)]
        self.logits, self.pre, self.out = z(t, e, dtype=f32), z(t, f), z(t, f)
        self.dpre, self.dbias, self.da, self.dw = z(t, f), z(f, dtype=f32), z(t, h), z(f, h, dtype=f32)
        self.drouter = z(e, h, dtype=f32)
        self.dl = z(t, e)
        self.ids, self.weights = z(t, top_k, dtype=i32), z(t, top_k, dtype=f32)
        self.counts, self.used = z(3, e, dtype=i32), z(3, dtype=i32)
        self.loss, self.zloss, self.dlogits = z(3, dtype=f32), z(3, dtype=f32), z(t, e, dtype=f32)
        need = max(zc.zc_norm_backward_workspace_bytes(t, h), zc.zc_activation_backward_workspace_bytes(t, f),
                   zc.zc_balance_workspace_bytes(t, e, 3), zc.ZC_MATMUL_WORKSPACE_MAX)
        self.ws = z(need, dtype=u8) if workspace is None else workspace
        self.outputs = ["r", "y", "yq", "ys", "dx", "dz", "logits", "pre", "out", "dpre", "dbias", "da", "dw", "drouter", "dl",
                        "ids", "counts", "used", "loss", "zloss", "dlogits"]
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(500 + seed)
        for v in (self.x, self.z, self.dr, self.dy, self.dout, self.add):
            v.copy_(torch.randn(v.shape, generator=g, device="cuda"))

    def run(self, stream=None):
        zc, (t, h, f, e, k) = self.zc, self.shape
        bf, f32 = zc.ZC_BF16, zc.ZC_F32
        kw, ws = {"stream": stream}, (self.ws, self.ws.numel())
        zc.zc_norm(self.x, bf, t, h, h, self.z, h, self.cfg, self.r, h, self.y, h, self.yq, self.ys, **kw)
        zc.zc_matmul(self.y, t, h, self.router, e, h, h, None, self.logits, f32, e, *ws, **kw)
        ep = zc.epilogue(self.bias, zc.ZC_ACT_GELU, pre=self.pre, pre_stride=f)
        zc.zc_matmul(self.y, t, h, self.w, f, h, h, ep, self.out, bf, f, *ws, **kw)
        zc.zc_route(self.logits, f32, t, e, None, self.rc, self.ids, self.weights, **kw)
        zc.zc_balance(self.logits, f32, t, e, self.rc, self.ids, self.mask, 3, self.offsets, *ws, self.counts, self.used,
                      self.loss, self.zloss, **kw)
        zc.zc_balance_backward(self.logits, f32, t, e, self.rc, self.mask, 3, self.offsets, self.counts, self.used, self.dloss,
                               self.dzl, None, 0, self.dlogits, e, **kw)
        zc.zc_activation_backward(self.dout, bf, t, f, f, self.pre, f, zc.ZC_ACT_GELU, 1.0, self.dpre, f, self.dbias, *ws, **kw)
        zc.zc_matmul_dgrad(self.dpre, t, f, f, self.w, h, h, self.add, bf, h, self.da, bf, h, *ws, **kw)
        zc.zc_matmul_wgrad(self.dpre, t, f, f, self.y, h, h, None, f32, h, self.dw, f32, h, *ws, **kw)
        zc.zc_activation_backward(self.dlogits, f32, t, e, e, None, 0, zc.ZC_ACT_NONE, 1.0, self.dl, e, **kw)
        zc.zc_matmul_wgrad(self.dl, t, e, e, self.y, h, h, None, f32, h, self.drouter, f32, h, *ws, **kw)
        zc.zc_matmul_dgrad(self.dl, t, e, e, self.router, h, h, self.da, bf, h, self.da, bf, h, *ws, **kw)
        zc.zc_norm_backward(self.r, bf, t, h, h, self.z, h, self.cfg, self.dr, h, self.da, h, self.dx, h, self.dz, h,
                            zc.norm_grads(*self.g), *ws, **kw)

    def results(self):
        torch.cuda.synchronize()
        return {**{n: getattr(self, n).clone() for n in self.outputs}, **{"g%d" % i: v.clone() for i, v in enumerate(self.g)}}


same = layer_test.same


@pytest.mark.parametrize("kw", [dict(), dict(tokens=33, hidden=300, inner=77, experts=5, top_k=2), dict(tokens=140, hidden=1032, inner=2000)])
def test_results_are_reproducible(zc, kw):
    s = Step(zc, **{**dict(tokens=200), **kw})
    s.run()
    first = s.results()
    for _ in range(3):
        s.run()
        same(s.results(), first, "the same inputs again")


def captured(step):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step.run()
    return graph


def test_graphs_replay_with_new_inputs(zc):
    """Two captured graphs of all calls that share a workspace, replayed in turn with new inputs between eager work: every
    replay equals the eager results."""
    a = Step(zc)
    b = Step(zc, tokens=450, hidden=264, inner=520, experts=40, workspace=a.ws)
    for s in (a, b):
        s.run()
    graphs = [captured(s) for s in (a, b)]
    eager = [Step(zc), Step(zc, tokens=450, hidden=264, inner=520, experts=40)]
    for seed in (1, 2, 3, 4):
        for s, graph, e in zip((a, b), graphs, eager):
            e.fill(seed)
            e.run()
            want = e.results()
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


def test_two_streams_at_once(zc):
    """Calls on two streams at the same time, each with its own buffers and workspace."""
    a, b = Step(zc), Step(zc, tokens=450)
    want = []
    for s in (a, b):
        s.run()
        want.append(s.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, st in zip((a, b), streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        same(s.results(), w, "two streams")


def test_a_pending_error_is_not_reported(zc):
    """An error that another call left pending in the HIP runtime is not a call's own."""
    s = Step(zc, tokens=40)
    torch.cuda.synchronize()
    run = {n: getattr(zc, n) for n in ("zc_norm", "zc_matmul", "zc_route", "zc_balance", "zc_balance_backward",
                                       "zc_activation_backward", "zc_matmul_dgrad", "zc_matmul_wgrad", "zc_norm_backward")}

    class Leaves:
        """The calls, each after an error that the runtime keeps until somebody asks for it."""

        def __getattr__(self, name):
            if name not in run:
                return getattr(zc, name)

            def call(*args, **kw):
                torch.cuda.synchronize()
                assert zc._lib.hipSetDevice(ctypes.c_int(1 << 20)) != 0
                run[name](*args, **kw)  # raises zc.ZcError for anything but ZC_OK
            return call

    s.zc = Leaves()
    s.run()
    torch.cuda.synchronize()


def test_workspace_too_small_is_not_used(zc):
    """A product whose workspace is too small, or not there, is not split and leaves it as it is."""
    m, n, k = 128, 128, 8192
    need = zc.zc_matmul_workspace_bytes(m, n, k)
    assert need
    a, w = torch.ones(m, k, dtype=torch.bfloat16, device="cuda"), torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
    for room in (0, need - 1):
        out, ws = Out((m, n), torch.float32), Out((need,), torch.uint8)
        zc.zc_matmul(a, m, k, w, n, k, k, None, out, zc.ZC_F32, n, ws, room)
        assert (out.numpy() == k).all() and bool((ws.raw == 0xA5).all())
