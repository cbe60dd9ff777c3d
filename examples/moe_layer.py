"""One mixture-of-experts layer, forward and backward, through the library's calls.

What a rank does around the all-to-all of such a layer, on one GPU that plays every
destination (the exchange itself is a copy here):

  forward   route the tokens; order their copies by expert; make the payload; compress one
            segment per destination and decompress it at the receiver; two 8-bit products
            per expert with the gated activation between them; weighted sum
  backward  gradients of the weights and of the experts' rows; of the second product, the
            activation (from its 8-bit checkpoint) and the first product; of the tokens and
            of the router's logits

    python examples/moe_layer.py [--tokens 2048 --hidden 1024 --inner 512 --experts 32 --top-k 4]

Prints the compressed size of the payload and how far the layer's output and its gradients
are from the same layer in 64 bits without any rounding: what 8-bit inputs cost, a few
percent.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_bf16_exponent_amd import zc, zc_moe as moe  # noqa: E402

E4M3, BF16, F32 = moe.ZC_FP8_E4M3, moe.ZC_BF16, moe.ZC_F32


def buf(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Weights:
    """The experts' matrices (one n x k matrix each) in 8-bit squares, and their transposes for the backward pass."""

    def __init__(self, w):
        self.groups, self.n, self.k = w.shape
        self.q, self.s = self._buffers(self.n, self.k)
        for g in range(self.groups):
            moe.zc_fp8_quantize(w[g], self.n, self.k, self.k, E4M3, 128, self.q[g], self.s[g])
        self.qt, self.st = self._buffers(self.k, self.n)
        moe.zc_fp8_transpose(self.q, self.s, self.groups, self.n, self.k, self.qt, self.st)

    def _buffers(self, rows, cols):
        return (buf(self.groups, rows, moe.zc_fp8_stride(cols), dtype=torch.uint8),
                buf(self.groups, (rows + 127) // 128, moe.zc_fp8_scale_stride(cols), dtype=torch.uint8))


class Layer:
    """w1: experts x 2 inner x hidden (gates, then ups); w2: experts x hidden x inner; BF16."""

    def __init__(self, config, w1, w2, destinations):
        self.config, self.destinations = config, destinations
        self.w1, self.w2 = Weights(w1), Weights(w2)
        self.hidden, self.inner = w2.shape[1], w2.shape[2]
        self.workspace = buf(moe.ZC_FP8_MATMUL_WORKSPACE_MAX, dtype=torch.uint8)

    # -- the pieces -----------------------------------------------------------------------------------------------

    def rows8(self, x):
        rows, cols = x.shape
        q = buf(rows, moe.zc_fp8_stride(cols), dtype=torch.uint8)
        s = buf(rows, moe.zc_fp8_scale_stride(cols), dtype=torch.uint8)
        moe.zc_fp8_quantize(x, rows, cols, cols, E4M3, 1, q, s)
        return q, s

    def product(self, x8, rows, q, s, n, k, offsets):
        out = buf(rows, n)
        moe.zc_fp8_matmul(x8[0], x8[1], E4M3, rows, q, s, E4M3, n, k, self.config.experts, offsets, out, BF16, n,
                          moe.ZC_FP8_SUM_FAST, self.workspace, self.workspace.numel())
        return out

    def transposed8(self, x, scales, kind, rows, cols, stride, offsets):
        """Blocks along every expert's tokens: what the weight gradient contracts."""
        padded = moe.zc_fp8_padded_rows(rows, self.config.experts)
        q, s = buf(cols, padded, dtype=torch.uint8), buf(cols, moe.zc_fp8_scale_stride(padded), dtype=torch.uint8)
        moe.zc_fp8_quantize_t(x, scales, kind, rows, cols, stride, self.config.experts, offsets, E4M3, q, s, padded)
        return q, s, padded

    def weight_gradient(self, dy, x8, rows, n, k, offsets):
        a, a_s, padded = self.transposed8(dy, None, BF16, rows, n, n, offsets)
        b, b_s, _ = self.transposed8(x8[0], x8[1], E4M3, rows, k, moe.zc_fp8_stride(k), offsets)
        dw = buf(self.config.experts, n, k, dtype=torch.float32)
        moe.zc_fp8_matmul_wgrad(a, a_s, E4M3, n, b, b_s, E4M3, k, padded, rows, self.config.experts, offsets, dw, F32)
        return dw

    def exchange(self, payload, offsets):
        """Compresses the payload's segment of every destination and decompresses it at the other side."""
        per = self.config.experts // self.destinations
        bounds = [int(offsets[d * per]) for d in range(self.destinations)] + [int(offsets[-1])]
        ns = [(b - a) * self.hidden for a, b in zip(bounds, bounds[1:])]
        plan = zc.zc_plan_from_sigma(1.0)
        room = [(zc.zc_max_compressed_bytes(n) + 255) // 256 * 256 for n in ns]
        streams = buf(sum(room), dtype=torch.uint8)
        starts = [sum(room[:d]) for d in range(self.destinations)]
        sizes = torch.zeros(self.destinations, dtype=torch.int64, device="cuda")
        ws = buf(max(256, sum(zc.zc_compress_workspace_bytes(n) for n in ns)), dtype=torch.uint8)
        arrived = torch.empty_like(payload)
        status = torch.full((self.destinations,), -1, dtype=torch.int32, device="cuda")
        at = [payload.data_ptr() + 2 * a * self.hidden for a in bounds]
        to = [arrived.data_ptr() + 2 * a * self.hidden for a in bounds]
        zc.zc_compress_batch_ws([(at[d], ns[d], plan, streams.data_ptr() + starts[d], room[d], sizes.data_ptr() + 8 * d)
                                 for d in range(self.destinations)], ws, ws.numel())
        got = sizes.tolist()
        zc.zc_decompress_batch([(streams.data_ptr() + starts[d], got[d], ns[d], to[d], status.data_ptr() + 4 * d)
                                for d in range(self.destinations)])
        if status.any():
            raise RuntimeError("a stream did not decompress: %s" % status.tolist())
        return arrived, sum(got)

    # -- the layer ------------------------------------------------------------------------------------------------

    def forward(self, x, logits):
        t, e, k = x.shape[0], self.config.experts, self.config.top_k
        rows, h, f = t * k, self.hidden, self.inner
        ids, weights = buf(t, k, dtype=torch.int32), buf(t, k, dtype=torch.float32)
        moe.zc_route(logits, F32, t, e, None, self.config, ids, weights)
        offsets, position = buf(e + 1, dtype=torch.int32), buf(t, k, dtype=torch.int32)
        ws = buf(moe.zc_dispatch_workspace_bytes(t, k, e), dtype=torch.uint8)
        moe.zc_dispatch_plan(ids, t, k, e, ws, ws.numel(), offsets, position)
        payload = buf(rows, h)
        moe.zc_dispatch(x, t, h, h, position, k, payload, rows, h)
        arrived, self.compressed = self.exchange(payload, offsets)
        x8 = self.rows8(arrived)
        gu = self.product(x8, rows, self.w1.q, self.w1.s, 2 * f, h, offsets)
        fs = moe.zc_fp8_stride(f)
        h8 = buf(rows, fs, dtype=torch.uint8), buf(rows, moe.zc_fp8_scale_stride(f), dtype=torch.uint8)
        kept = buf(rows, 2 * fs, dtype=torch.uint8), buf(rows, moe.zc_fp8_scale_stride(2 * fs), dtype=torch.uint8)
        moe.zc_swiglu(gu, rows, f, 2 * f, None, 0, *h8, *kept)
        z = self.product(h8, rows, self.w2.q, self.w2.s, h, f, offsets)
        y = buf(t, h)
        moe.zc_combine(z, rows, h, h, position, weights, t, k, y, h)
        self.saved = logits, ids, weights, offsets, position, x8, h8, kept, z, t, rows
        return y

    def backward(self, dy):
        logits, ids, weights, offsets, position, x8, h8, kept, z, t, rows = self.saved
        e, k, h, f = self.config.experts, self.config.top_k, self.hidden, self.inner
        dz, dweights = buf(rows, h), buf(t, k, dtype=torch.float32)
        moe.zc_combine_backward(dy, h, z, rows, h, h, position, weights, t, k, dz, h, dweights)
        dlogits = buf(t, e, dtype=torch.float32)
        moe.zc_route_backward(logits, F32, t, e, self.config, ids, dweights, dlogits, e)
        dh = self.product(self.rows8(dz), rows, self.w2.qt, self.w2.st, f, h, offsets)
        dw2 = self.weight_gradient(dz, h8, rows, h, f, offsets)
        dgu = buf(rows, 2 * f)
        moe.zc_swiglu_backward(*kept, rows, f, dh, f, dgu, 2 * f)
        dpayload = self.product(self.rows8(dgu), rows, self.w1.qt, self.w1.st, h, 2 * f, offsets)
        dw1 = self.weight_gradient(dgu, x8, rows, 2 * f, h, offsets)
        dx = buf(t, h)
        moe.zc_combine(dpayload, rows, h, h, position, None, t, k, dx, h)
        return dx, dlogits, dw1, dw2


def reference(config, x, logits, w1, w2, dy):
    """The layer in 64 bits on the CPU, without 8-bit rounding, by automatic differentiation; softmax or sigmoid
    scores, no groups, renormalised weights."""
    x, logits, w1, w2 = (v.double().cpu().requires_grad_() for v in (x, logits, w1, w2))
    s = torch.sigmoid(logits) if config.score == moe.ZC_SCORE_SIGMOID else torch.softmax(logits, dim=1)
    ids = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :config.top_k]
    p = s.gather(1, ids)
    weights = p / p.sum(dim=1, keepdim=True) * config.scale
    f = w2.shape[2]
    y = torch.zeros(x.shape, dtype=torch.float64)
    for e in range(config.experts):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ w1[e].T
        h = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
        y = y.index_add(0, t, weights[t, k, None] * (h @ w2[e].T))
    y.backward(dy.double().cpu())
    return y.detach(), x.grad, logits.grad, w1.grad, w2.grad


def inputs(tokens, hidden, inner, experts, seed=0):
    """x, dy, logits, w1, w2 of a layer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    return (normal(tokens, hidden).bfloat16(), normal(tokens, hidden, scale=1e-3).bfloat16(), normal(tokens, experts),
            normal(experts, 2 * inner, hidden, scale=hidden ** -0.5).bfloat16(),
            normal(experts, hidden, inner, scale=inner ** -0.5).bfloat16())


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--destinations", type=int, default=8)
    a = ap.parse_args()
    x, dy, logits, w1, w2 = inputs(a.tokens, a.hidden, a.inner, a.experts)
    config = moe.route_config(a.experts, a.top_k, "sigmoid", scale=2.0)
    layer = Layer(config, w1, w2, a.destinations)
    y = layer.forward(x, logits)
    got = y, *layer.backward(dy)
    torch.cuda.synchronize()
    print("payload of %d rows x %d compressed to %.1f %%" % (a.tokens * a.top_k, a.hidden,
                                                             100 * layer.compressed / (2 * a.tokens * a.top_k * a.hidden)))
    for name, v, r in zip(("y", "dx", "dlogits", "dw1", "dw2"), got, reference(config, x, logits, w1, w2, dy)):
        print("%-8s off by %.4f of the layer without 8-bit rounding" % (name, float((v.double().cpu() - r).norm() / r.norm())))


if __name__ == "__main__":
    main()
