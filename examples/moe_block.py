"""A whole block of a residual stream around the mixture-of-experts layer, forward and backward.

The layer of examples/moe_layer.py with what stands around it:

  forward   norm before the block; the router's logits in 32 bits; routing, exchange through the codec, experts and
            weighted sum; a shared expert that every token passes, added in the epilogue of its second product; balance
            and z loss; norm of the block's output, its gate, and the residual sum
  backward  the same way back: gradients of the input, of both norms and the gate, of the shared expert, of the
            router (with the losses' share), and of the experts

    python examples/moe_block.py [--tokens 2048 --hidden 1024 --inner 512 --shared 512 --experts 32 --top-k 4]

Prints the losses, and how far the block's output and its gradients are from the same block in 64 bits without any
rounding: what 8-bit inputs of the experts cost, up to a tenth.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import moe_layer  # noqa: E402
from lossless_bf16_exponent_amd import zc_moe as moe  # noqa: E402
from moe_layer import BF16, F32, buf  # noqa: E402

EPS = 1e-6
NAMES = ("router", "w1", "w2", "s1", "b1", "s2", "before", "after", "gate")


class Block:
    """params: router experts x hidden; w1, w2 as in moe_layer.Layer; the shared expert's s1 shared x hidden, b1 (its
    bias, floats) and s2 hidden x shared; weights of the norms before and after, and the gate, hidden each; BF16 but b1."""

    def __init__(self, config, params, destinations, loss_weight=0.01, z_weight=0.001):
        self.p, self.config = params, config
        self.layer = moe_layer.Layer(config, params["w1"], params["w2"], destinations)
        self.experts, self.hidden = params["router"].shape
        self.shared = params["s1"].shape[0]
        self.into = moe.norm_config(before=moe.norm_params(moe.ZC_NORM_RMS, params["before"], eps=EPS))
        self.out_of = moe.norm_config(after=moe.norm_params(moe.ZC_NORM_RMS, params["after"], eps=EPS), gate=params["gate"])
        self.workspace = buf(moe.ZC_MATMUL_WORKSPACE_MAX, dtype=torch.uint8)
        self.dloss = torch.full((1,), loss_weight, device="cuda")
        self.dz_loss = torch.full((1,), z_weight, device="cuda")

    def room(self, n):
        if n > self.workspace.numel():
            self.workspace = buf(n, dtype=torch.uint8)
        return self.workspace, self.workspace.numel()

    def forward(self, x):
        """r, and the balance and z loss."""
        p, (t, h), e, s = self.p, x.shape, self.experts, self.shared
        y, logits = buf(t, h), buf(t, e, dtype=torch.float32)
        moe.zc_norm(x, BF16, t, h, h, None, 0, self.into, None, 0, y, h)
        moe.zc_matmul(y, t, h, p["router"], e, h, h, None, logits, F32, e, *self.room(0))
        routed = self.layer.forward(y, logits)
        pre, hs, z, r = buf(t, s), buf(t, s), buf(t, h), buf(t, h)
        moe.zc_matmul(y, t, h, p["s1"], s, h, h, moe.epilogue(p["b1"], moe.ZC_ACT_SILU, pre=pre, pre_stride=s), hs, BF16, s,
                      *self.room(0))
        moe.zc_matmul(hs, t, s, p["s2"], h, s, s, moe.epilogue(residual=routed, residual_stride=h), z, BF16, h, *self.room(0))
        ids = self.layer.saved[1]
        counts, used = buf(1, e, dtype=torch.int32), buf(1, dtype=torch.int32)
        loss, z_loss = buf(1, dtype=torch.float32), buf(1, dtype=torch.float32)
        moe.zc_balance(logits, F32, t, e, self.config, ids, None, 1, None,
                       *self.room(moe.zc_balance_workspace_bytes(t, e, 1)), counts, used, loss, z_loss)
        moe.zc_norm(x, BF16, t, h, h, z, h, self.out_of, r, h)
        self.saved = x, y, logits, pre, hs, z, r, counts, used
        return r, loss, z_loss

    def backward(self, dr):
        """Gradients of the input and of every parameter, the latter in 32 bits."""
        p, (x, y, logits, pre, hs, z, r, counts, used) = self.p, self.saved
        (t, h), e, s = x.shape, self.experts, self.shared
        f32 = torch.float32
        g = {n: buf(*p[n].shape, dtype=f32) for n in NAMES if n not in ("w1", "w2")}
        dx, dz = buf(t, h), buf(t, h)
        room = self.room(max(moe.zc_norm_backward_workspace_bytes(t, h), moe.zc_activation_backward_workspace_bytes(t, max(s, e))))
        moe.zc_norm_backward(r, BF16, t, h, h, z, h, self.out_of, dr, h, None, 0, dx, h, dz, h,
                             moe.norm_grads(weight_after=g["after"], gate=g["gate"]), *room)
        dy, dlogits, g["w1"], g["w2"] = self.layer.backward(dz)
        dhs, dpre = buf(t, s), buf(t, s)
        moe.zc_matmul_wgrad(dz, t, h, h, hs, s, s, None, F32, s, g["s2"], F32, s, *room)
        moe.zc_matmul_dgrad(dz, t, h, h, p["s2"], s, s, None, BF16, s, dhs, BF16, s, *room)
        moe.zc_activation_backward(dhs, BF16, t, s, s, pre, s, moe.ZC_ACT_SILU, 1.0, dpre, s, g["b1"], *room)
        moe.zc_matmul_wgrad(dpre, t, s, s, y, h, h, None, F32, h, g["s1"], F32, h, *room)
        moe.zc_matmul_dgrad(dpre, t, s, s, p["s1"], h, h, dy, BF16, h, dy, BF16, h, *room)  # added to the experts' share
        moe.zc_balance_backward(logits, F32, t, e, self.config, None, 1, None, counts, used, self.dloss, self.dz_loss,
                                dlogits, e, dlogits, e)
        dl = buf(t, e)  # the products read BF16
        moe.zc_activation_backward(dlogits, F32, t, e, e, None, 0, moe.ZC_ACT_NONE, 1.0, dl, e)
        moe.zc_matmul_wgrad(dl, t, e, e, y, h, h, None, F32, h, g["router"], F32, h, *room)
        moe.zc_matmul_dgrad(dl, t, e, e, p["router"], h, h, dy, BF16, h, dy, BF16, h, *room)
        moe.zc_norm_backward(x, BF16, t, h, h, None, 0, self.into, dx, h, dy, h, dx, h, None, 0,
                             moe.norm_grads(weight_before=g["before"]), *room)
        return dx, g


def reference(config, x, params, dr, loss_weight=0.01, z_weight=0.001):
    """The block in 64 bits on the CPU, without any rounding, by automatic differentiation: (r, loss, z loss, dx, gradients)."""
    x = x.double().cpu().requires_grad_()
    p = {n: v.double().cpu().requires_grad_() for n, v in params.items()}

    def rms(v, w):
        return v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w

    y = rms(x, p["before"])
    logits = y @ p["router"].T
    s = torch.sigmoid(logits) if config.score == moe.ZC_SCORE_SIGMOID else torch.softmax(logits, dim=1)
    ids = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :config.top_k]
    chosen = s.gather(1, ids)
    weights = chosen / chosen.sum(dim=1, keepdim=True) * config.scale
    f = p["w2"].shape[2]
    z = torch.nn.functional.silu(y @ p["s1"].T + p["b1"]) @ p["s2"].T
    for e in range(config.experts):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        gu = y[t] @ p["w1"][e].T
        hidden = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]
        z = z.index_add(0, t, weights[t, k, None] * (hidden @ p["w2"][e].T))
    r = x + p["gate"] * rms(z, p["after"])
    share = s / (s.sum(dim=1, keepdim=True) + 1e-20) if config.score == moe.ZC_SCORE_SIGMOID else s
    hits = torch.bincount(ids.reshape(-1), minlength=config.experts).double()
    loss = config.experts / config.top_k * (hits / len(x) * share.mean(dim=0)).sum()
    z_loss = (torch.logsumexp(logits, dim=1) ** 2).mean()
    ((r * dr.double().cpu()).sum() + loss_weight * loss + z_weight * z_loss).backward()
    return r.detach(), loss.detach(), z_loss.detach(), x.grad, {n: v.grad for n, v in p.items()}


def inputs(tokens, hidden, inner, shared, experts, seed=0):
    """x, dr and the parameters of a block."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale + mean

    params = dict(router=normal(experts, hidden, scale=hidden ** -0.5), w1=normal(experts, 2 * inner, hidden, scale=hidden ** -0.5),
                  w2=normal(experts, hidden, inner, scale=inner ** -0.5), s1=normal(shared, hidden, scale=hidden ** -0.5),
                  b1=normal(shared, scale=0.1), s2=normal(hidden, shared, scale=shared ** -0.5),
                  before=normal(hidden, scale=0.1, mean=1.0), after=normal(hidden, scale=0.1, mean=1.0),
                  gate=normal(hidden, scale=0.1, mean=0.3))
    params = {n: v if n == "b1" else v.bfloat16() for n, v in params.items()}
    return normal(tokens, hidden, scale=2.0).bfloat16(), normal(tokens, hidden, scale=1e-3).bfloat16(), params


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 2048), ("hidden", 1024), ("inner", 512), ("shared", 512), ("experts", 32), ("top-k", 4),
                        ("destinations", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    x, dr, params = inputs(a.tokens, a.hidden, a.inner, a.shared, a.experts)
    config = moe.route_config(a.experts, a.top_k, "sigmoid", scale=2.0)
    block = Block(config, params, a.destinations)
    r, loss, z_loss = block.forward(x)
    dx, g = block.backward(dr)
    torch.cuda.synchronize()
    want = reference(config, x, params, dr)
    print("balance loss %.5f (%.5f in 64 bits), z loss %.5f (%.5f)" % (float(loss), float(want[1]), float(z_loss), float(want[2])))
    branch = x.double().cpu()
    for name, v, w in (("branch", r.double().cpu() - branch, want[0] - branch), ("dx", dx, want[3]),
                       *((n, g[n], want[4][n]) for n in NAMES)):
        print("%-8s off by %.4f of the block without rounding" % (name, float((v.double().cpu() - w).norm() / w.norm())))


if __name__ == "__main__":
    main()
