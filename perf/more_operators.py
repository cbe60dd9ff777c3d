"""The operators of a whole block around the mixture-of-experts layer, from residual to residual: what is measured.

Three operators, each with its forward and backward direction:

  norm     norm of a block's output, its gate and scale, the residual sum, and the norm before the next block
  product  BF16 matrix product with bias, activation and residual in its epilogue, and the gradients of its operands
  balance  copies per expert, the balance loss and the z loss of every sequence, and the logits' gradient

Sizes are those of the all-to-all payload (8192 tokens, 8 of 256 experts, hidden 7168) and of the 4096 x 14336 shard, and
generic ones beside them.

What a call stores in BF16 for a later one has that rounding in its definition: the sum r and the pre-activation, at
which gradients are evaluated, and the gradient of the pre-activation, which the products of the backward pass read.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, step, rows, cols, after, before, gate=False, row_gate=False, bias=False, stream="bfloat16",
          params="bfloat16", scale=1.0):
    return {"name": name, "op": "norm", "step": step, "rows": rows, "cols": cols, "after": after, "before": before,
            "gate": gate, "row_gate": row_gate, "bias": bias, "stream": stream, "params": params, "scale": scale}


def _product(name, step, m, n, k, act="none", bias=False, residual=False, out="bfloat16"):
    return {"name": name, "op": "product", "step": step, "m": m, "n": n, "k": k, "act": act, "bias": bias,
            "residual": residual, "out": out}


def _balance(name, step, tokens, experts, top_k, score, sequences=1, mask=False, z=True, dtype="float32"):
    return {"name": name, "op": "balance", "step": step, "tokens": tokens, "experts": experts, "top_k": top_k,
            "score": score, "sequences": sequences, "mask": mask, "z": z, "dtype": dtype}


def listed():
    return [
        # one token of a serving step: residual sum and the norm before the next block
        _norm("norm-decode", "forward", 1, 7168, "none", "rms"),
        # a training batch with norms on both sides of the block and a gate a channel
        _norm("norm-batch", "forward", 8192, 7168, "rms", "rms", gate=True, scale=0.5),
        # and its backward pass: gradients of the residual, the block's output, the gate and both weights
        _norm("norm-train", "backward", 8192, 7168, "rms", "rms", gate=True, scale=0.5),
        # layer norms with biases and a gate a token, a residual in 32 bits, rows of an odd length
        _norm("norm-odd", "backward", 2049, 5125, "layer", "layer", row_gate=True, bias=True, stream="float32",
              params="float32"),
        # one token of a serving step through a dense layer
        _product("product-decode", "forward", 1, 4096, 14336, bias=True, residual=True),
        # a batch of decoding sequences through a dense layer
        _product("product-few", "forward", 48, 14336, 4096, "silu", bias=True),
        # the router's logits of the all-to-all's batch, in 32 bits
        _product("product-router", "forward", 8192, 256, 7168, bias=True, out="float32"),
        # no size is a multiple of anything
        _product("product-odd", "forward", 1021, 4099, 7173, "gelu_tanh", bias=True, residual=True),
        # the backward pass of a dense layer with an activation: gradients of pre-activation, bias, input and weights
        _product("product-train", "backward", 8192, 4096, 7168, "silu", bias=True, residual=True),
        # a few tokens of a router: losses, counts and the gradient; only latency counts
        _balance("balance-small", "train", 48, 8, 2, "softmax"),
        # the all-to-all's batch
        _balance("balance-batch", "train", 8192, 256, 8, "sigmoid"),
        # packed sequences of uneven lengths with padding
        _balance("balance-packed", "train", 65536, 160, 6, "softmax", sequences=37, mask=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "product", "balance"))
    if op == "norm":
        cols = _log(rng, 64, 8192)
        after, before = rng.choice((("none", "rms"), ("rms", "rms"), ("rms", "none"), ("layer", "layer"), ("none", "layer")))
        c = _norm("", rng.choice(("forward", "backward")), _log(rng, 1, 8192), cols if rng.random() < 0.4 else (cols + 7) // 8 * 8,
                  after, before, rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.3,
                  rng.choice(("bfloat16", "bfloat16", "float32")), rng.choice(("bfloat16", "float32")),
                  rng.choice((1.0, 0.5)))
    elif op == "product":
        step = rng.choice(("forward", "forward", "backward"))
        n, k = _log(rng, 64, 14336), _log(rng, 64, 14336)
        if rng.random() < 0.6:
            n, k = (n + 63) // 64 * 64, (k + 63) // 64 * 64
        m = _log(rng, 1, min(16384, 8192 * 4096 * 7168 // (n * k)))
        act = rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"))
        # the weights' gradient leaves in 32 bits where its operand has no rounding of its own
        c = _product("", step, m, n, k, act, rng.random() < 0.5, rng.random() < 0.5,
                     rng.choice(("bfloat16", "float32")) if act == "none" else "bfloat16")
    else:
        experts = _log(rng, 8, 256)
        sequences = rng.choice((1, 1, 4, 37))
        c = _balance("", rng.choice(("forward", "train", "train")), _log(rng, max(16, sequences), 65536), experts,
                     rng.randint(1, 8), rng.choice(("softmax", "sigmoid")), sequences, rng.random() < 0.4,
                     rng.random() < 0.6, rng.choice(("float32", "float32", "bfloat16")))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _bounds(seed, tokens, sequences):
    """Uneven sequences, each of one token at least; a few tokens behind the last belong to none where there is room."""
    r = np.random.default_rng([seed, 5])
    if sequences == 1:
        return [0, tokens]
    w = r.exponential(size=sequences)
    spare = min(64, (tokens - sequences) // 8)
    counts = 1 + r.multinomial(tokens - sequences - spare, w / w.sum())
    return [0, *(int(v) for v in np.cumsum(counts))]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).add_(mean)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    bf, f32 = torch.bfloat16, torch.float32
    st = {"case": case}
    if case["op"] == "norm":
        t, h = case["rows"], case["cols"]
        rt, pt = getattr(torch, case["stream"]), getattr(torch, case["params"])
        # a residual stream some blocks in: larger than one block's output
        st["x"] = normal(t, h, scale=3.0, mean=0.1).to(rt)
        st["z"] = normal(t, h, scale=1.5, mean=-0.1).to(bf)
        for name, on, mean in (("w1", case["after"] != "none", 1.0), ("w2", case["before"] != "none", 1.0),
                               ("b1", case["after"] != "none" and case["bias"], 0.0),
                               ("b2", case["before"] != "none" and case["bias"], 0.0), ("gate", case["gate"], 0.3)):
            st[name] = normal(h, scale=0.1, mean=mean).to(pt) if on else None
        st["row_gate"] = torch.sigmoid(normal(t)) if case["row_gate"] else None
        if case["step"] == "forward":
            st["r"] = empty(t, h, dtype=rt)
            st["y"] = empty(t, h) if case["before"] != "none" else None
        else:
            # x holds the stored sum here, which the forward pass wrote
            st["dr"] = normal(t, h, scale=1e-3).to(rt)
            st["dy"] = normal(t, h, scale=1e-3).to(bf) if case["before"] != "none" else None
            st["dx"], st["dz"] = empty(t, h, dtype=rt), empty(t, h)
            for name in ("w1", "b1", "gate", "w2", "b2"):
                st["d" + name] = None if st[name] is None else empty(h, dtype=f32)
            st["drow_gate"] = empty(t, dtype=f32) if case["row_gate"] else None
            st["workspace"] = empty(128 << 20, dtype=torch.uint8)
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        ot = getattr(torch, case["out"])
        st["a"] = normal(m, k).to(bf)
        st["w"] = normal(n, k, scale=k ** -0.5).to(bf)
        st["bias"] = normal(n, scale=0.1) if case["bias"] else None
        st["workspace"] = empty(64 << 20, dtype=torch.uint8)
        if case["step"] == "forward":
            st["residual"] = normal(m, n).to(ot) if case["residual"] else None
            st["out"] = empty(m, n, dtype=ot)
        else:
            st["dout"] = normal(m, n, scale=1e-3).to(bf)
            # the pre-activation that the forward pass kept, and the gradient that another path left at the input
            st["pre"] = normal(m, n).to(bf) if case["act"] != "none" else None
            st["add"] = normal(m, k, scale=1e-3).to(bf) if case["residual"] else None
            st["dpre"] = empty(m, n)
            st["dx"], st["dw"] = empty(m, k), empty(n, k, dtype=ot)
            st["dbias"] = empty(n, dtype=f32) if case["bias"] else None
    else:
        t, e, k, s = case["tokens"], case["experts"], case["top_k"], case["sequences"]
        k = min(k, e)
        st["logits"] = normal(t, e).add_(normal(e, scale=0.5)).to(getattr(torch, case["dtype"]))
        st["bounds"] = _bounds(seed, t, s)
        st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device="cuda")
        # the router's choice; tokens that are padding have no experts
        st["ids"] = st["logits"].float().topk(k, dim=1).indices.int().contiguous()
        st["mask"] = None
        if case["mask"]:
            st["mask"] = (torch.rand(t, generator=gen, device="cuda") < 0.9).to(torch.uint8)
            st["ids"][st["mask"] == 0] = -1
        st["counts"], st["used"] = empty(s, e, dtype=torch.int32), empty(s, dtype=torch.int32)
        st["loss"], st["zloss"] = empty(s, dtype=f32), empty(s, dtype=f32) if case["z"] else None
        # weights of the losses in the whole
        st["dloss"], st["dzloss"] = normal(s, scale=1e-3, mean=1e-2), normal(s, scale=1e-4, mean=1e-3) if case["z"] else None
        # the gradient that the routing weights leave, to which the losses' is added
        st["dlogits0"] = normal(t, e, scale=1e-3 / t).to(getattr(torch, case["dtype"]))
        st["dlogits"] = torch.empty_like(st["dlogits0"])
        st["workspace"] = empty(64 << 20, dtype=torch.uint8)
    return st


# ---------------------------------------------------------------------------
# plain forms: elementary operations in 32 bits
# ---------------------------------------------------------------------------

def _normed(v, kind):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    rs = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    return v * rs, rs


def _affine(v, w, b):
    v = v if w is None else v * w.float()
    return v if b is None else v + b.float()


def _norm_slope(xhat, rs, d, kind):
    """The gradient at a norm's input from that at its normed value."""
    g = d - xhat * (d * xhat).mean(dim=1, keepdim=True)
    if kind == "layer":
        g = g - d.mean(dim=1, keepdim=True)
    return g * rs


def _plain_norm(st):
    c = st["case"]
    z = st["z"].float()
    zhat, zrs = _normed(z, c["after"]) if c["after"] != "none" else (z, None)
    h = _affine(zhat, st["w1"], st["b1"])
    weight = torch.full((1, 1), c["scale"], device=z.device)
    if st["gate"] is not None:
        weight = weight * st["gate"].float()[None, :]
    if st["row_gate"] is not None:
        weight = weight * st["row_gate"][:, None]
    if c["step"] == "forward":
        r = st["x"].float() + weight * h
        out = {"r": r.to(st["x"].dtype)}
        if c["before"] != "none":
            out["y"] = _affine(_normed(r, c["before"])[0], st["w2"], st["b2"]).bfloat16()
        return out
    out = {}
    total = st["dr"].float()
    if c["before"] != "none":
        dy = st["dy"].float()
        rhat, rrs = _normed(st["x"].float(), c["before"])
        out["dw2"] = (dy * rhat).sum(dim=0)
        if st["b2"] is not None:
            out["db2"] = dy.sum(dim=0)
        total = total + _norm_slope(rhat, rrs, dy * st["w2"].float(), c["before"])
    dh = total * weight
    out["dx"] = total.to(st["x"].dtype)
    if st["gate"] is not None:
        rows = c["scale"] if st["row_gate"] is None else c["scale"] * st["row_gate"][:, None]
        out["dgate"] = (total * h * rows).sum(dim=0)
    if st["row_gate"] is not None:
        cols = c["scale"] if st["gate"] is None else c["scale"] * st["gate"].float()[None, :]
        out["drow_gate"] = (total * h * cols).sum(dim=1)
    if c["after"] != "none":
        out["dw1"] = (dh * zhat).sum(dim=0)
        if st["b1"] is not None:
            out["db1"] = dh.sum(dim=0)
        out["dz"] = _norm_slope(zhat, zrs, dh * st["w1"].float(), c["after"]).bfloat16()
    else:
        out["dz"] = dh.bfloat16()
    return out


_R2 = math.sqrt(0.5)
_T0, _T1 = math.sqrt(2 / math.pi), 0.044715


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * _R2))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(_T0 * (v + _T1 * v * v * v)))
    return torch.sigmoid(v) if act == "sigmoid" else v


def _act_slope(v, act):
    if act == "relu":
        return (v > 0).float()
    if act == "silu":
        s = torch.sigmoid(v)
        return s * (1 + v * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * _R2)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_T0 * (v + _T1 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * _T0 * (1 + 3 * _T1 * v * v)
    s = torch.sigmoid(v)
    return s * (1 - s)


def _plain_product(st):
    c = st["case"]
    if c["step"] == "forward":
        v = st["a"].float() @ st["w"].float().t()
        if st["bias"] is not None:
            v = v + st["bias"]
        v = _act(v, c["act"])
        if st["residual"] is not None:
            v = v + st["residual"].float()
        return {"out": v.to(st["out"].dtype)}
    d = st["dout"].float()
    if c["act"] != "none":
        d = d * _act_slope(st["pre"].float(), c["act"])
    out = {"dpre": d.bfloat16()}
    if st["bias"] is not None:
        out["dbias"] = d.sum(dim=0)
    d = out["dpre"].float()
    dx = d @ st["w"].float()
    out["dx"] = (dx if st["add"] is None else dx + st["add"].float()).bfloat16()
    out["dw"] = (d.t() @ st["a"].float()).to(st["dw"].dtype)
    return out


def _plain_balance(st):
    c = st["case"]
    e, k, s = c["experts"], st["ids"].shape[1], c["sequences"]
    b = st["bounds"]
    x = st["logits"].float()
    seq = torch.zeros(x.shape[0], dtype=torch.long, device=x.device)
    for i in range(s):
        seq[b[i]:b[i + 1]] = i
    on = torch.arange(x.shape[0], device=x.device) < b[s]
    part = on if st["mask"] is None else on & (st["mask"] != 0)
    live = part.float()[:, None]
    ids = torch.where(part[:, None] & (st["ids"] >= 0), st["ids"], e).long()
    hits = torch.zeros(s, e + 1, device=x.device).index_put_((seq[:, None].expand_as(ids), ids), torch.ones_like(ids, dtype=torch.float32),
                                                             accumulate=True)[:, :e]
    used = torch.zeros(s, device=x.device).index_add_(0, seq, part.float())
    sg = torch.sigmoid(x)
    soft = torch.softmax(x, dim=1)
    p = soft if c["score"] == "softmax" else sg / (sg.sum(dim=1, keepdim=True) + 1e-20)
    n = used.clamp(min=1)
    f = hits * (e / (k * n))[:, None]
    mean = torch.zeros(s, e, device=x.device).index_add_(0, seq, p * live) / n[:, None]
    out = {"counts": hits.int(), "used": used.int(), "loss": (f * mean).sum(dim=1)}
    lse = torch.logsumexp(x, dim=1)
    if c["z"]:
        out["zloss"] = torch.zeros(s, device=x.device).index_add_(0, seq, lse * lse * live[:, 0]) / n
    if c["step"] == "train":
        ft = f[seq]
        d = p * (ft - (ft * p).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * torch.sigmoid(-x)
        d = d * (st["dloss"] / n)[seq][:, None]
        if c["z"]:
            d = d + soft * (2 * lse * (st["dzloss"] / n)[seq])[:, None]
        out["dlogits"] = (st["dlogits0"].float() + d * live).to(st["dlogits"].dtype)
    return out


# ---------------------------------------------------------------------------
# the calls a user makes
# ---------------------------------------------------------------------------

def _own_norm(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    t, h = c["rows"], c["cols"]
    kind = {"none": zc.ZC_NORM_NONE, "rms": zc.ZC_NORM_RMS, "layer": zc.ZC_NORM_LAYER}
    stream = zc.ZC_F32 if c["stream"] == "float32" else zc.ZC_BF16
    cfg = zc.norm_config(zc.norm_params(kind[c["after"]], st["w1"], st["b1"], EPS),
                         zc.norm_params(kind[c["before"]], st["w2"], st["b2"], EPS), st["gate"], st["row_gate"], c["scale"])
    if c["step"] == "forward":
        zc.zc_norm(st["x"], stream, t, h, h, st["z"], h, cfg, st["r"], h, st["y"], h, None, None)
        return {"r": st["r"]} if st["y"] is None else {"r": st["r"], "y": st["y"]}
    grads = zc.norm_grads(st["dw1"], st["db1"], st["dgate"], st["dw2"], st["db2"], st["drow_gate"])
    zc.zc_norm_backward(st["x"], stream, t, h, h, st["z"], h, cfg, st["dr"], h, st["dy"], h, st["dx"], h, st["dz"], h, grads,
                        st["workspace"], st["workspace"].numel())
    names = ("dw2", "db2", "dx", "dgate", "drow_gate", "dw1", "db1", "dz")
    return {name: st[name] for name in names if st[name] is not None}


def _own_product(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    m, n, k = c["m"], c["n"], c["k"]
    ws, room = st["workspace"], st["workspace"].numel()
    act = getattr(zc, "ZC_ACT_" + c["act"].upper())
    kind = zc.ZC_F32 if c["out"] == "float32" else zc.ZC_BF16
    if c["step"] == "forward":
        epilogue = zc.epilogue(bias=st["bias"], activation=act, residual=st["residual"], residual_stride=n)
        zc.zc_matmul(st["a"], m, k, st["w"], n, k, k, epilogue, st["out"], kind, n, ws, room)
        return {"out": st["out"]}
    zc.zc_activation_backward(st["dout"], zc.ZC_BF16, m, n, n, st["pre"], n, act, 1.0, st["dpre"], n, st["dbias"], ws, room)
    zc.zc_matmul_dgrad(st["dpre"], m, n, n, st["w"], k, k, st["add"], zc.ZC_BF16, k, st["dx"], zc.ZC_BF16, k, ws, room)
    zc.zc_matmul_wgrad(st["dpre"], m, n, n, st["a"], k, k, None, kind, k, st["dw"], kind, k, ws, room)
    out = {"dpre": st["dpre"], "dx": st["dx"], "dw": st["dw"]}
    return out if st["dbias"] is None else out | {"dbias": st["dbias"]}


def _own_balance(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    t, e, s = c["tokens"], c["experts"], c["sequences"]
    cfg = zc.route_config(e, st["ids"].shape[1], c["score"])
    kind = zc.ZC_BF16 if c["dtype"] == "bfloat16" else zc.ZC_F32
    zc.zc_balance(st["logits"], kind, t, e, cfg, st["ids"], st["mask"], s, st["offsets"], st["workspace"],
                  st["workspace"].numel(), st["counts"], st["used"], st["loss"], st["zloss"])
    out = {"counts": st["counts"], "used": st["used"], "loss": st["loss"]}
    if c["z"]:
        out["zloss"] = st["zloss"]
    if c["step"] == "train":
        zc.zc_balance_backward(st["logits"], kind, t, e, cfg, st["mask"], s, st["offsets"], st["counts"], st["used"],
                               st["dloss"], st["dzloss"], st["dlogits0"], e, st["dlogits"], e)
        out["dlogits"] = st["dlogits"]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "product": _own_product, "balance": _own_balance}[op](state)
    return {"norm": _plain_norm, "product": _plain_product, "balance": _plain_balance}[op](state)


def work(case):
    if case["op"] == "norm":
        t, h = case["rows"], case["cols"]
        r = 4 if case["stream"] == "float32" else 2
        if case["step"] == "forward":
            return {"bytes": t * h * (2 * r + 2 + (2 if case["before"] != "none" else 0)), "flops": 12 * t * h}
        return {"bytes": t * h * (3 * r + 4 + (2 if case["before"] != "none" else 0)), "flops": 30 * t * h}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        o = 4 if case["out"] == "float32" else 2
        if case["step"] == "forward":
            return {"bytes": 2 * m * k + 2 * n * k + m * n * o * (2 if case["residual"] else 1), "flops": 2 * m * n * k}
        pre = 2 if case["act"] != "none" else 0
        return {"bytes": m * n * (4 + pre) + 2 * n * k + 2 * m * k * (3 if case["residual"] else 2) + n * k * o,
                "flops": 4 * m * n * k}
    t, e, k, s = case["tokens"], case["experts"], case["top_k"], case["sequences"]
    size = 2 if case["dtype"] == "bfloat16" else 4
    b = t * e * size + 4 * t * k + 4 * s * e + (t if case["mask"] else 0)
    return {"bytes": b + (2 * t * e * size if case["step"] == "train" else 0),
            "flops": t * e * (20 if case["step"] == "train" else 10)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------

def _d(v):
    return None if v is None else v.double()


def _stats(v, kind):
    """Mean taken off and 1 / deviation of every row."""
    mu = v.sum(dim=1, keepdim=True) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, :1])
    var = ((v - mu) ** 2).sum(dim=1, keepdim=True) / v.shape[1]
    return mu, (var + EPS) ** -0.5


def _exact_norm(case, st):
    n = case["cols"]
    one = torch.ones(1, n, dtype=torch.float64, device="cuda")
    x, z, w1, b1, w2, b2, gate, rg = (_d(st[k]) for k in ("x", "z", "w1", "b1", "w2", "b2", "gate", "row_gate"))
    coef = case["scale"] * (one if gate is None else gate[None]) * (1 if rg is None else rg[:, None])
    if case["after"] == "none":
        h, u = z, z
    else:
        mu1, s1 = _stats(z, case["after"])
        u = (z - mu1) * s1
        h = u * w1 + (0 if b1 is None else b1)
    if case["step"] == "forward":
        r = x + coef * h
        if case["before"] == "none":
            return {"r": r}
        mu, s = _stats(r, case["before"])
        return {"r": r, "y": (r - mu) * s * w2 + (0 if b2 is None else b2)}
    out = {}
    g = _d(st["dr"])
    if case["before"] != "none":
        dy = _d(st["dy"])
        mu, s = _stats(x, case["before"])
        v = (x - mu) * s
        out["dw2"] = (v * dy).sum(dim=0)
        if b2 is not None:
            out["db2"] = dy.sum(dim=0)
        dv = dy * w2
        # through s: ds = -s^3 / n * (x - mu); through the mean: the sum of what arrives at x - mu
        back = s * dv - s * v * (dv * v).sum(dim=1, keepdim=True) / n
        if case["before"] == "layer":
            back = back - back.sum(dim=1, keepdim=True) / n
        g = g + back
    out["dx"] = g
    dh = g * coef
    if gate is not None:
        out["dgate"] = (g * h * (1 if rg is None else rg[:, None])).sum(dim=0) * case["scale"]
    if rg is not None:
        out["drow_gate"] = (g * h * (one if gate is None else gate[None])).sum(dim=1) * case["scale"]
    if case["after"] != "none":
        out["dw1"] = (dh * u).sum(dim=0)
        if b1 is not None:
            out["db1"] = dh.sum(dim=0)
        du = dh * w1
        back = s1 * du - s1 * u * (du * u).sum(dim=1, keepdim=True) / n
        if case["after"] == "layer":
            back = back - back.sum(dim=1, keepdim=True) / n
        out["dz"] = back
    else:
        out["dz"] = dh
    return out


def _activation(v, act):
    """Value and slope in 64 bits."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.where(v > 0, v, 0.0), torch.where(v > 0, 1.0, 0.0).double()
    if act in ("silu", "sigmoid"):
        s = 1 / (1 + torch.exp(-v))
        ds = torch.exp(-v) * s * s
        return (s, ds) if act == "sigmoid" else (v * s, s + v * ds)
    if act == "gelu":
        # the standard normal distribution and its density
        cdf = 0.5 * torch.erfc(-v / math.sqrt(2.0))
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh u) / 2 = 1 / (1 + e^-2u)
    c = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-c * (v + 0.044715 * v ** 3)))
    return v * s, s + v * s * (1 - s) * c * (1 + 3 * 0.044715 * v ** 2)


def _exact_product(case, st):
    a, w = _d(st["a"]), _d(st["w"])
    if case["step"] == "forward":
        v = torch.mm(a, w.t().contiguous())
        v = _activation(v if st["bias"] is None else v + _d(st["bias"])[None], case["act"])[0]
        return {"out": v if st["residual"] is None else v + _d(st["residual"])}
    d = _d(st["dout"])
    if case["act"] != "none":
        d = d * _activation(_d(st["pre"]), case["act"])[1]
    stored = d.bfloat16().double()
    dx = torch.mm(stored, w)
    out = {"dpre": d, "dx": dx if st["add"] is None else dx + _d(st["add"]), "dw": torch.mm(stored.t().contiguous(), a)}
    if st["bias"] is not None:
        out["dbias"] = d.sum(dim=0)
    return out


def _exact_balance(case, st):
    e, k, s = case["experts"], st["ids"].shape[1], case["sequences"]
    x, ids = _d(st["logits"]), st["ids"].cpu().numpy()
    t = x.shape[0]
    on = np.ones(t, dtype=bool) if st["mask"] is None else st["mask"].cpu().numpy() != 0
    out = {"counts": np.zeros((s, e), dtype=np.int32), "used": np.zeros(s, dtype=np.int32), "loss": np.zeros(s)}
    if case["z"]:
        out["zloss"] = np.zeros(s)
    grad = _d(st["dlogits0"]).clone()
    for i in range(s):
        rows = np.arange(st["bounds"][i], st["bounds"][i + 1])
        rows = rows[on[rows]]
        if not rows.size:
            continue
        mine = ids[rows].reshape(-1)
        out["counts"][i] = np.bincount(mine[(mine >= 0) & (mine < e)], minlength=e)
        out["used"][i] = rows.size
        at = torch.from_numpy(rows).cuda()
        v = x[at]
        top = v.max(dim=1, keepdim=True).values
        z = top + torch.log(torch.exp(v - top).sum(dim=1, keepdim=True))
        soft = torch.exp(v - z)
        sig = 1 / (1 + torch.exp(-v))
        p = soft if case["score"] == "softmax" else sig / (sig.sum(dim=1, keepdim=True) + 1e-20)
        f = torch.from_numpy(out["counts"][i]).cuda().double() * e / (k * rows.size)
        out["loss"][i] = float((p.sum(dim=0) / rows.size * f).sum())
        if case["z"]:
            out["zloss"][i] = float((z * z).sum() / rows.size)
        if case["step"] == "train":
            own_share = p * f - p * (p @ f)[:, None]
            if case["score"] == "sigmoid":
                own_share = own_share / (1 + torch.exp(v))
            g = own_share * float(st["dloss"][i]) / rows.size
            if case["z"]:
                g = g + soft * z * (2 * float(st["dzloss"][i]) / rows.size)
            grad[at] += g
    if case["step"] == "train":
        out["dlogits"] = grad
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "product": _exact_product, "balance": _exact_balance}[case["op"]](case, st)
