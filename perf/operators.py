"""The operators of a mixture-of-experts layer around the compressed all-to-all: what is measured.

Four operators, each with its forward and backward direction:

  route    scores of the experts, groups, top-k and weights of every token
  exchange the order of the token copies by expert, the payload in that order, and the weighted sum back
  product  8-bit floating-point product with a scale for each block of 128, per expert
  gate     gated activation that keeps its input in 8 bits for the backward pass

Sizes are those of the all-to-all payload (8192 tokens, 8 of 256 experts, hidden 7168, 8 destinations with 32 experts
each) and of the 4096 x 14336 shard, and generic ones beside them.

An 8-bit block holds 128 values (or 128 x 128) and one scale 2^(b - 127), b an 8-bit number: the smallest power of two
at which the largest magnitude of the block is at most the largest of the 8-bit type (448 for e4m3, 57344 for e5m2).
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}  # the largest value of either type is 1.75 * 2^TOP


def _up(v, m):
    return (v + m - 1) // m * m


def _scaled(x, e):
    """x * 2^e exactly (e: whole numbers of any shape that spreads over x)."""
    return x * ((e.long() + 1023) << 52).view(torch.float64).float()


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _route(name, tokens, experts, top_k, score, groups=1, group_top=1, group_score=1, bias=False, renorm=True, scale=1.0,
           dtype="float32", train=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score,
            "groups": groups, "group_top": group_top, "group_score": group_score, "bias": bias, "renorm": renorm,
            "scale": scale, "dtype": dtype, "train": train}


def _exchange(name, step, tokens, top_k, experts, hidden):
    return {"name": name, "op": "exchange", "step": step, "tokens": tokens, "top_k": top_k, "experts": experts,
            "hidden": hidden}


def _product(name, step, rows, groups, n, k, skew, grad="e4m3"):
    return {"name": name, "op": "product", "step": step, "rows": rows, "groups": groups, "n": n, "k": k, "skew": skew,
            "grad": grad}


def _gate(name, rows, cols, train):
    return {"name": name, "op": "gate", "rows": rows, "cols": cols, "train": train}


def listed():
    return [
        # one token of a serving step: only latency counts
        _route("route-decode", 1, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
        # the all-to-all's batch: sigmoid scores, balance bias, 4 of 8 groups
        _route("route-batch", 8192, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
        # a training step of a layer with softmax scores and a ragged batch: ids, weights and the logits' gradient
        _route("route-train", 8191, 128, 8, "softmax", train=True),
        # the payload of the all-to-all, from the router's ids
        _exchange("dispatch-batch", "dispatch", 8192, 8, 256, 7168),
        # the weighted sum of a few tokens of a serving step
        _exchange("combine-decode", "combine", 16, 8, 256, 7168),
        # the weighted sum and its gradients in a training step
        _exchange("combine-train", "combine_train", 8192, 8, 256, 7168),
        # one token's eight experts: every row meets another expert's weights
        _product("product-decode", "forward", 8, 8, 4096, 7168, 0.0),
        # what one destination's 32 experts receive from 8 peers, with the payload's uneven loads
        _product("product-batch", "forward", 65536, 32, 4096, 7168, 1.2),
        # a dense layer at odd sizes: no size is a multiple of the block
        _product("product-odd", "forward", 1537, 1, 4100, 14344, 0.0),
        # the backward pass of an expert layer: gradients of its input and of its weights
        _product("product-train", "backward", 8192, 8, 4096, 7168, 1.2),
        # the experts' activation in a serving step
        _gate("gate-decode", 8, 2048, False),
        # the experts' activation in a training step, kept in 8 bits between its two passes
        _gate("gate-train", 65536, 2048, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "exchange", "product", "gate"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        group_top = rng.randint((groups + 1) // 2, groups)
        top_k = rng.randint(1, min(8, group_top * (experts // groups)))
        c = _route("", _log(rng, 1, 8192), experts, top_k, rng.choice(("softmax", "sigmoid")), groups, group_top,
                   rng.choice((1, 2)), rng.random() < 0.5, rng.random() < 0.7, rng.choice((1.0, 2.5)),
                   rng.choice(("float32", "bfloat16")), rng.random() < 0.5)
    elif op == "exchange":
        experts = _log(rng, 8, 256)
        top_k = rng.randint(1, 8)
        hidden = _log(rng, 512, 7168)
        c = _exchange("", rng.choice(("dispatch", "combine", "combine_train")), _log(rng, 1, 8192), top_k, experts,
                      hidden if rng.random() < 0.3 else _up(hidden, 8))
    elif op == "product":
        step = rng.choice(("forward", "forward", "backward"))
        n, k = _log(rng, 512, 8192), _log(rng, 512, 8192)
        if rng.random() < 0.6:
            n, k = _up(n, 128), _up(k, 128)
        groups = rng.choice((1, 1, 2, 8, 32))
        c = _product("", step, _log(rng, 1, 16384), groups, n, k, rng.choice((0.0, 1.2)), rng.choice(("e4m3", "e5m2")))
    else:
        cols = _log(rng, 512, 8192)
        c = _gate("", _log(rng, 1, 16384), cols if rng.random() < 0.4 else _up(cols, 128), rng.random() < 0.6)
    del c["name"]
    return {key: (v + 1 if key in ("n", "k", "cols", "hidden") and v == 3072 else v) for key, v in c.items()}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _loads(seed, rows, groups, skew):
    """Rows of each group: one at least for as many groups as there are rows, the others by popularity rank^-skew."""
    r = np.random.default_rng([seed, 77])
    w = (r.permutation(groups) + 1.0) ** -skew
    least = np.zeros(groups, dtype=np.int64)
    least[r.permutation(groups)[:rows]] = 1
    return least + r.multinomial(rows - int(least.sum()), w / w.sum())


def _quantised_weights(groups, n, k, gen):
    """e4m3 weights with a scale for each block of 128 x 128, and the same transposed: what a program keeps of a layer."""
    np_, kp = _up(n, BLOCK), _up(k, BLOCK)
    q = torch.zeros(groups, np_, kp, dtype=F8["e4m3"], device="cuda")
    s = torch.zeros(groups, np_ // BLOCK, _up(kp // BLOCK, 4), dtype=torch.uint8, device="cuda")
    for g in range(groups):
        w = torch.zeros(np_, kp, device="cuda")
        w[:n, :k] = (torch.randn(n, k, generator=gen, device="cuda") * 0.02).bfloat16()
        t = w.view(np_ // BLOCK, BLOCK, kp // BLOCK, BLOCK)
        m, e = torch.frexp(t.abs().amax(dim=(1, 3)))
        b = torch.where(m > 0, e + 126 - TOP["e4m3"] + (m > 0.875).int(), 0).clamp(min=0)
        q[g] = _scaled(t, (127 - b)[:, None, :, None]).reshape(np_, kp).to(F8["e4m3"])
        s[g, :, :kp // BLOCK] = b.to(torch.uint8)
    qt = torch.empty(groups, kp, np_, dtype=F8["e4m3"], device="cuda")
    qt.view(torch.uint8).copy_(q.view(torch.uint8).transpose(1, 2))
    st = torch.zeros(groups, kp // BLOCK, _up(np_ // BLOCK, 4), dtype=torch.uint8, device="cuda")
    st[:, :, :np_ // BLOCK] = s[:, :, :kp // BLOCK].transpose(1, 2)
    # rows past n are left out: a layer of n outputs has n rows
    return (q[:, :n].contiguous(), s), (qt[:, :k].contiguous(), st)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    st = {"case": case}
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        dt = getattr(torch, case["dtype"])
        st["logits"] = normal(t, e).to(dt)
        st["bias"] = normal(e, scale=0.05) if case["bias"] else None
        st["dweights"] = normal(t, k)
        st["ids"], st["weights"] = empty(t, k, dtype=torch.int32), empty(t, k, dtype=torch.float32)
        st["dlogits"] = empty(t, e, dtype=dt)
    elif case["op"] == "exchange":
        t, k, e, h = case["tokens"], case["top_k"], case["experts"], case["hidden"]
        # distinct experts of every token, popular ones more often: the k largest of noise plus log popularity
        w = torch.from_numpy(np.log((np.random.default_rng([seed, 3]).permutation(e) + 1.0) ** -0.6)).to("cuda")
        noise = -torch.log(-torch.log(torch.rand(t, e, generator=gen, device="cuda").clamp(1e-20, 1 - 1e-7)))
        st["ids"] = (noise + w).topk(min(k, e), dim=1).indices.int().contiguous()
        rows = t * k
        order = torch.sort(st["ids"].reshape(-1).long(), stable=True).indices
        st["position"] = torch.empty_like(order)
        st["position"][order] = torch.arange(rows, device="cuda")
        st["position"] = st["position"].int().view(t, k)
        st["weights"] = torch.softmax(normal(t, k), dim=1)
        st["offsets"] = empty(e + 1, dtype=torch.int32)
        st["plan_position"], st["plan_source"] = empty(t, k, dtype=torch.int32), empty(rows, dtype=torch.int32)
        if case["step"] == "dispatch":
            st["x"] = normal(t, h).bfloat16()
            st["out"] = empty(rows, h, dtype=torch.bfloat16)
            st["workspace"] = empty(16 * rows + (4 << 20), dtype=torch.uint8)
        else:
            st["z"] = normal(rows, h).bfloat16()
            st["y"] = empty(t, h, dtype=torch.bfloat16)
            if case["step"] == "combine_train":
                st["dy"] = normal(t, h, scale=1e-3).bfloat16()
                st["dz"], st["dweights"] = empty(rows, h, dtype=torch.bfloat16), empty(t, k, dtype=torch.float32)
    elif case["op"] == "product":
        m, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
        counts = _loads(seed, m, g, case["skew"])
        st["bounds"] = [int(v) for v in np.concatenate([[0], np.cumsum(counts)])]
        st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device="cuda")
        st["w"], st["wt"] = _quantised_weights(g, n, k, gen)
        x = normal(m, k).bfloat16()
        kp, np_ = _up(k, BLOCK), _up(n, BLOCK)
        st["workspace"] = empty(64 << 20, dtype=torch.uint8)
        if case["step"] == "forward":
            st["x"] = x
            st["wt"] = None
            st["xq"] = empty(m, kp, dtype=F8["e4m3"]), empty(m, _up(kp // BLOCK, 4), dtype=torch.uint8)
            st["out"] = empty(m, n, dtype=torch.bfloat16)
        else:
            st["w"] = None
            # the layer's input, which its forward pass kept in 8 bits
            q, s = _quantised_rows(x, "e4m3")
            st["xq"] = q.to(F8["e4m3"]), torch.zeros(m, _up(kp // BLOCK, 4), dtype=torch.uint8, device="cuda")
            st["xq"][1][:, :kp // BLOCK] = s
            # gradients: rows of very different sizes
            st["dy"] = (normal(m, n, scale=1e-4) * torch.exp2(torch.randint(-6, 7, (m, 1), generator=gen, device="cuda"))).bfloat16()
            most = _up(m, BLOCK) + BLOCK * g
            st["dyq"] = empty(m, np_, dtype=F8[case["grad"]]), empty(m, _up(np_ // BLOCK, 4), dtype=torch.uint8)
            st["dyt"] = empty(n, most, dtype=F8[case["grad"]]), empty(n, _up(most // BLOCK, 4), dtype=torch.uint8)
            st["xt"] = empty(k, most, dtype=F8["e4m3"]), empty(k, _up(most // BLOCK, 4), dtype=torch.uint8)
            st["dx"], st["dw"] = empty(m, k, dtype=torch.bfloat16), empty(g, n, k, dtype=torch.bfloat16)
            st["most"] = most
    else:
        m, f = case["rows"], case["cols"]
        fp = _up(f, BLOCK)
        st["gu"] = normal(m, 2 * f).bfloat16()
        st["h"] = empty(m, f, dtype=torch.bfloat16)
        if case["train"]:
            st["dh"] = normal(m, f, scale=1e-3).bfloat16()
            st["kept"] = empty(m, 2 * fp, dtype=F8["e4m3"]), empty(m, _up(2 * fp // BLOCK, 4), dtype=torch.uint8)
            st["dgu"] = empty(m, 2 * f, dtype=torch.bfloat16)
    return st


# ---------------------------------------------------------------------------
# plain forms: elementary operations in 32 bits (64 where experts are ranked)
# ---------------------------------------------------------------------------

def _quantised_rows(x, fmt):
    """Blocks of 128 along the rows of x, padded with zeros: values of the 8-bit type (in 32 bits) and scale bytes."""
    m, k = x.shape
    t = torch.zeros(m, _up(k, BLOCK), device=x.device)
    t[:, :k] = x
    t = t.view(m, -1, BLOCK)
    f, e = torch.frexp(t.abs().amax(dim=2))
    b = torch.where(f > 0, e + 126 - TOP[fmt] + (f > 0.875).int(), 0).clamp(min=0)
    return _scaled(t, (127 - b)[:, :, None]).to(F8[fmt]).float().view(m, -1), b.to(torch.uint8)


def _values(q, s):
    """What blocks of 128 along the rows stand for."""
    m = q.shape[0]
    t = q.float().view(m, -1, BLOCK)
    return _scaled(t, s[:, :t.shape[1], None].int() - 127).view(m, -1)


def _weights(q, s, cols):
    """What blocks of 128 x 128 stand for, one matrix per group."""
    rows = q.shape[1]
    t = q.float().view(q.shape[0], rows, -1, BLOCK)
    e = s[:, :, :t.shape[2]].int().repeat_interleave(BLOCK, dim=1)[:, :rows] - 127
    return _scaled(t, e[..., None]).view(q.shape[0], rows, -1)[:, :, :cols]


def _along_tokens(x, bounds, fmt):
    """x with each group's rows in blocks of 128 of their own, as the values that their 8-bit form stands for."""
    def one(a, b):
        if a == b:
            return x[a:b]
        v = x[a:b].t().contiguous()
        return _values(*_quantised_rows(v, fmt))[:, :b - a].t()
    return [one(a, b) for a, b in zip(bounds, bounds[1:])]


def _plain_route(st):
    c = st["case"]
    t, e, k, groups = c["tokens"], c["experts"], c["top_k"], c["groups"]
    logits = st["logits"].double()
    s = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    rank = s if st["bias"] is None else s + st["bias"].double()
    if groups > 1:
        best = torch.sort(rank.view(t, groups, -1), dim=2, descending=True).values[:, :, :c["group_score"]].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["group_top"]]
        off = torch.ones(t, groups, dtype=torch.bool, device=rank.device).scatter_(1, kept, False)
        rank = rank.masked_fill(off.repeat_interleave(e // groups, dim=1), -math.inf)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :k]
    p = s.gather(1, ids).float()
    total = p.sum(dim=1, keepdim=True) + 1e-20
    w = (p / total if c["renorm"] else p) * c["scale"]
    out = {"ids": ids.int(), "weights": w}
    if c["train"]:
        d = st["dweights"] * c["scale"]
        if c["renorm"]:
            d = (d - (d * p / total).sum(dim=1, keepdim=True)) / total
        ds = torch.zeros(t, e, device=d.device).scatter_(1, ids, d)
        s = s.float()
        dl = ds * s * torch.sigmoid(-logits).float() if c["score"] == "sigmoid" else s * (ds - (d * p).sum(dim=1, keepdim=True))
        out["dlogits"] = dl.to(st["logits"].dtype)
    return out


def _plain_exchange(st):
    c = st["case"]
    t, k, e = c["tokens"], c["top_k"], c["experts"]
    if c["step"] == "dispatch":
        ids = st["ids"].reshape(-1).long()
        source = torch.sort(ids, stable=True).indices
        position = torch.empty_like(source)
        position[source] = torch.arange(t * k, device=ids.device)
        offsets = torch.zeros(e + 1, dtype=torch.int64, device=ids.device)
        offsets[1:] = torch.cumsum((ids[:, None] == torch.arange(e, device=ids.device)).sum(dim=0), dim=0)
        return {"offsets": offsets.int(), "position": position.int().view(t, k), "source": source.int(),
                "payload": st["x"][source // k]}
    at = st["position"].long()
    z = st["z"][at].float()
    out = {"y": (z * st["weights"][:, :, None]).sum(dim=1).bfloat16()}
    if c["step"] == "combine_train":
        dy = st["dy"].float()[:, None, :]
        out["dweights"] = (z * dy).sum(dim=2)
        dz = torch.empty_like(st["z"])
        dz[at.reshape(-1)] = (st["weights"][:, :, None] * dy).bfloat16().view(t * k, -1)
        out["dz"] = dz
    return out


def _plain_product(st):
    c = st["case"]
    n, k, bounds = c["n"], c["k"], st["bounds"]
    spans = list(zip(bounds, bounds[1:]))
    if c["step"] == "forward":
        x = _values(*_quantised_rows(st["x"], "e4m3"))[:, :k]
        w = _weights(*st["w"], k)
        return {"y": torch.cat([x[a:b] @ w[g].t() for g, (a, b) in enumerate(spans)]).bfloat16()}
    dy = _values(*_quantised_rows(st["dy"], c["grad"]))[:, :n]
    w = _weights(*st["wt"], n)
    dx = torch.cat([dy[a:b] @ w[g].t() for g, (a, b) in enumerate(spans)]).bfloat16()
    x = _along_tokens(_values(*st["xq"])[:, :k], bounds, "e4m3")
    dw = [(v.t() @ u).bfloat16() for v, u in zip(_along_tokens(st["dy"].float(), bounds, c["grad"]), x)]
    return {"dx": dx, "dw": torch.stack(dw)}


def _plain_gate(st):
    c = st["case"]
    f = c["cols"]
    gu = st["gu"].float()
    g, u = gu[:, :f], gu[:, f:]
    out = {"h": (g * torch.sigmoid(g) * u).bfloat16()}
    if c["train"]:
        g = _values(*_quantised_rows(g, "e4m3"))[:, :f]
        u = _values(*_quantised_rows(u, "e4m3"))[:, :f]
        s, dh = torch.sigmoid(g), st["dh"].float()
        out["dgu"] = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1).bfloat16()
    return out


# ---------------------------------------------------------------------------
# the calls a user makes
# ---------------------------------------------------------------------------

def _own_route(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    cfg = zc.route_config(experts=c["experts"], top_k=c["top_k"], score=c["score"], groups=c["groups"],
                          group_top=c["group_top"], group_score=c["group_score"], renormalise=c["renorm"], scale=c["scale"])
    kind = zc.ZC_BF16 if c["dtype"] == "bfloat16" else zc.ZC_F32
    zc.zc_route(st["logits"], kind, c["tokens"], c["experts"], st["bias"], cfg, st["ids"], st["weights"])
    out = {"ids": st["ids"], "weights": st["weights"]}
    if c["train"]:
        zc.zc_route_backward(st["logits"], kind, c["tokens"], c["experts"], cfg, st["ids"], st["dweights"], st["dlogits"],
                             c["experts"])
        out["dlogits"] = st["dlogits"]
    return out


def _own_exchange(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    t, k, e, h = c["tokens"], c["top_k"], c["experts"], c["hidden"]
    if c["step"] == "dispatch":
        zc.zc_dispatch_plan(st["ids"], t, k, e, st["workspace"], st["workspace"].numel(), st["offsets"],
                            st["plan_position"], st["plan_source"])
        zc.zc_dispatch(st["x"], t, h, h, st["plan_position"], k, st["out"], t * k, h)
        return {"offsets": st["offsets"], "position": st["plan_position"], "source": st["plan_source"],
                "payload": st["out"]}
    zc.zc_combine(st["z"], t * k, h, h, st["position"], st["weights"], t, k, st["y"], h)
    out = {"y": st["y"]}
    if c["step"] == "combine_train":
        zc.zc_combine_backward(st["dy"], h, st["z"], t * k, h, h, st["position"], st["weights"], t, k, st["dz"], h,
                               st["dweights"])
        out |= {"dweights": st["dweights"], "dz": st["dz"]}
    return out


def _own_product(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    m, g, n, k = c["rows"], c["groups"], c["n"], c["k"]
    e4 = zc.ZC_FP8_E4M3
    if c["step"] == "forward":
        (xq, xs), (wq, ws) = st["xq"], st["w"]
        zc.zc_fp8_quantize(st["x"], m, k, k, e4, 1, xq, xs)
        zc.zc_fp8_matmul(xq, xs, e4, m, wq, ws, e4, n, k, g, st["offsets"], st["out"], zc.ZC_BF16, n,
                         zc.ZC_FP8_SUM_FAST, st["workspace"], st["workspace"].numel())
        return {"y": st["out"]}
    gf = zc.ZC_FP8_E5M2 if c["grad"] == "e5m2" else e4
    (dq, ds), (dt, dts), (xt, xts), (wq, ws) = st["dyq"], st["dyt"], st["xt"], st["wt"]
    zc.zc_fp8_quantize(st["dy"], m, n, n, gf, 1, dq, ds)
    zc.zc_fp8_matmul(dq, ds, gf, m, wq, ws, e4, k, n, g, st["offsets"], st["dx"], zc.ZC_BF16, k,
                     zc.ZC_FP8_SUM_FAST, st["workspace"], st["workspace"].numel())
    zc.zc_fp8_quantize_t(st["dy"], None, zc.ZC_BF16, m, n, n, g, st["offsets"], gf, dt, dts, st["most"])
    zc.zc_fp8_quantize_t(st["xq"][0], st["xq"][1], e4, m, k, _up(k, BLOCK), g, st["offsets"], e4, xt, xts, st["most"])
    zc.zc_fp8_matmul_wgrad(dt, dts, gf, n, xt, xts, e4, k, st["most"], m, g, st["offsets"], st["dw"], zc.ZC_BF16,
                           zc.ZC_FP8_SUM_FAST)
    return {"dx": st["dx"], "dw": st["dw"]}


def _own_gate(st):
    from lossless_bf16_exponent_amd import zc_moe as zc
    c = st["case"]
    m, f = c["rows"], c["cols"]
    kq, ks = st["kept"] if c["train"] else (None, None)
    zc.zc_swiglu(st["gu"], m, f, 2 * f, st["h"], f, None, None, kq, ks)
    out = {"h": st["h"]}
    if c["train"]:
        zc.zc_swiglu_backward(kq, ks, m, f, st["dh"], f, st["dgu"], 2 * f)
        out["dgu"] = st["dgu"]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "exchange": _own_exchange, "product": _own_product, "gate": _own_gate}[op](state)
    return {"route": _plain_route, "exchange": _plain_exchange, "product": _plain_product, "gate": _plain_gate}[op](state)


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        size = 2 if case["dtype"] == "bfloat16" else 4
        b = t * e * size + 8 * t * k + (4 * e if case["bias"] else 0)
        if case["train"]:
            b += 4 * t * k + t * e * size
        return {"bytes": b, "flops": t * e * (16 if case["train"] else 8)}
    if case["op"] == "exchange":
        t, k, e, h = case["tokens"], case["top_k"], case["experts"], case["hidden"]
        if case["step"] == "dispatch":
            return {"bytes": 2 * h * (t + t * k) + 12 * t * k + 4 * e, "flops": 0}
        if case["step"] == "combine":
            return {"bytes": 2 * h * (t + t * k) + 8 * t * k, "flops": 2 * t * k * h}
        # the rows' values are read once for the sum and its gradients together
        return {"bytes": 2 * h * (2 * t + 2 * t * k) + 12 * t * k, "flops": 5 * t * k * h}
    if case["op"] == "product":
        m, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
        used = min(m, g)
        if case["step"] == "forward":
            return {"bytes": 2 * m * k + used * n * k + 2 * m * n, "flops": 2 * m * n * k}
        return {"bytes": m * k + 2 * m * n + used * n * k + 2 * m * k + 2 * g * n * k, "flops": 4 * m * n * k}
    m, f = case["rows"], case["cols"]
    return {"bytes": m * f * ((6 + 2 + 4) if case["train"] else 6), "flops": m * f * (20 if case["train"] else 6)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e in 64 bits, from a table."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=e.device)[e.long() + 300]


def _to_8_bits(v, fmt, dims):
    """64-bit values rounded to the 8-bit type under one scale over `dims`, as the values they then stand for."""
    largest, least, bits = {"e4m3": (448.0, -6, 3), "e5m2": (57344.0, -14, 2)}[fmt]
    m, e = torch.frexp(v.abs().amax(dim=dims, keepdim=True) / largest)
    scale = _two_to(torch.where(m > 0.5, e, e - 1).clamp(min=-127))
    v = v / scale
    step = _two_to((torch.frexp(v)[1] - 1).clamp(min=least) - bits)
    return torch.round(v / step) * step * scale


def _rows_8(v, fmt):
    m, k = v.shape
    pad = torch.nn.functional.pad(v, (0, -k % BLOCK))
    return _to_8_bits(pad.reshape(m, -1, BLOCK), fmt, (2,)).reshape(m, -1)[:, :k]


def _stood_for(q, s, g):
    """64-bit values of group g's 128 x 128 blocks."""
    rows, cols = q.shape[1:]
    scale = _two_to(s[g, :, :cols // BLOCK].long() - 127)
    return q[g].double() * torch.kron(scale, torch.ones(BLOCK, BLOCK, dtype=torch.float64, device=q.device))[:rows, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        t, k = case["tokens"], case["top_k"]
        x = st["logits"].cpu().double().numpy()
        if case["score"] == "sigmoid":
            s = 1 / (1 + np.exp(-x))
        else:
            s = np.exp(x - x.max(axis=1, keepdims=True))
            s /= s.sum(axis=1, keepdims=True)
        rank = s + (0 if st["bias"] is None else st["bias"].cpu().double().numpy()[None])
        if case["groups"] > 1:
            per = rank.reshape(t, case["groups"], -1)
            best = np.partition(per, per.shape[2] - case["group_score"], axis=2)[:, :, -case["group_score"]:].sum(axis=2)
            place = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
            rank = np.where((place < case["group_top"])[:, :, None], per, -np.inf).reshape(t, -1)
        ids = np.argsort(-rank, axis=1, kind="stable")[:, :k]
        p = np.take_along_axis(s, ids, axis=1)
        norm = p.sum(axis=1, keepdims=True) if case["renorm"] else 1.0
        w = p / norm * case["scale"]
        out = {"ids": ids.astype(np.int32), "weights": w}
        if case["train"]:
            dw = st["dweights"].cpu().double().numpy()
            dp = case["scale"] * dw / norm
            if case["renorm"]:
                dp = dp - (dw * w).sum(axis=1, keepdims=True) / norm
            ds = np.zeros_like(s)
            np.put_along_axis(ds, ids, dp, axis=1)
            if case["score"] == "sigmoid":
                out["dlogits"] = ds * s / (1 + np.exp(x))
            else:
                out["dlogits"] = s * ds - s * (s * ds).sum(axis=1, keepdims=True)
        return out
    if case["op"] == "exchange":
        t, k, h = case["tokens"], case["top_k"], case["hidden"]
        if case["step"] == "dispatch":
            ids = st["ids"].cpu().numpy().reshape(-1)
            source = np.lexsort((np.arange(ids.size), ids))
            position = np.argsort(source).reshape(t, k)
            offsets = np.searchsorted(ids[source], np.arange(case["experts"] + 1))
            payload = st["x"].double()[torch.from_numpy(source // k).cuda()]
            return {"offsets": offsets.astype(np.int32), "position": position.astype(np.int32),
                    "source": source.astype(np.int32), "payload": payload}
        at, w = st["position"].long(), st["weights"].double()
        y = torch.zeros(t, h, dtype=torch.float64, device="cuda")
        for j in range(k):
            y += w[:, j, None] * st["z"][at[:, j]].double()
        out = {"y": y}
        if case["step"] == "combine_train":
            dy = st["dy"].double()
            dz = torch.empty(t * k, h, dtype=torch.float64, device="cuda")
            dw = torch.empty(t, k, dtype=torch.float64, device="cuda")
            for j in range(k):
                dw[:, j] = (st["z"][at[:, j]].double() * dy).sum(dim=1)
                dz[at[:, j]] = dy * w[:, j, None]
            out |= {"dweights": dw, "dz": dz}
        return out
    if case["op"] == "product":
        n, k, bounds = case["n"], case["k"], st["bounds"]
        m, g = case["rows"], case["groups"]
        if case["step"] == "forward":
            x = _rows_8(st["x"].double(), "e4m3")
            y = torch.empty(m, n, dtype=torch.float64, device="cuda")
            for i in range(g):
                a, b = bounds[i], bounds[i + 1]
                if a < b:
                    y[a:b] = torch.mm(x[a:b], _stood_for(*st["w"], i)[:, :k].t())
            return {"y": y}
        dyr = st["dy"].double()
        dy = _rows_8(dyr, case["grad"])
        scale = _two_to(st["xq"][1].long() - 127)
        kept = st["xq"][0].double() * scale.repeat_interleave(BLOCK, dim=1)[:, :_up(k, BLOCK)]
        dx = torch.empty(m, k, dtype=torch.float64, device="cuda")
        dw = torch.zeros(g, n, k, dtype=torch.float64, device="cuda")
        for i in range(g):
            a, b = bounds[i], bounds[i + 1]
            if a < b:
                dx[a:b] = torch.mm(dy[a:b], _stood_for(*st["wt"], i)[:, :n].t())
                dw[i] = torch.mm(_rows_8(dyr[a:b].t(), case["grad"]), _rows_8(kept[a:b, :k].t(), "e4m3").t())
        return {"dx": dx, "dw": dw}
    f = case["cols"]
    g, u = st["gu"].double()[:, :f], st["gu"].double()[:, f:]
    out = {"h": u * g / (1 + torch.exp(-g))}
    if case["train"]:
        g, u, dh = _rows_8(g, "e4m3"), _rows_8(u, "e4m3"), st["dh"].double()
        slope = (1 + torch.exp(-g) + g * torch.exp(-g)) / (1 + torch.exp(-g)) ** 2
        out["dgu"] = torch.cat([dh * u * slope, dh * g / (1 + torch.exp(-g))], dim=1)
    return out
