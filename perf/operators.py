"""Cases, plain forms and 64-bit values of the block operators around the expert epilogue:

* ``norm_fwd`` / ``norm_bwd``: layer norm over the hidden axis and its gradients (the weight's and
  the bias's reduced over all rows), ahead of the router and the experts of every block;
* ``router_fwd`` / ``router_bwd``: softmax or sigmoid scores, the top-k experts of each token and
  their routing weights, and the gradient of the logits;
* ``layer``: a whole mixture-of-experts layer for a few tokens (router product, top-k, both expert
  products with the clamped SwiGLU between them, the combine and the residual), the decode step.

``run`` computes them with elementary torch operations, or, where ``own`` is true, through
``moe_expert_epilogue_b200.ops``.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
INF = float("inf")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm of one decode step of four sequences: launch latency
        {"name": "norm_fwd_decode", "op": "norm_fwd", "rows": 4, "hidden": 7168, "dtype": "bf16",
         "wdtype": "bf16", "bias": True},
        # a training step's activations (the router-weight workload's shape)
        {"name": "norm_fwd_train", "op": "norm_fwd", "rows": 16384, "hidden": 7168, "dtype": "bf16",
         "wdtype": "bf16", "bias": True},
        # its backward pass, the parameters kept in 32 bits
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 16384, "hidden": 7168, "dtype": "bf16",
         "wdtype": "fp32", "bias": True},
        # an odd width in 32 bits, no bias: no row but the first is aligned
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 4099, "hidden": 1001, "dtype": "fp32",
         "wdtype": "fp32", "bias": False},
        # routing of one decode step: latency
        {"name": "router_fwd_decode", "op": "router_fwd", "tokens": 16, "experts": 64, "top_k": 8,
         "dtype": "fp32", "score": "softmax", "normalise": True, "scale": 1.0, "masked": 0.0},
        # routing of a long prompt over many experts, half of them closed to each token
        {"name": "router_fwd_prompt", "op": "router_fwd", "tokens": 32768, "experts": 256, "top_k": 8,
         "dtype": "bf16", "score": "sigmoid", "normalise": True, "scale": 2.5, "masked": 0.5},
        # the training workload of the permuted activation: 8192 tokens, top-8 of 64
        {"name": "router_bwd_train", "op": "router_bwd", "tokens": 8192, "experts": 64, "top_k": 8,
         "dtype": "fp32", "score": "softmax", "normalise": True, "scale": 1.0, "masked": 0.0},
        # odd counts, probabilities over all experts kept as they are
        {"name": "router_bwd_odd", "op": "router_bwd", "tokens": 30001, "experts": 161, "top_k": 6,
         "dtype": "bf16", "score": "softmax", "normalise": False, "scale": 1.0, "masked": 0.25},
        # one token: the shortest step, eight experts' weights read once
        {"name": "layer_one_token", "op": "layer", "tokens": 1, "valid": 1, "hidden": 4096,
         "inter": 2048, "experts": 64, "top_k": 8, "dtype": "bf16", "score": "softmax",
         "normalise": True, "limit": 7.0, "router": "weight", "masked": 0.0},
        # a padded batch (11 of 13 tokens live) over a narrow, odd layer routed by the caller's logits
        {"name": "layer_odd_padded", "op": "layer", "tokens": 13, "valid": 11, "hidden": 1224,
         "inter": 616, "experts": 60, "top_k": 6, "dtype": "fp16", "score": "softmax",
         "normalise": False, "limit": INF, "router": "logits", "masked": 0.3},
        # a small serving batch on a wide layer
        {"name": "layer_batch", "op": "layer", "tokens": 16, "valid": 16, "hidden": 7168,
         "inter": 2048, "experts": 32, "top_k": 4, "dtype": "bf16", "score": "sigmoid",
         "normalise": True, "limit": 10.0, "router": "weight", "masked": 0.0},
        # the largest batch of the range: every expert is read
        {"name": "layer_full", "op": "layer", "tokens": 64, "valid": 64, "hidden": 4096,
         "inter": 2048, "experts": 64, "top_k": 8, "dtype": "bf16", "score": "softmax",
         "normalise": True, "limit": 7.0, "router": "weight", "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "router_fwd", "router_bwd", "layer", "layer"])
    if op.startswith("norm"):
        hidden = _log(rng, 48, 8192)
        if rng.random() < 0.75:
            hidden = -(-hidden // 16) * 16
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 16384 * 7168 * 2 // SIZE[dtype] // hidden
        return {"op": op, "rows": _log(rng, 1, min(65536, most)), "hidden": hidden, "dtype": dtype,
                "wdtype": rng.choice([dtype, "fp32"]), "bias": rng.random() < 0.7}
    if op.startswith("router"):
        experts = rng.choice([8, 16, 60, 64, 96, 128, 160, 161, 256, 384])
        return {"op": op, "tokens": _log(rng, 1, 32768 * 256 // max(experts, 256)), "experts": experts,
                "top_k": rng.randint(1, 8), "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "normalise": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.0, 0.25, 0.5])}
    hidden, inter = _log(rng, 256, 7168), _log(rng, 64, 4096)
    if rng.random() < 0.85:
        hidden, inter = -(-hidden // 8) * 8, -(-inter // 8) * 8
    most = 64 * 4096 * 2048 // (hidden * inter)
    experts = max(8, min(rng.choice([8, 16, 32, 60, 64, 128]), most))
    tokens = _log(rng, 1, 64)
    return {"op": "layer", "tokens": tokens, "valid": tokens - rng.randint(0, 2) * (tokens > 4),
            "hidden": hidden, "inter": min(inter, 64 * 4096 * 2048 // (hidden * experts)),
            "experts": experts, "top_k": rng.randint(1, 8), "dtype": rng.choice(["bf16", "bf16", "fp16"]),
            "score": rng.choice(["softmax", "sigmoid"]), "normalise": rng.random() < 0.7,
            "limit": rng.choice([7.0, 10.0, INF]), "router": rng.choice(["weight", "logits"]),
            "masked": 0.0}


# ------------------------------------------------------------------ inputs

def _logits(case, g):
    """N(0, 1) logits; with ``masked`` that share of the experts is closed (-inf) to each token."""
    t, e = case["tokens"], case["experts"]
    logits = torch.randn(t, e, generator=g, device=DEV)
    if case["masked"] > 0:
        shut = torch.rand(t, e, generator=g, device=DEV).argsort(1) < int(case["masked"] * e)
        logits = logits.masked_fill(shut, -INF)
    return logits


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 2 + 1)
    s = dict(case)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"].startswith("norm"):
        n, h, wdt = case["rows"], case["hidden"], DTYPES[case["wdtype"]]
        s["x"] = (randn(n, h) * 1.5 + 0.4 * randn(h)).to(dt)   # channels with means of their own
        s["weight"] = (1 + 0.1 * randn(h)).to(wdt)
        s["bias_"] = (0.1 * randn(h)).to(wdt) if case["bias"] else None
        if case["op"] == "norm_bwd":
            s["grad_y"] = randn(n, h).to(dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = ((x - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
    elif case["op"].startswith("router"):
        s["logits"] = _logits(case, g).to(dt)
        if case["op"] == "router_bwd":
            s["ids"] = _top(s["logits"].float(), case["top_k"])[1]
            s["grad_weights"] = randn(case["tokens"], case["top_k"])
    else:
        t, h, i, e = case["tokens"], case["hidden"], case["inter"], case["experts"]
        s["x"] = randn(t, h).to(dt)
        s["w1"] = torch.randn(e, 2 * i, h, generator=g, device=DEV, dtype=dt).mul_(h ** -0.5)
        s["w2"] = torch.randn(e, h, i, generator=g, device=DEV, dtype=dt).mul_(i ** -0.5)
        s["router_weight"] = (randn(e, h) * h ** -0.5).to(dt) if case["router"] == "weight" else None
        s["logits"] = _logits(case, g) if case["router"] == "logits" else None
        s["shared"], s["residual"] = randn(t, h).to(dt), randn(t, h).to(dt)
        s["valid_tokens"] = torch.tensor([case["valid"]], dtype=torch.int32, device=DEV)
        # what a serving loop keeps: the outputs (rows of padding tokens stay as they are)
        s["out"] = torch.zeros(t, h, dtype=dt, device=DEV)
        s["out_ids"] = torch.full((t, case["top_k"]), -1, dtype=torch.int32, device=DEV)
        s["out_weights"] = torch.zeros(t, case["top_k"], device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _top(logits, k):
    """The k largest of each row, ties to the lowest index, and their int32 indices; -1 where
    nothing but -inf is left."""
    v, i = logits.sort(dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k].int()
    return v, torch.where(v == -INF, torch.full_like(i, -1), i)


def _weights(s, logits, v, ids):
    if s["score"] == "softmax":
        m = logits.amax(1, keepdim=True)
        e = (v - m).exp()
        w = e / (e.sum(1, keepdim=True) if s["normalise"] else (logits - m).exp().sum(1, keepdim=True))
    else:
        e = 1 / (1 + (-v).exp())
        w = e / e.sum(1, keepdim=True) if s["normalise"] else e
    return torch.where(ids < 0, torch.zeros_like(w), w * s.get("scale", 1.0))


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["weight"].float()
    if s["bias_"] is not None:
        y = y + s["bias_"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    gy, rstd = s["grad_y"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    a = gy * s["weight"].float()
    gx = rstd * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
    out = {"grad_x": gx.to(s["x"].dtype), "grad_weight": (gy * xhat).sum(0).to(s["weight"].dtype)}
    if s["bias_"] is not None:
        out["grad_bias"] = gy.sum(0).to(s["bias_"].dtype)
    return out


def _plain_router_fwd(s):
    logits = s["logits"].float()
    v, ids = _top(logits, s["top_k"])
    return {"weights": _weights(s, logits, v, ids), "ids": ids}


def _plain_router_bwd(s):
    logits, live = s["logits"].float(), s["ids"] >= 0
    i = s["ids"].clamp(min=0).long()
    v = logits.gather(1, i).masked_fill(~live, -INF)
    g = torch.where(live, s["grad_weights"] * s["scale"], torch.zeros_like(s["grad_weights"]))
    if s["score"] == "softmax":
        m = logits.amax(1, keepdim=True)
        e = (v - m).exp()
        if s["normalise"]:
            w = e / e.sum(1, keepdim=True)
            d = w * (g - (g * w).sum(1, keepdim=True))
            full = torch.zeros_like(logits)
        else:
            p = (logits - m).exp()
            p = p / p.sum(1, keepdim=True)
            w = p.gather(1, i)
            d = w * g
            full = -p * d.sum(1, keepdim=True)
    else:
        z = 1 / (1 + (-v).exp())
        if s["normalise"]:
            w = z / z.sum(1, keepdim=True)
            d = w * (g - (g * w).sum(1, keepdim=True)) * (1 - z)
        else:
            d = g * z * (1 - z)
        full = torch.zeros_like(logits)
    d = torch.where(live, d, torch.zeros_like(d))
    return {"grad_logits": full.scatter_add(1, i, d).to(s["logits"].dtype)}


def _plain_layer(s):
    x, (t, k, e) = s["x"].float(), (s["tokens"], s["top_k"], s["experts"])
    inter = s["inter"]
    if s["logits"] is None:   # 64-bit sums: a sum's order must not choose between two near experts
        logits = (s["x"].double() @ s["router_weight"].double().t()).float()
    else:
        logits = s["logits"]
    v, ids = _top(logits, k)
    w = _weights(s, logits, v, ids)
    i = ids.clamp(min=0).long()
    if t * k < e:             # few slots: their experts' weights alone
        flat = i.reshape(-1)
        slot = x.repeat_interleave(k, 0)[:, :, None]
        z = torch.bmm(s["w1"][flat].float(), slot)[:, :, 0]
        w2, weight = s["w2"][flat].float(), w.reshape(-1, 1)
    else:                     # every expert over every token, weighted by 0 where not chosen
        z = torch.matmul(x, s["w1"].float().transpose(1, 2))
        w2 = s["w2"].float()
        weight = torch.zeros(t, e, device=DEV).scatter_add(1, i, w).t()[:, :, None]
    gate, up = z[..., :inter].clamp(max=s["limit"]), z[..., inter:].clamp(-s["limit"], s["limit"])
    h = gate / (1 + (-gate).exp()) * up * weight
    if t * k < e:
        y = torch.bmm(w2, h[:, :, None])[:, :, 0].reshape(t, k, -1).sum(1)
    else:
        y = torch.matmul(h, w2.transpose(1, 2)).sum(0)
    y = (s["residual"].float() + (y + s["shared"].float())).to(s["x"].dtype)
    live = torch.arange(t, device=DEV)[:, None] < s["valid_tokens"]
    return {"out": torch.where(live, y, s["out"]), "ids": torch.where(live, ids, s["out_ids"]),
            "weights": torch.where(live, w, s["out_weights"])}


PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "router_fwd": _plain_router_fwd,
         "router_bwd": _plain_router_bwd, "layer": _plain_layer}


def _own(s):
    from moe_expert_epilogue_b200 import ops
    op = s["op"]
    if op == "norm_fwd":
        y, mean, rstd = ops.layer_norm_fwd(s["x"], s["weight"], s["bias_"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        gx, gw, gb = ops.layer_norm_bwd(s["grad_y"], s["x"], s["weight"], s["mean"], s["rstd"],
                                        has_bias=s["bias_"] is not None)
        out = {"grad_x": gx, "grad_weight": gw}
        if gb is not None:
            out["grad_bias"] = gb
        return out
    score = ops.MOE_SCORE_SOFTMAX if s["score"] == "softmax" else ops.MOE_SCORE_SIGMOID
    if op == "router_fwd":
        weights, ids = ops.router_topk_fwd(s["logits"], s["top_k"], score, s["normalise"], s["scale"])
        return {"weights": weights, "ids": ids}
    if op == "router_bwd":
        return {"grad_logits": ops.router_topk_bwd(s["logits"], s["ids"], s["grad_weights"], score,
                                                   s["normalise"], s["scale"])}
    out = ops.moe_layer_small_batch(
        s["x"], s["w1"], s["w2"], s["top_k"], router_weight=s["router_weight"], logits=s["logits"],
        score=score, normalise=s["normalise"], limit=s["limit"], shared_expert_output=s["shared"],
        residual=s["residual"], valid_tokens=s["valid_tokens"], out=s["out"],
        topk_weights=s["out_weights"], topk_ids=s["out_ids"])
    return {"out": out, "ids": s["out_ids"], "weights": s["out_weights"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    es = SIZE[case["dtype"]]
    if case["op"].startswith("norm"):
        n, h, ws = case["rows"], case["hidden"], SIZE[case["wdtype"]]
        params = h * ws * (2 if case["bias"] else 1)
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * h * es + params + 8 * n, "flops": 8 * n * h}
        return {"bytes": 3 * n * h * es + h * ws + params + 8 * n, "flops": 16 * n * h}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if case["op"] == "router_fwd":
        return {"bytes": t * e * es + 8 * t * k, "flops": 4 * t * e}
    if case["op"] == "router_bwd":
        # a normalised weight depends on the chosen logits alone, as a sigmoid does
        read = t * e if case["score"] == "softmax" and not case["normalise"] else t * k
        return {"bytes": (read + t * e) * es + 8 * t * k, "flops": 4 * t * e}
    t, h, i = case["valid"], case["hidden"], case["inter"]
    active = e * (1 - (1 - k / e) ** t)       # experts that some token chose, on average
    router = e * h * es if case["router"] == "weight" else 4 * t * e
    return {"bytes": active * 3 * h * i * es + router + 4 * t * h * es + 8 * t * k,
            "flops": 6 * t * k * h * i + (2 * t * e * h if case["router"] == "weight" else 0)}


# ------------------------------------------------------------------ 64 bits

def _exact_weights(case, logits, ids):
    """Routing weights from the definition: score of each chosen expert, over the chosen ones' sum
    where normalised.  logits and the result in 64 bits."""
    chosen = ids >= 0
    at = ids.long().clamp(min=0)
    if case["score"] == "softmax":
        score = torch.softmax(logits, dim=1)
    else:
        score = torch.sigmoid(logits)
    w = score.gather(1, at) * chosen
    if case["normalise"]:
        w = w / w.sum(1, keepdim=True)
    return torch.where(chosen, w * case.get("scale", 1.0), 0.0)


def _exact_ids(logits, k):
    """Expert by expert: the largest left, the first of equals."""
    left, ids = logits.clone(), []
    n = torch.arange(logits.shape[1], device=DEV)
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        i = torch.where(left == top, n, logits.shape[1]).amin(1)
        ids.append(torch.where(top[:, 0] == -INF, -1, i))
        left.scatter_(1, i[:, None], -INF)
    return torch.stack(ids, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = torch.addcmul(torch.zeros((), dtype=torch.float64, device=DEV) if s["bias_"] is None
                          else s["bias_"].double(),
                          (x - mean[:, None]) / (var + EPS).sqrt()[:, None], s["weight"].double())
        return {"y": y, "mean": mean, "rstd": 1 / (var + EPS).sqrt()}
    if case["op"] == "norm_bwd":
        # the gradients of sum(grad_y * y), y = xhat * weight + bias, for the statistics given
        xhat = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        gy, n = s["grad_y"].double(), case["hidden"]
        gw = torch.einsum("rh,rh->h", gy, xhat)
        gxhat = gy * s["weight"].double()
        gx = (n * gxhat - gxhat.sum(1, keepdim=True)
              - xhat * torch.einsum("rh,rh->r", gxhat, xhat)[:, None]) * (s["rstd"].double()[:, None] / n)
        out = {"grad_x": gx, "grad_weight": gw}
        if s["bias_"] is not None:
            out["grad_bias"] = gy.sum(0)
        return out
    if case["op"] == "router_fwd":
        logits = s["logits"].double()
        return {"weights": _exact_weights(case, logits, _exact_ids(logits, case["top_k"])), "ids": None}
    if case["op"] == "router_bwd":
        with torch.enable_grad():
            z = s["logits"].double().requires_grad_()
            chosen = s["ids"] >= 0
            at = s["ids"].long().clamp(min=0)
            if case["score"] == "softmax" and case["normalise"]:   # softmax of the chosen logits
                w = torch.softmax(z.gather(1, at).masked_fill(~chosen, -INF), dim=1)
            elif case["score"] == "softmax":
                w = torch.softmax(z, dim=1).gather(1, at)
            else:
                w = torch.sigmoid(z).gather(1, at) * chosen
                if case["normalise"]:
                    w = w / w.sum(1, keepdim=True)
            w = torch.where(chosen, w * case["scale"], 0.0)
            (gz,) = torch.autograd.grad((w * s["grad_weights"].double()).sum(), z)
        return {"grad_logits": torch.nan_to_num(gz, nan=0.0)}
    x, i = s["x"].double(), case["inter"]
    if s["logits"] is None:   # the logits are rounded to 32 bits before anything is chosen by them
        logits = torch.stack([x @ r for r in s["router_weight"].double()], 1).float().double()
    else:
        logits = s["logits"].double()
    ids = _exact_ids(logits, case["top_k"])
    w = _exact_weights(case, logits, ids)
    out = s["residual"].double() + s["shared"].double()
    for e in range(case["experts"]):
        t, k = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            gate, up = (x[t] @ s["w1"][e].double().t()).split(i, dim=1)
            act = torch.nn.functional.silu(gate.clamp(max=case["limit"])) \
                * up.clamp(-case["limit"], case["limit"])
            out.index_add_(0, t, act @ s["w2"][e].double().t() * w[t, k][:, None])
    live = torch.arange(case["tokens"], device=DEV)[:, None] < case["valid"]
    return {"out": torch.where(live, out, s["out"].double()), "ids": None,
            "weights": torch.where(live, w, s["out_weights"].double())}
