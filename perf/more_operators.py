"""Timed cases of what stands around the library's products in a language model.

Three operators, each forward and backward, in float32 like the products:

  route           a router's scores to each token's experts and their weights
  route_backward  the gradient of the weights back to the router's scores
  norm            layer norm over rows, with the statistics its gradient needs
  norm_backward   its gradients: of the rows, of the weight and of the bias
  loss            softmax cross entropy of rows times a vocabulary's weight
  loss_backward   its gradients: of the rows and of that weight

``run`` computes a case with elementary torch operations; with ``own`` set it
makes the library's calls instead.
"""
import math

import torch

own = False

WORKSPACE_BYTES = 1 << 30       # what a training program keeps for its layers' calls
EPS = 1e-5


def listed():
    return [
        # a decoding batch choosing two of eight experts
        {"name": "route 16 tokens", "op": "route", "t": 16, "e": 8, "top": 2, "scoring": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "renorm": True,
         "scale": 1.0, "masked": False},
        # a training batch of odd length over 64 experts, weights as the softmax gives them
        {"name": "route 8191 tokens", "op": "route", "t": 8191, "e": 64, "top": 6,
         "scoring": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_best": 1,
         "renorm": False, "scale": 1.0, "masked": False},
        # a long batch over many experts in groups, balanced by a bias
        {"name": "route 32768 tokens", "op": "route", "t": 32768, "e": 256, "top": 8,
         "scoring": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2,
         "renorm": True, "scale": 2.5, "masked": False},
        # the gradient of such a batch through a whole softmax
        {"name": "route backward 32768 tokens", "op": "route_backward", "t": 32768, "e": 256,
         "top": 8, "scoring": "softmax", "renorm": False, "scale": 1.0, "masked": False},
        # a decoding batch
        {"name": "norm 16 rows", "op": "norm", "t": 16, "h": 1024, "affine": True, "pad": False},
        # a long training batch
        {"name": "norm 32768 rows", "op": "norm", "t": 32768, "h": 4096, "affine": True,
         "pad": False},
        # a prompt of odd length and width
        {"name": "norm backward 1000 rows", "op": "norm_backward", "t": 1000, "h": 777,
         "affine": True, "residual": False, "pad": True},
        # the gradients of a long batch, joined with the residual's
        {"name": "norm backward 32768 rows", "op": "norm_backward", "t": 32768, "h": 1024,
         "affine": True, "residual": True, "pad": False},
        # a few tokens scored against a vocabulary stored out x in
        {"name": "loss 16 tokens", "op": "loss", "t": 16, "h": 1024, "v": 32768, "tb": True,
         "ignored": 0, "pad": False},
        # a training batch, a quarter of it padding or prompt
        {"name": "loss 8192 tokens", "op": "loss", "t": 8192, "h": 1024, "v": 32768, "tb": True,
         "ignored": 2048, "pad": False},
        # the gradients at odd sizes, the weight stored in x out
        {"name": "loss backward 1000 tokens", "op": "loss_backward", "t": 1000, "h": 777,
         "v": 5003, "tb": False, "ignored": 123, "pad": False},
        # the gradients of the training batch, every token counted
        {"name": "loss backward 8192 tokens", "op": "loss_backward", "t": 8192, "h": 1024,
         "v": 32768, "tb": True, "ignored": 0, "pad": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "norm", "norm_backward", "loss", "loss_backward"])
    yes = lambda p=0.5: rng.random() < p  # noqa: E731
    if op in ("route", "route_backward"):
        t = _log(rng, 1, 32768)
        c = {"op": op, "t": t, "scoring": rng.choice(["softmax", "sigmoid"]), "renorm": yes(),
             "scale": rng.choice([1.0, 2.5])}
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        e = _log(rng, 2, 256 // groups) * groups
        c["masked"] = e >= 16 and yes(0.3)
        least = 2 if c["renorm"] else 1     # one weight alone is renormalised to a constant
        if op == "route":
            top_groups = rng.randint(1, groups)
            c |= {"bias": yes(), "groups": groups, "top_groups": top_groups,
                  "group_best": rng.randint(1, min(2, e // groups))}
            c["top"] = rng.randint(least, min(8, e // groups * top_groups))
        else:
            c["top"] = rng.randint(least, min(8, e))
        return c | {"e": e}
    if op in ("norm", "norm_backward"):
        h = _log(rng, 16, 8192)
        t = _log(rng, 1, min(65536, 30_000_000 // h))
        c = {"op": op, "t": t, "h": h, "affine": yes(0.8), "pad": yes(0.3)}
        return c | {"residual": yes()} if op == "norm_backward" else c
    h, v = _log(rng, 64, 4096), _log(rng, 100, 65536)
    most = min(8192, 200_000_000_000 // (h * v), 400_000_000 // v)
    t = _log(rng, 1, most)
    ignored = rng.randint(0, t // 2) if yes() else 0
    return {"op": op, "t": t, "h": h, "v": v, "tb": yes(), "ignored": ignored, "pad": yes(0.3)}


# Inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _matrix(g, rows, cols, scale=1.0, pad=False):
    """rows x cols values; with `pad`, inside a wider buffer."""
    wide = torch.randn(rows, cols + (3 if pad else 0), generator=g, device="cuda")
    return wide.mul_(scale)[:, :cols]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("route", "route_backward"):
        t, e, top = case["t"], case["e"], case["top"]
        liking = 0.5 * torch.randn(e, generator=g, device="cuda")
        s["logits"] = torch.randn(t, e, generator=g, device="cuda") + liking
        if case["masked"]:   # experts that a token may not choose
            out = torch.rand(t, e, generator=g, device="cuda") < 0.2
            s["logits"] = torch.where(out, -math.inf, s["logits"])
        if op == "route":
            s["bias"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        else:
            chosen = torch.sort(s["logits"], dim=1, descending=True, stable=True)
            ids = chosen.indices[:, :top]
            kept = chosen.values[:, :top] > -math.inf
            s["experts"] = torch.where(kept, ids, -1).to(torch.int32)
            s["weights"] = _route_weights(case, s["logits"], s["experts"]).float()
            s["dw"] = torch.randn(t, top, generator=g, device="cuda")
        return s
    if op in ("norm", "norm_backward"):
        t, h, pad = case["t"], case["h"], case["pad"]
        s["x"] = _matrix(g, t, h, 1.5, pad)
        s["x"] += 0.3 * torch.randn(t, 1, generator=g, device="cuda")
        s["w"] = 1 + 0.1 * _matrix(g, 1, h)[0] if case["affine"] else None
        s["b"] = 0.1 * _matrix(g, 1, h)[0] if case["affine"] else None
        if op == "norm_backward":
            s["dy"] = _matrix(g, t, h, 1.0, pad)
            s["residual"] = _matrix(g, t, h, 1.0, pad) if case["residual"] else None
            s["mean"], s["rstd"] = _norm_stats(s["x"])
            s["ws"] = torch.empty(WORKSPACE_BYTES // 4, device="cuda")
        return s
    t, h, v, pad = case["t"], case["h"], case["v"], case["pad"]
    s["x"] = _matrix(g, t, h, 1.0, pad)
    s["b"] = _matrix(g, *((v, h) if case["tb"] else (h, v)), 2.0 * h ** -0.5, pad)
    s["targets"] = torch.randint(0, v, (t,), generator=g, device="cuda")
    if case["ignored"]:
        at = torch.randperm(t, generator=g, device="cuda")[:case["ignored"]]
        s["targets"][at] = -100
    s["ws"] = torch.empty(WORKSPACE_BYTES // 4, device="cuda")
    if op == "loss_backward":
        s["lse"] = _logits_lse(s)[1]
        counted = t - case["ignored"]
        s["dloss"] = torch.full((t,), 1.0 / max(counted, 1), device="cuda")
    return s


# The plain forms

def _route_scores(case, logits):
    """Scores in 64 bits: the choice compares values that may be next to each other."""
    x = logits.double()
    if case["scoring"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    return p / p.sum(1, keepdim=True)


def _route_weights(case, logits, experts):
    s = _route_scores(case, logits)
    kept = experts >= 0
    w = torch.where(kept, s.gather(1, experts.clamp(min=0).long()), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return case["scale"] * w


def _route(s):
    c = s["case"]
    t, e, top, groups = c["t"], c["e"], c["top"], c["groups"]
    choice = _route_scores(c, s["logits"])
    if s["bias"] is not None:
        choice = choice + s["bias"]
    choice = torch.where(s["logits"] > -math.inf, choice, -math.inf)
    if groups > 1:
        best = torch.sort(choice.reshape(t, groups, -1), dim=2, descending=True).values
        best = best[:, :, :c["group_best"]]
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, -math.inf)
        order = torch.sort(total, dim=1, descending=True, stable=True).indices
        stays = torch.zeros(t, groups, dtype=torch.bool, device=choice.device)
        stays.scatter_(1, order[:, :c["top_groups"]], True)
        choice = torch.where(stays.repeat_interleave(e // groups, 1), choice, -math.inf)
    found = torch.sort(choice, dim=1, descending=True, stable=True)
    ids = found.indices[:, :top]
    experts = torch.where(found.values[:, :top] > -math.inf, ids, -1).to(torch.int32)
    return {"experts": experts, "weights": _route_weights(c, s["logits"], experts).float()}


def _route_backward(s):
    c = s["case"]
    kept = s["experts"] >= 0
    ids = s["experts"].clamp(min=0).long()
    dw = torch.where(kept, s["dw"], 0.0)
    back = torch.zeros_like(s["logits"])
    if c["renorm"]:
        d = s["weights"] * (dw - (dw * s["weights"]).sum(1, keepdim=True) / c["scale"])
        if c["scoring"] == "sigmoid":
            d = d * (1 / (1 + torch.exp(s["logits"].gather(1, ids))))
        return {"dlogits": back.scatter_add_(1, ids, torch.where(kept, d, 0.0))}
    back.scatter_add_(1, ids, c["scale"] * dw)
    if c["scoring"] == "sigmoid":
        p = 1 / (1 + torch.exp(-s["logits"]))
        return {"dlogits": back * p * (1 - p)}
    top = s["logits"].amax(1, keepdim=True)
    p = torch.exp(s["logits"] - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    return {"dlogits": p * (back - (back * p).sum(1, keepdim=True))}


def _norm_stats(x):
    mean = x.sum(1) / x.shape[1]
    off = x - mean.unsqueeze(1)
    return mean, 1 / torch.sqrt((off * off).sum(1) / x.shape[1] + EPS)


def _logits_lse(s):
    z = torch.matmul(s["x"], s["b"].t() if s["case"]["tb"] else s["b"])
    top = z.amax(1, keepdim=True)
    return z, (top + torch.log(torch.exp(z - top).sum(1, keepdim=True))).squeeze(1)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        return _route(s)
    if op == "route_backward":
        return _route_backward(s)
    if op == "norm":
        mean, rstd = _norm_stats(s["x"])
        y = (s["x"] - mean.unsqueeze(1)) * rstd.unsqueeze(1)
        if s["w"] is not None:
            y = y * s["w"] + s["b"]
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        rstd = s["rstd"].unsqueeze(1)
        xh = (s["x"] - s["mean"].unsqueeze(1)) * rstd
        g = s["dy"] if s["w"] is None else s["dy"] * s["w"]
        h = c["h"]
        dx = rstd * (g - g.sum(1, keepdim=True) / h - xh * ((g * xh).sum(1, keepdim=True) / h))
        if s["residual"] is not None:
            dx = dx + s["residual"]
        return {"dx": dx, "dw": (s["dy"] * xh).sum(0), "db": s["dy"].sum(0)}
    kept = s["targets"] >= 0
    at = s["targets"].clamp(min=0).unsqueeze(1)
    if op == "loss":
        z, lse = _logits_lse(s)
        return {"loss": torch.where(kept, lse - z.gather(1, at).squeeze(1), 0.0),
                "lse": torch.where(kept, lse, 0.0)}
    z = torch.matmul(s["x"], s["b"].t() if c["tb"] else s["b"])
    g = torch.where(kept, s["dloss"], 0.0).unsqueeze(1)
    dz = torch.exp(z - s["lse"].unsqueeze(1)) * g
    dz.scatter_add_(1, at, -g)
    if c["tb"]:
        return {"da": torch.matmul(dz, s["b"]), "db": torch.matmul(dz.t(), s["x"])}
    return {"da": torch.matmul(dz, s["b"].t()), "db": torch.matmul(s["x"].t(), dz)}


# The library's calls

def _own(s):
    import tiled_fp32_gemm_amd as sg
    c = s["case"]
    op = c["op"]
    if op == "route":
        experts, weights = sg.moe_route(
            s["logits"], c["top"], c["scoring"], s["bias"], groups=c["groups"],
            top_groups=c["top_groups"], group_best=c["group_best"], renormalize=c["renorm"],
            scale=c["scale"])
        return {"experts": experts, "weights": weights}
    if op == "route_backward":
        return {"dlogits": sg.moe_route_backward(s["dw"], s["logits"], s["experts"], s["weights"],
                                                 c["scoring"], renormalize=c["renorm"],
                                                 scale=c["scale"])}
    if op == "norm":
        mean, rstd = (torch.empty(c["t"], device="cuda") for _ in range(2))
        y = sg.layer_norm(s["x"], s["w"], s["b"], EPS, mean=mean, rstd=rstd)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dx, dw, db = sg.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"],
                                            s["residual"], workspace=s["ws"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "loss":
        lse = torch.empty(c["t"], device="cuda")
        loss = sg.linear_cross_entropy(s["x"], s["b"], s["targets"], transpose_b=c["tb"], lse=lse,
                                       workspace=s["ws"])
        return {"loss": loss, "lse": lse}
    da, db = sg.linear_cross_entropy_backward(s["dloss"], s["x"], s["b"], s["targets"], s["lse"],
                                              transpose_b=c["tb"], workspace=s["ws"])
    return {"da": da, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, t = case["op"], case["t"]
    if op in ("route", "route_backward"):
        e, top = case["e"], case["top"]
        if op == "route":
            return {"bytes": 4 * t * e + 4 * e * case["bias"] + 8 * t * top, "flops": 4 * t * e}
        whole = case["scoring"] == "softmax" and not case["renorm"]
        read = 4 * t * e if whole else 4 * t * top * (case["scoring"] == "sigmoid")
        return {"bytes": 4 * t * e + read + 4 * t * top * (2 + case["renorm"]),
                "flops": 4 * t * e if whole else 4 * t * top}
    if op in ("norm", "norm_backward"):
        h, a = case["h"], case["affine"]
        if op == "norm":
            return {"bytes": 4 * (2 * t * h + 2 * t + 2 * h * a), "flops": 7 * t * h}
        return {"bytes": 4 * (t * h * (3 + case["residual"]) + 2 * t + h * (2 + a)),
                "flops": 14 * t * h}
    h, v, n = case["h"], case["v"], case["t"] - case["ignored"]
    if op == "loss":
        return {"bytes": 4 * (n * h + h * v + 2 * t) + 8 * t, "flops": 2 * n * v * h}
    return {"bytes": 4 * (n * h + t * h + 2 * h * v + 2 * n) + 8 * t, "flops": 6 * n * v * h}


# The same in 64 bits, from the definitions

def _exact_route(case, s):
    t, e, top = case["t"], case["e"], case["top"]
    x = s["logits"].double()
    if case["op"] == "route_backward":
        experts = s["experts"].long()
    else:
        # For each token the experts by rank: how many others come before it.
        score = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
        score = score.nan_to_num(0.0) + (0 if s["bias"] is None else s["bias"].double())
        score = score.masked_fill(x == -math.inf, -math.inf)
        if case["groups"] > 1:
            in_group = score.view(t, case["groups"], -1)
            best = torch.topk(in_group, case["group_best"], dim=2).values
            group = best.masked_fill(best == -math.inf, 0.0).sum(2)
            group = group.masked_fill((in_group == -math.inf).all(2), -math.inf)
            last = torch.topk(group, case["top_groups"], dim=1).values[:, -1:]
            keep = (group >= last).unsqueeze(2).expand_as(in_group).reshape(t, e)
            score = score.masked_fill(~keep, -math.inf)
        best, experts = torch.topk(score, top, dim=1)
        experts = experts.masked_fill(best == -math.inf, -1)
    some = experts >= 0
    at = torch.where(some, experts, 0)
    picked = x.gather(1, at).masked_fill(~some, -math.inf)
    logp = torch.nn.functional.logsigmoid(picked) if case["scoring"] == "sigmoid" \
        else picked - torch.logsumexp(x, 1, keepdim=True)
    logp = logp.masked_fill(~some, -math.inf)
    w = torch.softmax(logp, 1) if case["renorm"] else torch.exp(logp)
    w = w.masked_fill(~some, 0.0) * case["scale"]
    if case["op"] == "route":
        return {"experts": None, "weights": w}
    dw = s["dw"].double().masked_fill(~some, 0.0)
    if case["renorm"]:
        w = s["weights"].double()      # as handed to the call
    dlogp = w * dw
    if case["renorm"]:
        dlogp = dlogp - w / case["scale"] * dlogp.sum(1, keepdim=True)
    if case["scoring"] == "sigmoid":
        dlogp = dlogp * torch.sigmoid(-picked)
    dlogp = dlogp.masked_fill(~some, 0.0)
    dx = torch.zeros_like(x).scatter_add_(1, at, dlogp)
    if case["scoring"] == "softmax" and not case["renorm"]:
        dx -= torch.softmax(x, 1).nan_to_num(0.0) * dlogp.sum(1, keepdim=True)
    return {"dlogits": dx}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_backward"):
        return _exact_route(case, s)
    if op in ("norm", "norm_backward"):
        x, h = s["x"].double(), case["h"]
        w = s["w"].double() if case["affine"] else torch.ones(h, device="cuda").double()
        if op == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS).rsqrt()
            b = s["b"].double() if case["affine"] else 0
            return {"y": torch.addcmul(-mean * rstd, x.t(), rstd).t() * w + b, "mean": mean,
                    "rstd": rstd}
        mean, rstd, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
        xh = ((x.t() - mean) * rstd).t()
        g = dy * w
        along = torch.einsum("th,th->t", g, xh) / h
        dx = ((g.t() - g.mean(1) - xh.t() * along) * rstd).t()
        if case["residual"]:
            dx = dx + s["residual"].double()
        return {"dx": dx, "dw": torch.einsum("th,th->h", dy, xh), "db": dy.sum(0)}
    x, targets = s["x"].double(), s["targets"]
    b = s["b"].double().t() if case["tb"] else s["b"].double()
    z = x @ b
    rows = torch.nonzero(targets >= 0).squeeze(1)
    if op == "loss":
        loss, lse = (torch.zeros(case["t"], device="cuda", dtype=torch.float64) for _ in range(2))
        lse[rows] = torch.logsumexp(z[rows], 1)
        loss[rows] = lse[rows] - z[rows, targets[rows]]
        return {"loss": loss, "lse": lse}
    dz = torch.zeros_like(z)
    dz[rows] = torch.exp(z[rows] - s["lse"].double()[rows].unsqueeze(1))
    dz[rows, targets[rows]] -= 1
    dz *= s["dloss"].double().unsqueeze(1)
    db = x.t() @ dz
    return {"da": dz @ b.t(), "db": db.t() if case["tb"] else db}
