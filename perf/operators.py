"""Timed cases of the library's language-model operators.

Three groups, all in float32 like the products they stand beside:

  linear            C = act(A.B + bias) + residual, B as in x out or out x in
  linear_backward   its gradients: of A, of B and of the bias
  route             tokens sorted by expert, their rows gathered in that order,
                    and the experts' rows brought back with the router's weights
  route_backward    the gradients of both moves and of the weights
  experts           one product per expert over the sorted rows, same epilogue
  experts_backward  its gradients

``run`` computes a case with elementary torch operations; with ``own`` set it
makes the library's calls instead.
"""
import math

import torch

own = False

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
WORKSPACE_BYTES = 64 << 20      # what a program keeps for split sums


def listed():
    return [
        # one token of a decoder through a weight stored out x in
        {"name": "linear one row", "op": "linear", "m": 1, "n": 4096, "k": 4096, "tb": True,
         "act": "silu", "bias": True, "residual": False, "preact": False, "pad": False},
        # a small product whose time is its launches
        {"name": "linear 256 cube", "op": "linear", "m": 256, "n": 256, "k": 256, "tb": False,
         "act": "gelu", "bias": True, "residual": True, "preact": False, "pad": False},
        # a prompt of odd length through odd widths, kept for training
        {"name": "linear ragged", "op": "linear", "m": 1000, "n": 1500, "k": 777, "tb": False,
         "act": "gelu_tanh", "bias": True, "residual": True, "preact": True, "pad": False},
        # the feed-forward of a long prompt, kept for training
        {"name": "linear 4096 cube", "op": "linear", "m": 4096, "n": 4096, "k": 4096, "tb": False,
         "act": "gelu", "bias": True, "residual": True, "preact": True, "pad": False},
        # many tokens and narrow widths: the weight's gradient is one long sum
        {"name": "linear backward skinny", "op": "linear_backward", "m": 65536, "n": 128, "k": 256,
         "tb": False, "act": "silu", "pad": False},
        # the gradients of a full feed-forward
        {"name": "linear backward 4096 cube", "op": "linear_backward", "m": 4096, "n": 4096,
         "k": 4096, "tb": True, "act": "gelu", "pad": False},
        # a decoding batch choosing two of eight experts
        {"name": "route 16 tokens", "op": "route", "t": 16, "top": 2, "e": 8, "h": 1024,
         "drop": False},
        # a training batch choosing four of sixty-four, some choices dropped
        {"name": "route 32768 tokens", "op": "route", "t": 32768, "top": 4, "e": 64, "h": 1024,
         "drop": True},
        # the gradients of a batch of odd sizes
        {"name": "route backward 8191 tokens", "op": "route_backward", "t": 8191, "top": 2, "e": 16,
         "h": 777, "drop": True},
        # that decoding batch through its experts
        {"name": "experts 32 rows", "op": "experts", "rows": 32, "e": 8, "n": 4096, "k": 1024,
         "tb": False, "act": "silu", "bias": True, "preact": False},
        # a training batch through sixteen experts
        {"name": "experts 16384 rows", "op": "experts", "rows": 16384, "e": 16, "n": 4096,
         "k": 1024, "tb": False, "act": "gelu", "bias": True, "preact": True},
        # the gradients through experts of odd widths
        {"name": "experts backward 8190 rows", "op": "experts_backward", "rows": 8190, "e": 16,
         "n": 1500, "k": 777, "tb": False, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_backward", "route", "route_backward", "experts",
                     "experts_backward"])
    act = rng.choice(ACTIVATIONS)
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("linear", "linear_backward"):
        if rng.random() < 0.2:
            m, n, k = _log(rng, 4096, 65536), _log(rng, 16, 512), _log(rng, 16, 512)
        else:
            m, n, k = _log(rng, 1, 4096), _log(rng, 16, 4096), _log(rng, 16, 4096)
        c = {"op": op, "m": m, "n": n, "k": k, "tb": yes(), "act": act, "pad": yes()}
        if op == "linear":
            c |= {"bias": yes(), "residual": yes(), "preact": yes()}
        return c
    e = _log(rng, 2, 64)
    if op in ("route", "route_backward"):
        top = rng.randint(1, min(8, e))
        h = _log(rng, 16, 2048)
        t = _log(rng, 1, max(1, min(32768, 100_000_000 // (top * h))))
        return {"op": op, "t": t, "top": top, "e": e, "h": h, "drop": yes()}
    n, k = _log(rng, 16, 2048), _log(rng, 16, 2048)
    c = {"op": op, "rows": _log(rng, 1, 16384), "e": e, "n": n, "k": k, "tb": yes(), "act": act}
    if op == "experts":
        c |= {"bias": yes(), "preact": yes()}
    return c


# Inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _matrix(g, rows, cols, scale=1.0, pad=False):
    """rows x cols values; with `pad`, inside a wider buffer."""
    wide = torch.randn(rows, cols + (3 if pad else 0), generator=g, device="cuda")
    return wide.mul_(scale)[:, :cols]


def _counts(rows, e, seed):
    """How many of `rows` each expert gets: uneven, as a router's choices are."""
    g = torch.Generator().manual_seed(int(seed) * 3 + 1)
    p = torch.softmax(0.4 * torch.randn(e, generator=g), 0)
    got = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(got, minlength=e)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case, "ws": torch.empty(WORKSPACE_BYTES // 4, device="cuda")}
    if op in ("linear", "linear_backward"):
        m, n, k, pad = case["m"], case["n"], case["k"], case["pad"]
        s["a"] = _matrix(g, m, k, 1.0, pad)
        s["b"] = _matrix(g, *((n, k) if case["tb"] else (k, n)), k ** -0.5, pad)
        if op == "linear":
            s["bias"] = _matrix(g, 1, n, 0.1)[0] if case["bias"] else None
            s["residual"] = _matrix(g, m, n, 1.0, pad) if case["residual"] else None
        else:
            s["z"] = _matrix(g, m, n, 1.0, pad)
            s["dc"] = _matrix(g, m, n, 1.0, pad)
        return s
    if op in ("route", "route_backward"):
        t, top, e, h = case["t"], case["top"], case["e"], case["h"]
        bias = 0.5 * torch.randn(e, generator=g, device="cuda")
        scores = torch.randn(t, e, generator=g, device="cuda") + bias
        best, ids = torch.topk(scores, top, dim=1)
        if case["drop"]:   # choices past an expert's capacity
            ids = torch.where(torch.rand(t, top, generator=g, device="cuda") < 0.03, -1, ids)
        s["ids"], s["w"] = ids.contiguous(), torch.softmax(best, 1).contiguous()
        s["yp"] = _matrix(g, t * top, h)
        if op == "route":
            s["x"] = _matrix(g, t, h)
            s["xp"] = torch.zeros(t * top, h, device="cuda")
        else:
            s["dy"] = _matrix(g, t, h)
            s["dxp"] = _matrix(g, t * top, h)
            s["dyp"] = torch.zeros(t * top, h, device="cuda")
            s["place"] = _sorted(s["ids"], e)[2]
        return s
    rows, e, n, k = case["rows"], case["e"], case["n"], case["k"]
    counts = _counts(rows, e, seed)
    s["longest"] = int(counts.max())    # the padded length a batched product needs
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(
        torch.int32).cuda()
    s["a"] = _matrix(g, rows, k)
    s["b"] = (torch.randn(e, *((n, k) if case["tb"] else (k, n)), generator=g, device="cuda")
              .mul_(k ** -0.5))
    if op == "experts":
        s["bias"] = _matrix(g, e, n, 0.1) if case["bias"] else None
    else:
        s["z"], s["dc"] = _matrix(g, rows, n), _matrix(g, rows, n)
    return s


# The plain forms

def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
                + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _sorted(ids, e):
    """Where each expert's rows begin, the choices in expert order (ties in
    token order, dropped ones last as -1) and each choice's place."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < e), flat, e)
    keys, at = torch.sort(key, stable=True)
    ends = torch.bincount(key, minlength=e + 1).cumsum(0)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = ends[:e]
    order = torch.where(keys < e, at, -1).to(torch.int32)
    place = torch.empty_like(flat)
    place[at] = torch.arange(flat.numel(), device=ids.device)
    place = torch.where(key < e, place, -1).to(torch.int32).reshape(ids.shape)
    return offsets, order, place


def _back(rows, place, w=None):
    """Each token's rows summed, times its weights."""
    kept = (place >= 0).to(rows.dtype)
    w = kept if w is None else torch.where(place >= 0, w, 0.0)
    return (rows[place.clamp(min=0).long()] * w.unsqueeze(2)).sum(1)


def _row_experts(offsets, rows):
    """Each row's expert and its position among that expert's rows."""
    r = torch.arange(rows, device=offsets.device, dtype=offsets.dtype)
    of = torch.searchsorted(offsets[1:].contiguous(), r, right=True)
    return of, r - offsets[of]


def _padded(x, offsets, longest):
    """The rows of every expert as one e x longest batch, zeros behind them."""
    at = torch.arange(longest, device=x.device)
    i = offsets[:-1].unsqueeze(1) + at
    inside = i < offsets[1:].unsqueeze(1)
    return torch.where(inside.unsqueeze(2), x[i.clamp(max=x.shape[0] - 1)], 0.0)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear":
        z = torch.matmul(s["a"], s["b"].t() if c["tb"] else s["b"])
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(c["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"]
        return {"c": y, "z": z} if c["preact"] else {"c": y}
    if op == "linear_backward":
        dz = s["dc"] * _act_slope(c["act"], s["z"])
        if c["tb"]:
            return {"da": torch.matmul(dz, s["b"]), "db": torch.matmul(dz.t(), s["a"]),
                    "dbias": dz.sum(0)}
        return {"da": torch.matmul(dz, s["b"].t()), "db": torch.matmul(s["a"].t(), dz),
                "dbias": dz.sum(0)}
    if op == "route":
        offsets, order, place = _sorted(s["ids"], c["e"])
        kept = (order >= 0).unsqueeze(1)
        rows = s["x"][order.clamp(min=0).long() // c["top"]]
        return {"offsets": offsets, "order": order, "place": place,
                "xp": torch.where(kept, rows, s["xp"]), "y": _back(s["yp"], place, s["w"])}
    if op == "route_backward":
        place, h = s["place"].long(), c["h"]
        kept = place >= 0
        to = torch.where(kept, place, place.numel()).reshape(-1)
        dyp = torch.cat([s["dyp"], s["dyp"][:1]])    # one row more, for dropped choices
        dyp[to] = (s["w"].unsqueeze(2) * s["dy"].unsqueeze(1)).reshape(-1, h)
        dw = (s["yp"][place.clamp(min=0)] * s["dy"].unsqueeze(1)).sum(2)
        return {"dyp": dyp[:-1], "dw": torch.where(kept, dw, 0.0), "dx": _back(s["dxp"], place)}
    of, at = _row_experts(s["offsets"], c["rows"])
    if op == "experts":
        b = s["b"].transpose(1, 2) if c["tb"] else s["b"]
        z = torch.bmm(_padded(s["a"], s["offsets"], s["longest"]), b)[of, at]
        if s["bias"] is not None:
            z = z + s["bias"][of]
        y = _act(c["act"], z)
        return {"c": y, "z": z} if c["preact"] else {"c": y}
    dz = _padded(s["dc"] * _act_slope(c["act"], s["z"]), s["offsets"], s["longest"])
    a = _padded(s["a"], s["offsets"], s["longest"])
    if c["tb"]:
        return {"da": torch.bmm(dz, s["b"])[of, at], "db": torch.bmm(dz.transpose(1, 2), a),
                "dbias": dz.sum(1)}
    return {"da": torch.bmm(dz, s["b"].transpose(1, 2))[of, at],
            "db": torch.bmm(a.transpose(1, 2), dz), "dbias": dz.sum(1)}


# The library's calls

def _own(s):
    import tiled_fp32_gemm_amd as sg
    c = s["case"]
    op = c["op"]
    if op == "linear":
        z = torch.empty(c["m"], c["n"], device="cuda") if c["preact"] else None
        y = sg.linear(s["a"], s["b"], s["bias"], c["act"], s["residual"], transpose_b=c["tb"],
                      preact=z, workspace=s["ws"])
        return {"c": y, "z": z} if c["preact"] else {"c": y}
    if op == "linear_backward":
        da, db, dbias = sg.linear_backward(s["dc"], s["a"], s["b"], c["act"], s["z"],
                                           transpose_b=c["tb"], workspace=s["ws"])
        return {"da": da, "db": db, "dbias": dbias}
    if op == "route":
        offsets, order, place = sg.moe_sort(s["ids"], c["e"], workspace=s["ws"])
        xp = sg.moe_permute(s["x"], place, out=s["xp"])
        return {"offsets": offsets, "order": order, "place": place, "xp": xp,
                "y": sg.moe_unpermute(s["yp"], place, s["w"])}
    if op == "route_backward":
        dyp, dw = sg.moe_unpermute_backward(s["dy"], s["yp"], s["place"], s["w"], out=s["dyp"])
        return {"dyp": dyp, "dw": dw, "dx": sg.moe_unpermute(s["dxp"], s["place"])}
    if op == "experts":
        z = torch.empty(c["rows"], c["n"], device="cuda") if c["preact"] else None
        y = sg.grouped_linear(s["a"], s["b"], s["offsets"], s["bias"], c["act"],
                              transpose_b=c["tb"], preact=z, workspace=s["ws"])
        return {"c": y, "z": z} if c["preact"] else {"c": y}
    da, db, dbias = sg.grouped_linear_backward(s["dc"], s["a"], s["b"], s["offsets"], c["act"],
                                               s["z"], transpose_b=c["tb"], workspace=s["ws"])
    return {"da": da, "db": db, "dbias": dbias}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "linear":
            outs = m * n * (1 + case["residual"] + case["preact"]) + n * case["bias"]
            return {"bytes": 4 * (m * k + k * n + outs), "flops": 2 * m * n * k}
        return {"bytes": 4 * (2 * m * n + 2 * m * k + 2 * k * n + n), "flops": 4 * m * n * k}
    if op in ("route", "route_backward"):
        t, top, e, h = case["t"], case["top"], case["e"], case["h"]
        if op == "route":
            return {"bytes": t * top * (8 + 4 + 4 + 4) + 4 * (e + 1) + 8 * t * h * (1 + top),
                    "flops": 2 * t * top * h}
        return {"bytes": t * top * 12 + 4 * t * h * (2 + 3 * top), "flops": 4 * t * top * h}
    rows, e, n, k = case["rows"], case["e"], case["n"], case["k"]
    if op == "experts":
        # no more experts' weights than there are rows
        outs = rows * n * (1 + case["preact"]) + min(e, rows) * n * case["bias"]
        return {"bytes": 4 * (rows * k + min(e, rows) * k * n + outs), "flops": 2 * rows * n * k}
    return {"bytes": 4 * (2 * rows * n + 2 * rows * k + (min(e, rows) + e) * k * n + e * n),
            "flops": 4 * rows * n * k}


# The same in 64 bits, from the definitions

def _phi(name, z):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), z.gt(0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
    p = torch.sigmoid(2 * u)      # (1 + tanh u) / 2
    du = math.sqrt(2 / math.pi) * (1 + 0.134145 * z.square())
    return z * p, p + z * 2 * p * (1 - p) * du


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() and k != "ws" else v
         for k, v in s.items()}
    op = case["op"]
    if op in ("linear", "linear_backward"):
        b = s["b"].t() if case["tb"] else s["b"]
        if op == "linear":
            z = s["a"] @ b + (s["bias"] if case["bias"] else 0)
            y = _phi(case["act"], z)[0] + (s["residual"] if case["residual"] else 0)
            return {"c": y, "z": z} if case["preact"] else {"c": y}
        dz = s["dc"] * _phi(case["act"], s["z"])[1]
        db = s["a"].t() @ dz
        return {"da": dz @ b.t(), "db": db.t() if case["tb"] else db, "dbias": dz.sum(0)}
    if op in ("route", "route_backward"):
        t, top, e, h = case["t"], case["top"], case["e"], case["h"]
        ids = s["ids"].reshape(-1).tolist()
        where = [[] for _ in range(e)]
        for i, x in enumerate(ids):
            if 0 <= x < e:
                where[x].append(i)
        order = torch.tensor([i for w in where for i in w], device="cuda", dtype=torch.int64)
        kept = order.numel()
        tok, w = order // top, s["w"].reshape(-1)[order].unsqueeze(1)
        if op == "route":
            y = torch.zeros(t, h, device="cuda", dtype=torch.float64)
            y.index_add_(0, tok, w * s["yp"][:kept])
            s["xp"][:kept] = s["x"][tok]
            return {"offsets": None, "order": None, "place": None, "xp": s["xp"], "y": y}
        dx = torch.zeros(t, h, device="cuda", dtype=torch.float64)
        dx.index_add_(0, tok, s["dxp"][:kept])
        s["dyp"][:kept] = w * s["dy"][tok]
        dw = torch.zeros(t * top, device="cuda", dtype=torch.float64)
        dw[order] = (s["dy"][tok] * s["yp"][:kept]).sum(1)
        return {"dyp": s["dyp"], "dw": dw.reshape(t, top), "dx": dx}
    edges = s["offsets"].tolist()
    parts = []
    for e, (i, j) in enumerate(zip(edges, edges[1:])):
        b = s["b"][e].t() if case["tb"] else s["b"][e]
        if op == "experts":
            z = s["a"][i:j] @ b + (s["bias"][e] if case["bias"] else 0)
            parts.append((_phi(case["act"], z)[0], z))
        else:
            dz = s["dc"][i:j] * _phi(case["act"], s["z"][i:j])[1]
            db = s["a"][i:j].t() @ dz
            parts.append((dz @ b.t(), db.t() if case["tb"] else db, dz.sum(0)))
    if op == "experts":
        y, z = (torch.cat(p) for p in zip(*parts))
        return {"c": y, "z": z} if case["preact"] else {"c": y}
    da, db, dbias = zip(*parts)
    return {"da": torch.cat(da), "db": torch.stack(db), "dbias": torch.stack(dbias)}
