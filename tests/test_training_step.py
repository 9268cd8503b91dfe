"""A layer of experts trained with its loss, by the library's calls alone: norm,
router, routing, the experts' products, norm and cross entropy over a vocabulary,
and every gradient back to the input, against 64-bit autograd.

Tolerance: every sum here has at most 200 terms, so it is within S(200) = 203 u of
its terms' sizes; twelve such stages follow each other there and back, over values
of about unit size, and the weights' norms (up to 2) let an error grow about
fourfold: 10^4 u of a result's largest value bounds them all.
"""
from __future__ import annotations

import pytest

import tiled_fp32_gemm_amd as sg
from test_linear import U, gen
from test_route import choose64

torch = pytest.importorskip("torch")

T, H, F, E, TOP, V = 190, 96, 72, 12, 3, 200
ROUTER = dict(groups=4, top_groups=2, group_best=2)
SCALE = 1.5


def parameters(g):
    r = lambda *s, scale=1.0: scale * torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return {"w1": 1 + r(H, scale=0.1), "b1": r(H, scale=0.1), "wr": r(E, H, scale=H ** -0.5),
            "W1": r(E, H, F, scale=H ** -0.5), "c1": r(E, F, scale=0.1),
            "W2": r(E, H, F, scale=F ** -0.5), "c2": r(E, H, scale=0.1),
            "w2": 1 + r(H, scale=0.1), "b2": r(H, scale=0.1), "wv": r(V, H, scale=H ** -0.5)}


def step(x, p, balance, targets, dloss, ws):
    """The loss of every token, the choices, and the gradients of x and p."""
    stats = [torch.empty(T, device="cuda") for _ in range(5)]
    mean1, rstd1, mean2, rstd2, lse = stats
    h1 = sg.layer_norm(x, p["w1"], p["b1"], mean=mean1, rstd=rstd1)
    logits = sg.linear(h1, p["wr"], transpose_b=True, workspace=ws)
    experts, weights = sg.moe_route(logits, TOP, "sigmoid", balance, scale=SCALE, **ROUTER)
    offsets, _, place = sg.moe_sort(experts, E, workspace=ws)
    xp = sg.moe_permute(h1, place)
    z = torch.empty(T * TOP, F, device="cuda")
    up = sg.grouped_linear(xp, p["W1"], offsets, p["c1"], "silu", preact=z, workspace=ws)
    yp = sg.grouped_linear(up, p["W2"], offsets, p["c2"], transpose_b=True, workspace=ws)
    x2 = x + sg.moe_unpermute(yp, place, weights)
    h2 = sg.layer_norm(x2, p["w2"], p["b2"], mean=mean2, rstd=rstd2)
    loss = sg.linear_cross_entropy(h2, p["wv"], targets, transpose_b=True, lse=lse, workspace=ws)

    d = {}
    dh2, d["wv"] = sg.linear_cross_entropy_backward(dloss, h2, p["wv"], targets, lse,
                                                    transpose_b=True, workspace=ws)
    dx2, d["w2"], d["b2"] = sg.layer_norm_backward(dh2, x2, mean2, rstd2, p["w2"], workspace=ws)
    dyp, dweights = sg.moe_unpermute_backward(dx2, yp, place, weights)
    dup, d["W2"], d["c2"] = sg.grouped_linear_backward(dyp, up, p["W2"], offsets,
                                                       transpose_b=True, workspace=ws)
    dxp, d["W1"], d["c1"] = sg.grouped_linear_backward(dup, xp, p["W1"], offsets, "silu", z,
                                                       workspace=ws)
    dlogits = sg.moe_route_backward(dweights, logits, experts, weights, "sigmoid", scale=SCALE)
    dh1, d["wr"], _ = sg.linear_backward(dlogits, h1, p["wr"], transpose_b=True, bias_grad=False,
                                         workspace=ws)
    dh1 = dh1 + sg.moe_unpermute(dxp, place)
    d["x"], d["w1"], d["b1"] = sg.layer_norm_backward(dh1, x, mean1, rstd1, p["w1"], dx2,
                                                      workspace=ws)
    return loss, experts, logits, d


def plain(x, p, targets, experts):
    """The losses by the definitions, the choices given."""
    def norm(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w + b

    h1 = norm(x, p["w1"], p["b1"])
    s = torch.sigmoid(h1 @ p["wr"].t()).gather(1, experts)
    weights = SCALE * s / s.sum(1, keepdim=True)
    y = 0
    for j in range(TOP):
        e = experts[:, j]
        z = torch.bmm(h1[:, None], p["W1"][e])[:, 0] + p["c1"][e]
        out = torch.bmm(p["W2"][e], (z * torch.sigmoid(z))[:, :, None])[:, :, 0] + p["c2"][e]
        y = y + weights[:, j, None] * out
    z = norm(x + y, p["w2"], p["b2"]) @ p["wv"].t()
    kept = targets >= 0
    hit = z.gather(1, targets.clamp(min=0)[:, None]).squeeze(1)
    return torch.where(kept, torch.logsumexp(z, 1) - hit, 0.0)


@pytest.mark.gpu
def test_a_training_step_of_a_layer_of_experts():
    g = gen(41)
    p = parameters(g)
    x = torch.randn(T, H, device="cuda", generator=g)
    balance = 0.05 * torch.randn(E, device="cuda", generator=g)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    targets[::7] = -100
    dloss = torch.rand(T, device="cuda", generator=g)
    ws = torch.empty(1 << 22, device="cuda")
    loss, experts, logits, d = step(x, p, balance, targets, dloss, ws)
    assert torch.equal(experts.cpu(), choose64(logits, TOP, "sigmoid", balance, **ROUTER))
    leaves = {k: v.double().cpu().requires_grad_() for k, v in (p | {"x": x}).items()}
    want = plain(leaves["x"], leaves, targets.cpu(), experts.cpu().long())
    near = lambda a, b: (a.double().cpu() - b).abs().max() <= 1e4 * U * b.abs().max()  # noqa: E731
    assert near(loss, want)
    (want * dloss.double().cpu()).sum().backward()
    for k, v in leaves.items():
        assert near(d[k], v.grad), k

    # captured, and replayed with other tokens, targets and gradients
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, p, balance, targets, dloss, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, p, balance, targets, dloss, ws)
    for rep in range(4):
        x.normal_(generator=g)
        targets.random_(-V // 4, V, generator=g)
        dloss.uniform_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        got = [out[0].clone(), out[1].clone()] + [t.clone() for t in out[3].values()]
        again = step(x, p, balance, targets, dloss, ws)
        for a, b in zip(got, [again[0], again[1]] + list(again[3].values())):
            assert torch.equal(a, b), rep
