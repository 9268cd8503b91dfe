"""A router's choice of experts, its weights and their gradient, against the
definition in 64 bits.  The ids have to be equal.

Tolerances of the weights, relative, from FP32 arithmetic (u = 2^-24): an
exponential is within 8 u and its argument's rounding, u times the distance d from
the largest logit; a softmax's sum adds 31 u and the same of its terms, a quotient
or reciprocal 3 u, the scale u; a sum over the chosen 32 u.
  softmax              (d + 48) u          softmax, renormalised   (d + D + 64) u
  sigmoid              16 u                sigmoid, renormalised   (d + D + 80) u
with D the largest d of the chosen.  The gradients multiply such weights by
differences of sums of at most 32 terms: the bounds above, and 48 u more, over the
terms' sizes.
"""
from __future__ import annotations

import pytest

import tiled_fp32_gemm_amd as sg
from test_linear import U, gen, wide

torch = pytest.importorskip("torch")
INF = float("inf")


def scores64(x, scoring):
    x = x.double()
    if scoring == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top > -INF, top, 0.0))
    return p / p.sum(1, keepdim=True)


def choose64(x, top, scoring="softmax", bias=None, groups=1, top_groups=1, group_best=1):
    """Ids by exact scores: by the logits themselves where those say it."""
    x = x.cpu().double()
    T, E = x.shape
    c = x.clone()
    if bias is not None or (groups > 1 and group_best > 1):
        c = scores64(x, scoring)
        if bias is not None:
            c = c + bias.cpu().double()
    c = torch.where(c.isnan(), INF, c)
    c[x == -INF] = -INF
    if groups > 1:
        best = c.reshape(T, groups, -1).sort(dim=2, descending=True).values[:, :, :group_best]
        total = torch.where(best == -INF, 0.0, best).sum(2)
        total[best[:, :, 0] == -INF] = -INF
        order = total.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        stays = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, order, True)
        c[~stays.repeat_interleave(E // groups, 1)] = -INF
    v, ids = c.sort(dim=1, descending=True, stable=True)
    return torch.where(v[:, :top] == -INF, -1, ids[:, :top]).to(torch.int32)


def weights64(x, ids, scoring, renorm, scale):
    """The weights of given ids and their bounds."""
    kept = ids >= 0
    at = ids.clamp(min=0).long()
    l = x.double().gather(1, at)
    s = scores64(x, scoring).gather(1, at)
    s = torch.where(kept, s, 0.0)
    l = torch.where(kept, l, -INF)
    if renorm:
        if scoring == "softmax":
            most = l.amax(1, keepdim=True)
            s = torch.where(kept, torch.exp(l - torch.where(most > -INF, most, 0.0)), 0.0)
        else:
            lg = torch.nn.functional.logsigmoid(l)
            most = lg.amax(1, keepdim=True)
            s = torch.where(kept, torch.exp(lg - torch.where(most > -INF, most, 0.0)), 0.0)
        total = s.sum(1, keepdim=True)
        s = s / torch.where(total == 0, 1.0, total)
        d = torch.where(kept, l.amax(1, keepdim=True) - l, 0.0)
        rel = d + d.amax(1, keepdim=True) + (64 if scoring == "softmax" else 80)
    elif scoring == "softmax":
        rel = torch.where(kept, x.double().amax(1, keepdim=True) - l, 0.0) + 48
    else:
        rel = torch.full_like(s, 16.0)
    w = s * scale
    # below the normal numbers results are flushed
    return w, rel * U * w.abs() + 2.0 ** -126 * abs(scale)


def check(x, top, scoring="softmax", bias=None, renormalize=True, scale=1.0, **groups):
    ids, w = sg.moe_route(x, top, scoring, bias, renormalize=renormalize, scale=scale, **groups)
    assert ids.dtype is torch.int32 and ids.shape == w.shape == (x.shape[0], top)
    want = choose64(x, top, scoring, bias, **groups)
    assert torch.equal(ids.cpu(), want), (ids.cpu() != want).nonzero()[:4]
    w64, tol = weights64(x, ids, scoring, renormalize, scale)
    good = ((w.double() - w64).abs() <= tol) | (w64.isnan() & w.isnan())
    assert good.all(), ((w.double() - w64).abs() / tol).max().item()
    assert (w[ids < 0] == 0).all()
    return ids, w


SHAPES = [(1, 1, 1), (5, 2, 1), (5, 3, 2), (300, 4, 4), (1, 8, 2), (64, 8, 8), (65, 15, 3),
          (130, 16, 5), (33, 17, 1), (40, 32, 32), (100, 33, 9), (1000, 64, 6), (7, 65, 17),
          (50, 100, 8), (129, 128, 16), (2000, 160, 6), (3000, 256, 8), (31, 257, 4), (20, 300, 32),
          (100, 512, 10), (17, 513, 1), (90, 1000, 8), (70, 1024, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,top", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route(T, E, top, scoring):
    g = gen(T + E)
    for pad, off, bias, renorm, scale in ((0, 0, False, True, 1.0), (3, 1, True, True, 2.5),
                                          (1, 2, False, False, 1.0), (0, 0, True, False, -0.5)):
        x = wide(T, E, pad, off, g, 1.5)
        b = 0.1 * torch.randn(E, device="cuda", generator=g) if bias else None
        check(x, top, scoring, b, renorm, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,groups,top_groups,top", [
    (100, 8, 2, 1, 3), (77, 8, 8, 3, 3), (50, 12, 3, 2, 5), (300, 64, 4, 2, 8), (65, 96, 32, 5, 6),
    (400, 256, 8, 4, 8), (33, 160, 8, 3, 6), (40, 320, 16, 4, 12), (20, 1024, 32, 8, 32),
    (20, 1022, 7, 6, 9), (64, 30, 15, 4, 4), (9, 16, 2, 2, 16), (60, 96, 6, 4, 8),
    (31, 128, 32, 16, 20), (50, 512, 32, 1, 16), (45, 24, 6, 2, 8), (70, 64, 16, 1, 4),
    (33, 256, 8, 4, 32), (40, 1024, 16, 8, 32), (20, 480, 12, 5, 8), (66, 256, 32, 16, 1)])
@pytest.mark.parametrize("group_best", [1, 2])
def test_groups(T, E, groups, top_groups, top, group_best):
    if E // groups < group_best:
        group_best = 1
    kw = dict(groups=groups, top_groups=top_groups, group_best=group_best)
    g = gen(E + groups)
    for scoring in ("softmax", "sigmoid"):
        for biased in (False, True):
            x = torch.randn(T, E, device="cuda", generator=g)
            b = 0.2 * torch.randn(E, device="cuda", generator=g) if biased else None
            check(x, top, scoring, b, **kw)
            x[torch.rand(T, E, device="cuda", generator=g) < 0.5] = -INF
            x[0] = -INF
            x[-1, : E // groups * (groups - 1)] = -INF     # one group only
            check(x, top, scoring, b, renormalize=False, **kw)
            if b is not None:
                b[::3] = -INF
                check(x, top, scoring, b, scale=2.0, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("E,top", [(8, 3), (64, 8), (200, 8), (256, 20), (1024, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_scores_that_fp32_cannot_tell_apart(E, top, scoring):
    """The bias takes each score away but for its rounding: what is left is some
    2^-26 of it, and its order has to be that of 64 bits."""
    g = gen(E)
    x = torch.randn(1, E, device="cuda", generator=g).expand(50, E).contiguous()
    b = -scores64(x[:1], scoring)[0].float()
    left = (scores64(x[:1].cpu(), scoring)[0] + b.cpu().double()).sort().values
    # 64 bits tell apart what is chosen and the first that is not (the order of the
    # others, 1023 gaps at E = 1024, decides nothing): a score of at most 1 is within
    # (d + 48) 2^-53 of its value there, less than 1e-14 of it, and scores are below
    # 0.1 where a gap may be below 1e-14.
    assert (left[-top - 1:].diff() > 1e-14 * min(1.0, 10 * float(b.abs().max()))).all()
    check(x, top, scoring, b)
    check(x, top, scoring, b, renormalize=False)
    if E % 8 == 0:
        check(x, min(top, E // 8 * 3), scoring, b, groups=8, top_groups=3,
              group_best=min(2, E // 8))
    # some rows only, at every place in a wave
    x[::7] += 0.1 * torch.randn(x[::7].shape, device="cuda", generator=g)
    check(x, top, scoring, b)


def apart64(x, top, scoring, bias, groups, top_groups):
    """The tokens whose choice 64 bits tell apart for certain, with groups of two
    scores: the last group that stays and the first that does not, and each choice and
    the next one.  A score is within 2^-48 of its value there, and c and a total of two
    round by 2^-53 of the largest bias each: 8 such roundings lie below `least`."""
    x, b = x.cpu().double(), bias.cpu().double()
    T, E = x.shape
    least = 1e-13 + 8 * 2.0 ** -53 * b.abs().max()
    c = scores64(x, scoring) + b
    total = c.reshape(T, groups, -1).sort(dim=2, descending=True).values[:, :, :2].sum(2)
    total, order = total.sort(dim=1, descending=True, stable=True)
    good = total[:, top_groups - 1] - total[:, top_groups] > least
    stays = torch.zeros(T, groups, dtype=torch.bool)
    stays.scatter_(1, order[:, :top_groups], True)
    c[~stays.repeat_interleave(E // groups, 1)] = -INF
    c = c.sort(dim=1, descending=True).values[:, :top + 1]
    return (good & ((c[:, :-1] - c[:, 1:])[:, :top] > least).all(1)).nonzero().squeeze(1)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,top_groups,top", [(4, 2, 1, 2), (16, 8, 3, 4), (32, 4, 2, 8),
                                                     (96, 16, 5, 6), (256, 8, 4, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_two_scores_of_a_group_that_cancel(E, groups, top_groups, top, scoring):
    """A group's best two have large biases of opposite signs: each was rounded at its
    own size, and their sum, which decides, is far smaller.  Neighbouring groups have
    nearly the same scores, so that the roundings would decide in FP32."""
    g = gen(E + groups)
    T, size = 4000, E // groups
    kw = dict(groups=groups, top_groups=top_groups, group_best=2)
    for X in (64.0, 1000.0, 1e4):
        x = torch.randn(T, 1, size, device="cuda", generator=g).repeat(1, groups, 1)
        # of a last place of X, once the scores' slope (at most 1/4) has made it smaller
        near = X * 2.0 ** -22 * (1 if scoring == "sigmoid" else groups)
        x = (x + near * torch.randn(x.shape, device="cuda", generator=g)).reshape(T, E)
        b = torch.full((groups, size), -2 * X, device="cuda")
        b[:, 0], b[:, 1] = X, -X
        if X == 1e4:
            b[::3, :2] = 0.0        # groups of both kinds
        b = b.reshape(E)
        rows = apart64(x, top, scoring, b, groups, top_groups)
        assert rows.numel() >= T // 4
        check(x[rows.cuda()].contiguous(), top, scoring, b, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_totals_of_a_group_past_fp32(scoring):
    """The sums of two biases of some 3e38 are infinite in FP32, not in 64 bits; a
    group of scores that are infinite themselves is larger than those."""
    x = torch.randn(70, 12, device="cuda", generator=gen(3))
    for rows in ([[3e38, 2e38], [3e38, 2.5e38], [2e38, 2e38]],
                 [[-3e38, -3e38], [-3e38, -2e38], [-2e38, -3.3e38]],
                 [[3e38, 3e38], [INF, -3e38], [3e38, 3.2e38]],
                 [[-INF, -INF], [-3e38, -3e38], [-INF, -3.3e38]],
                 [[1e9, -1e9], [1.0, 1.0], [-1e9, -1e9]]):
        b = torch.full((3, 4), -3.4e38, device="cuda")
        b[:, 1:3] = torch.tensor(rows, device="cuda")
        for top_groups in (1, 2):
            # one choice a group: the scores beside 3e38 are nothing in 64 bits either
            ids, _ = sg.moe_route(x, top_groups, scoring, b.reshape(12), groups=3,
                                  top_groups=top_groups, group_best=2)
            assert torch.equal(ids.cpu(), choose64(x, top_groups, scoring, b.reshape(12), groups=3,
                                                   top_groups=top_groups, group_best=2))


@pytest.mark.gpu
@pytest.mark.parametrize("E,top", [(5, 2), (16, 4), (64, 8), (130, 31), (1024, 16)])
def test_ties_go_to_the_lowest(E, top):
    for value in (0.0, -0.0, 7.5, -3.4e38):
        x = torch.full((9, E), value, device="cuda")
        x[:, E // 2:] = abs(value) if value == 0 else value      # +0 and -0 are equal
        for scoring in ("softmax", "sigmoid"):
            for b in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.3, device="cuda")):
                ids, w = sg.moe_route(x, top, scoring, b)
                assert torch.equal(ids.cpu(), torch.arange(top, dtype=torch.int32).expand(9, top))
                # equal parts: top - 1 sums of them, and a quotient
                assert ((w - 1 / top).abs() <= (top + 4) * U / top).all()
                if E % 4 == 0:
                    ids, _ = sg.moe_route(x, min(top, E // 2), scoring, b, groups=4, top_groups=2,
                                          group_best=2 if E > 4 else 1)
                    assert (ids.cpu() == torch.arange(min(top, E // 2), dtype=torch.int32)).all()
    # pairs of equal scores in shuffled rows
    g = gen(E)
    x = torch.randint(0, 4, (200, E), device="cuda", generator=g).float()
    for scoring in ("softmax", "sigmoid"):
        check(x, top, scoring)
        check(x, top, scoring, 0.25 * torch.randint(0, 3, (E,), device="cuda",
                                                    generator=g).float())


@pytest.mark.gpu
def test_masked_experts_and_rows_without_any():
    g = gen(5)
    for E, top in ((8, 2), (40, 6), (256, 8), (600, 4)):
        x = torch.randn(64, E, device="cuda", generator=g)
        x[torch.rand(64, E, device="cuda", generator=g) < 0.6] = -INF
        x[3] = -INF
        x[5, 1:] = -INF
        x[6] = torch.finfo(torch.float32).min
        x[7, : E // 2] = torch.finfo(torch.float32).min
        b = 0.1 * torch.randn(E, device="cuda", generator=g)
        for scoring in ("softmax", "sigmoid"):
            for bias in (None, b):
                for renorm in (True, False):
                    ids, w = check(x, top, scoring, bias, renorm)
                    assert (ids[3] == -1).all() and (w[3] == 0).all()
                    dw = torch.randn(64, top, device="cuda", generator=g)
                    d = sg.moe_route_backward(dw, x, ids, w, scoring, renormalize=renorm)
                    assert torch.isfinite(d).all() and (d[3] == 0).all()
                    assert (d[x == -INF] == 0).all()


@pytest.mark.gpu
def test_far_logits_keep_their_weights():
    # scores that vanish in FP32, but not their parts of the chosen ones' sum
    x = torch.tensor([[-200.0, -201.0, -203.0, -300.0], [-1e4, -1e4 - 1, -2e4, -3e4],
                      [300.0, 299.0, -300.0, 0.0]], device="cuda")
    for scoring in ("softmax", "sigmoid"):
        check(x, 2, scoring)
        check(x, 3, scoring)


@pytest.mark.gpu
def test_nan_and_infinity_count_as_the_largest():
    nan = float("nan")
    x = torch.zeros(4, 20, device="cuda")
    x[0, 7], x[1, 5], x[2, [3, 9]], x[3, 11] = nan, INF, nan, nan
    x[3, 4] = -INF
    for scoring in ("softmax", "sigmoid"):
        ids, w = sg.moe_route(x, 3, scoring)
        assert ids[:, 0].tolist() == [7, 5, 3, 11] and ids[2, 1] == 9
        assert w[0].isnan().all() and w[2].isnan().all() and w[3].isnan().all()
        ids, w = sg.moe_route(x, 3, scoring, torch.zeros(20, device="cuda"))
        # a softmax with a NaN is NaN throughout, so equal; never the masked one
        first = [[7, 0, 1], [0, 1, 2], [3, 9, 0], [11, 0, 1]] if scoring == "sigmoid" else \
            [[0, 1, 2]] * 4
        if scoring == "sigmoid":
            first[1] = [5, 0, 1]
        assert ids.tolist() == first


def backward64(dw, x, ids, w, scoring, renorm, scale):
    """dlogits and its bound, term by term."""
    E = x.shape[1]
    kept = (ids >= 0) & (ids < E)
    at = torch.where(kept, ids, 0).long()
    dw = torch.where(kept, dw.double(), 0.0)
    l = x.double().gather(1, at)
    zero = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    if renorm:
        w = torch.where(kept, w.double(), 0.0)
        dot = (dw * w).sum(1, keepdim=True) / scale
        size = w.abs() * (dw.abs() + (dw * w).abs().sum(1, keepdim=True) / abs(scale))
        d, tol = w * (dw - dot), 64 * U * size
        if scoring == "sigmoid":
            d, tol = d * torch.sigmoid(-l), tol * torch.sigmoid(-l) + 16 * U * d.abs()
        d, tol = torch.where(kept, d, 0.0), torch.where(kept, tol, 0.0)
        return zero.scatter_add(1, at, d), zero.scatter_add(1, at, tol)
    p = scores64(x, scoring)
    p = torch.where(p.isnan(), 0.0, p)
    own = zero.scatter_add(1, at, scale * dw)
    size = zero.scatter_add(1, at, abs(scale) * dw.abs())
    if scoring == "sigmoid":
        s = p * torch.sigmoid(-x.double())
        return own * s, 64 * U * size * s
    far = torch.where(x == -INF, 0.0, x.double().amax(1, keepdim=True) - x.double())
    dot = (own * p).sum(1, keepdim=True)
    off = ((far + 96) * size * p).sum(1, keepdim=True)
    return (p * (own - dot),
            U * p * ((far + 96) * (size + (size * p).sum(1, keepdim=True)) + off))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,top", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(T, E, top, scoring, renorm):
    g = gen(T * 3 + E)
    for pad, off, scale in ((0, 0, 1.0), (3, 1, -2.5)):
        x = wide(T, E, pad, off, g, 1.5)
        ids, w = sg.moe_route(x, top, scoring, renormalize=renorm, scale=scale)
        dw = torch.randn(T, top, device="cuda", generator=g)
        out = wide(T, E, pad, off, g, fill=7.0)
        got = sg.moe_route_backward(dw, x, ids, w, scoring, renormalize=renorm, scale=scale,
                                    out=out)
        assert got is out
        want, tol = backward64(dw, x, ids, w, scoring, renorm, scale)
        err = (got.double() - want).abs()
        assert (err <= tol + 2.0 ** -126).all(), (err / tol).nan_to_num(0).max().item()
        if pad and T > 1:
            assert (out.as_strided((T - 1, pad), (out.stride(0), 1),
                                   out.storage_offset() + E) == 7.0).all()
        over = wide(T, E, pad, off, g)
        over.copy_(x)
        again = sg.moe_route_backward(dw, over, ids, w, scoring, renormalize=renorm, scale=scale,
                                      out=over)
        assert torch.equal(again, got)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_dropped_and_repeated_choices_have_their_gradients(scoring, renorm):
    g = gen(77)
    T, E, top = 60, 37, 7
    x = torch.randn(T, E, device="cuda", generator=g)
    ids = torch.randint(-2, E + 2, (T, top), device="cuda", generator=g, dtype=torch.int32)
    ids[0] = -1
    ids[1] = 5                                  # one expert, seven times
    ids[2, :4] = torch.tensor([3, 9, 3, 3], device="cuda", dtype=torch.int32)
    ids[3] = torch.iinfo(torch.int32).max
    ids[4] = torch.iinfo(torch.int32).min
    w = torch.rand(T, top, device="cuda", generator=g)
    dw = torch.randn(T, top, device="cuda", generator=g)
    dw[ids < 0] = float("nan")                  # never read into a result
    d = sg.moe_route_backward(dw, x, ids, w, scoring, renormalize=renorm, scale=1.5)
    want, tol = backward64(dw, x, ids, w, scoring, renorm, 1.5)
    assert ((d.double() - want).abs() <= 7 * tol).all()      # up to seven terms of an expert
    assert (d[[0, 3, 4]] == 0).all()
    for _ in range(3):
        assert torch.equal(sg.moe_route_backward(dw, x, ids, w, scoring, renormalize=renorm,
                                                 scale=1.5), d)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_against_differences(scoring, renorm):
    """sum(weights * C) for the experts that were chosen, moved along a direction."""
    g = gen(31)
    x = torch.randn(40, 48, device="cuda", generator=g)
    C = torch.randn(40, 6, device="cuda", generator=g)
    ids, w = sg.moe_route(x, 6, scoring, renormalize=renorm, scale=2.0)
    d = sg.moe_route_backward(C, x, ids, w, scoring, renormalize=renorm, scale=2.0)
    v = torch.randn(x.shape, device="cuda", generator=g).double()

    def loss(x):
        s = scores64(x, scoring).gather(1, ids.long())
        if renorm:
            s = s / s.sum(1, keepdim=True)
        return (2.0 * s * C.double()).sum()

    h = 1e-5
    num = ((loss(x.double() + h * v) - loss(x.double() - h * v)) / (2 * h)).item()
    terms = (d.double() * v).abs().sum().item()
    # some 150 half steps of each term, and the difference's own error
    assert abs((d.double() * v).sum().item() - num) <= (150 * U + 1e-6) * terms


@pytest.mark.gpu
def test_replays_from_a_graph_and_runs_on_a_stream():
    g = gen(9)
    x = torch.randn(500, 64, device="cuda", generator=g)
    b = 0.05 * torch.randn(64, device="cuda", generator=g)
    dw = torch.randn(500, 6, device="cuda", generator=g)

    def step(**kw):
        ids, w = sg.moe_route(x, 6, "sigmoid", b, groups=8, top_groups=3, group_best=2, **kw)
        d = sg.moe_route_backward(dw, x, ids, w, "sigmoid", **kw)
        return (ids, w, d, *sg.moe_sort(ids, 64, **kw))

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        x.normal_(generator=g)
        for o in out:
            o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for p, q in zip(got, step()):
            assert torch.equal(p, q), rep


@pytest.mark.gpu
def test_offsets_past_32_bits():
    T, E, ld = 3, 40, (1 << 31) - 4
    buf = torch.empty((T - 1) * ld + E, device="cuda")
    x = buf.as_strided((T, E), (ld, 1))
    rows = torch.randn(T, E, device="cuda", generator=gen(2))
    x.copy_(rows)
    for scoring, renorm in (("softmax", False), ("sigmoid", True)):
        want = sg.moe_route(rows, 4, scoring, renormalize=renorm)
        got = sg.moe_route(x, 4, scoring, renormalize=renorm)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        dw = torch.randn(T, 4, device="cuda", generator=gen(3))
        d = sg.moe_route_backward(dw, rows, *want, scoring, renormalize=renorm)
        assert torch.equal(sg.moe_route_backward(dw, x, *got, scoring, renormalize=renorm, out=x),
                           d)
        x.copy_(rows)


@pytest.mark.gpu
def test_no_tokens():
    x = torch.empty(0, 8, device="cuda")
    ids, w = sg.moe_route(x, 2)
    assert ids.shape == w.shape == (0, 2)
    assert sg.moe_route_backward(w, x, ids, w).shape == (0, 8)


# Refusals (CPU).

BIG = 1 << 33
FAR = BIG + (1 << 40)


@pytest.fixture(scope="module")
def lib():
    from tiled_fp32_gemm_amd import build
    build.ensure_built()
    return sg.load()


def router(scoring=0, renormalize=1, scale=1.0, bias=0, groups=1, top_groups=1, group_best=1):
    return sg.Router(scoring, renormalize, scale, bias, groups, top_groups, group_best)


def route(T=4, E=8, top=2, x=BIG, ld=8, ids=FAR, w=FAR * 2, **r):
    return sg.sgemm_moe_route(T, E, top, x, ld, router(**r), ids, w, 0)


@pytest.mark.parametrize("args", [
    dict(T=-1), dict(E=0), dict(E=-8), dict(top=0), dict(top=-1), dict(top=9), dict(ld=7),
    dict(scoring=2), dict(scoring=-1), dict(renormalize=2), dict(scale=0.0),
    dict(scale=INF), dict(scale=float("nan")), dict(groups=0), dict(groups=3), dict(groups=-1),
    dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(groups=4, group_best=0),
    dict(groups=4, group_best=3), dict(groups=8, group_best=2), dict(groups=4, top=3),
    dict(x=0), dict(ids=0), dict(w=0), dict(x=BIG + 2), dict(ids=FAR + 1), dict(w=FAR * 2 + 3),
    dict(bias=FAR * 3 + 2), dict(ids=BIG), dict(w=BIG + 64), dict(w=FAR), dict(bias=FAR),
    dict(bias=FAR * 2 + 16)])
def test_route_refuses(lib, args):
    assert route(**args) == sg.ERR_INVALID_ARG


def back(T=4, E=8, top=2, x=BIG, ld=8, ids=FAR, w=FAR * 2, dw=FAR * 3, d=FAR * 4, ldd=8, **r):
    return sg.sgemm_moe_route_backward(T, E, top, x, ld, router(**r), ids, w, dw, d, ldd, 0)


@pytest.mark.parametrize("args", [
    dict(T=-1), dict(E=0), dict(top=0), dict(top=9), dict(ldd=7), dict(scoring=2), dict(scale=0.0),
    dict(renormalize=-1), dict(ids=0), dict(w=0), dict(dw=0), dict(d=0), dict(d=FAR * 4 + 1),
    dict(dw=FAR * 3 + 2), dict(scoring=1, ld=7), dict(scoring=1, x=0),
    dict(scoring=1, x=BIG, d=BIG + 4), dict(scoring=1, x=BIG, d=BIG, ldd=9),
    dict(renormalize=0, x=0), dict(d=FAR), dict(d=FAR * 2), dict(d=FAR * 3 + 16)])
def test_route_backward_refuses(lib, args):
    assert back(**args) == sg.ERR_INVALID_ARG


def test_route_unsupported_and_nothing_to_do(lib):
    assert route(T=1 << 31) == sg.ERR_UNSUPPORTED
    assert route(E=1025, ld=1025) == sg.ERR_UNSUPPORTED
    assert route(E=64, ld=64, top=33) == sg.ERR_UNSUPPORTED
    assert route(E=64, ld=64, groups=64, top_groups=4) == sg.ERR_UNSUPPORTED
    assert route(T=1 << 30, ld=1 << 61) == sg.ERR_UNSUPPORTED
    assert back(E=1025, ldd=1025) == sg.ERR_UNSUPPORTED
    assert back(T=1 << 30, ldd=1 << 61) == sg.ERR_UNSUPPORTED
    assert route(T=0, x=0, ids=0, w=0) == sg.OK
    assert back(T=0, x=0, ids=0, w=0, dw=0, d=0) == sg.OK
    for fn in (sg.sgemm_moe_route(4, 8, 2, BIG, 8, None, FAR, FAR * 2, 0),
               sg.sgemm_moe_route_backward(4, 8, 2, BIG, 8, None, FAR, FAR * 2, FAR * 3, FAR * 4,
                                           8, 0)):
        assert fn == sg.ERR_INVALID_ARG


@pytest.mark.gpu
def test_the_binding_refuses_bad_tensors():
    x, b = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    for kw in (dict(scoring="tanh"), dict(scoring=None), dict(bias=b[:4]), dict(bias=b.double()),
               dict(groups=0), dict(groups=1 << 32), dict(top_groups=-1), dict(group_best=0)):
        with pytest.raises(ValueError):
            sg.moe_route(x, 2, **kw)
    for bad in (x.half(), x.cpu(), x.t(), b):
        with pytest.raises(ValueError):
            sg.moe_route(bad, 2)
    for kw in (dict(top=0), dict(top=9), dict(top=33), dict(scale=0.0), dict(scale=1e300),
               dict(scale=float("nan")), dict(groups=3), dict(top=3, groups=4)):
        with pytest.raises(sg.SgemmError):
            sg.moe_route(x, **(dict(top=2) | kw))
    ids, w = sg.moe_route(x, 2)
    for args in ((w[:3], x, ids, w), (w, x, ids.long(), w), (w, x, ids, w[:, :1]),
                 (w, x, ids[:, :1], w), (w.half(), x, ids, w), (w[0], x, ids, w),
                 (w, x.half(), ids, w), (w, x, ids, w.double())):
        with pytest.raises(ValueError):
            sg.moe_route_backward(*args)
    with pytest.raises(ValueError):
        sg.moe_route_backward(w, x, ids, w, out=x[:, :4])
