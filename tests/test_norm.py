"""Layer norm and its gradients, against the definition in 64 bits.

Tolerances, from FP32 arithmetic (u = 2^-24, half a step; S(n) = min(1e-5, (n + 3) u)
bounds the relative error of a sum of n terms in any order, over their sizes):
  mean  S(N) mean|x|
  rstd  the mean's error e shifts every deviation: the mean square moves by at most
        e^2 + 2 u e sd and, rounded, by (S(N) + 6 u) (var + e^2); the root halves
        its relative error and adds four roundings
  y     |w| rstd (e + |d| (that + 4 u)) and a rounding of y and of bias
  dx    from the statistics as given: xh is two roundings, g one more, the means of
        g and g xh are sums of N, and what is left fewer than eight roundings
  dw    S(M) and four roundings a term over |dy xh|;  db  S(M) over |dy|
"""
from __future__ import annotations

import pytest

import tiled_fp32_gemm_amd as sg
from test_linear import U, gen, sum_tol, wide

torch = pytest.importorskip("torch")


def stats64(x, eps):
    x = x.double()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    return mean, d, 1 / torch.sqrt((d * d).sum(1) / x.shape[1] + eps)


def forward64(x, w, b, eps):
    """y, mean, rstd and their bounds."""
    N = x.shape[1]
    mean, d, rstd = stats64(x, eps)
    var = (d * d).sum(1) / N
    e = sum_tol(N) * x.double().abs().sum(1) / N + U * mean.abs()
    off = e * e + 2 * U * e * var.sqrt() + (sum_tol(N) + 6 * U) * (var + e * e)
    rel = 0.5 * off / (var + eps) + 4 * U
    w = torch.ones(N, device="cuda").double() if w is None else w.double()
    b = torch.zeros(N, device="cuda").double() if b is None else b.double()
    y = d * rstd[:, None] * w + b
    ytol = w.abs() * rstd[:, None] * (e[:, None] + d.abs() * (rel + 4 * U)[:, None])
    # second order: the products of the bounds
    ytol = ytol * (1 + rel[:, None]) + 2 * U * (y.abs() + b.abs())
    return y, mean, rstd, ytol, e, rel * rstd * (1 + rel)


def backward64(dy, x, mean, rstd, w, res):
    """dx, dw, db and their bounds."""
    M, N = x.shape
    dy, rstd = dy.double(), rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * rstd
    g = dy if w is None else dy * w.double()
    s1, s2 = g.sum(1, keepdim=True) / N, (g * xh).sum(1, keepdim=True) / N
    e1 = (sum_tol(N) + 3 * U) * g.abs().sum(1, keepdim=True) / N
    e2 = (sum_tol(N) + 6 * U) * (g * xh).abs().sum(1, keepdim=True) / N
    dx = rstd * (g - s1 - xh * s2)
    tol = rstd * (e1 + xh.abs() * e2 + 8 * U * (g.abs() + s1.abs() + (xh * s2).abs()))
    if res is not None:
        dx = dx + res.double()
    tol = tol + 2 * U * dx.abs()
    terms = dy * xh
    return (dx, terms.sum(0), dy.sum(0), tol, (sum_tol(M) + 4 * U) * terms.abs().sum(0),
            sum_tol(M) * dy.abs().sum(0))


def near(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, {(err / tol)[bad].max().item()} bounds"


def untouched(view, fill):
    """The columns beside a padded matrix still hold `fill`."""
    M, N = view.shape
    pad = view.stride(0) - N
    if pad and M > 1:
        assert (view.as_strided((M - 1, pad), (view.stride(0), 1),
                                view.storage_offset() + N) == fill).all()


SHAPES = [(1, 1), (1, 5), (3, 16), (7, 63), (64, 64), (5, 65), (100, 128), (33, 129), (10, 256),
          (17, 257), (9, 512), (12, 515), (1000, 777), (50, 1024), (21, 1025), (8, 2048),
          (7, 2049), (6, 4096), (5, 4099), (4, 8192), (3, 8193), (2, 16384), (2, 16387),
          (3, 40001), (70000, 20), (9000, 256), (5000, 1500), (4100, 2050), (9001, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", SHAPES)
def test_norm_and_its_gradients(M, N):
    g = gen(M * 7 + N)
    for pad, off, affine in ((0, 0, "wb"), (3, 1, ""), (4, 0, "w"), (1, 3, "b")):
        x = wide(M, N, pad, off, g, 1.7)
        x += 3 * torch.randn(M, 1, device="cuda", generator=g)
        w = 1 + 0.3 * torch.randn(N, device="cuda", generator=g) if "w" in affine else None
        b = torch.randn(N, device="cuda", generator=g) if "b" in affine else None
        out = wide(M, N, pad, off, g, fill=7.0)
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        assert sg.layer_norm(x, w, b, 1e-5, out=out, mean=mean, rstd=rstd) is out
        y, m64, r64, ytol, mtol, rtol = forward64(x, w, b, 1e-5)
        near(out, y, ytol, "y")
        near(mean, m64, mtol, "mean")
        near(rstd, r64, rtol, "rstd")
        untouched(out, 7.0)
        assert torch.equal(sg.layer_norm(x, w, b, 1e-5), out)       # without statistics
        over = wide(M, N, pad, off, g)
        over.copy_(x)
        assert torch.equal(sg.layer_norm(over, w, b, out=over), out)  # in place
        # gradients, from statistics as given
        dy, res = wide(M, N, pad, off, g), wide(M, N, pad, off, g)
        for r in (None, res):
            dout = wide(M, N, pad, off, g, fill=7.0)
            dx, dw, db = sg.layer_norm_backward(dy, x, mean, rstd, w, r, out=dout)
            assert dx is dout
            want = backward64(dy, x, mean, rstd, w, r)
            near(dx, want[0], want[3], "dx")
            near(dw, want[1], want[4], "dw")
            near(db, want[2], want[5], "db")
            untouched(dout, 7.0)
            alone, none, nil = sg.layer_norm_backward(dy, x, mean, rstd, w, r, weight_grad=False)
            assert none is None and nil is None and torch.equal(alone, dx)
            for over in (dy, x) + (() if r is None else (r,)):
                kept = over.clone()
                again = sg.layer_norm_backward(dy, x, mean, rstd, w, r, out=over)
                assert again[0] is over
                for p, q in zip(again, (dx, dw, db)):
                    assert torch.equal(p, q)
                over.copy_(kept)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [48, 256, 2000, 20000])
def test_sums_alone_through_the_library(N):
    """dX is NULL; dweight or dbias is."""
    g = gen(N)
    M = 300
    x, dy = (torch.randn(M, N, device="cuda", generator=g) for _ in range(2))
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    sg.layer_norm(x, mean=mean, rstd=rstd)
    dx, dw, db = sg.layer_norm_backward(dy, x, mean, rstd)
    ws = torch.empty(sg.sgemm_layer_norm_backward_workspace_bytes(M, N) // 4, device="cuda")
    for a, b in ((1, 1), (1, 0), (0, 1)):
        got = torch.full((2, N), 7.0, device="cuda")
        st = sg.sgemm_layer_norm_backward(
            M, N, dy.data_ptr(), N, x.data_ptr(), N, mean.data_ptr(), rstd.data_ptr(), 0, 0, 1, 0,
            1, got[0].data_ptr() if a else 0, got[1].data_ptr() if b else 0,
            torch.cuda.current_stream().cuda_stream, ws.data_ptr(), 4 * ws.numel())
        assert st == sg.OK
        assert torch.equal(got[0], dw if a else torch.full_like(dw, 7.0))
        assert torch.equal(got[1], db if b else torch.full_like(db, 7.0))


@pytest.mark.gpu
def test_no_rows_and_no_columns():
    empty = torch.empty(0, 40, device="cuda")
    none = torch.empty(0, device="cuda")
    assert sg.layer_norm(empty, mean=none, rstd=none).shape == (0, 40)
    dx, dw, db = sg.layer_norm_backward(empty, empty, none, none)
    assert dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()
    flat = torch.empty(5, 0, device="cuda")
    assert sg.layer_norm(flat).shape == (5, 0)
    rows = torch.ones(5, device="cuda")
    dx, dw, db = sg.layer_norm_backward(flat, flat, rows, rows)
    assert dx.shape == (5, 0) and dw.numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [64, 1000, 4096, 16500])
def test_rows_of_one_value_and_a_large_mean(N):
    # sums of a small whole number are exact, so is their mean: nothing is left of it
    x = torch.full((4, N), 3.0, device="cuda")
    mean, rstd = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    y = sg.layer_norm(x, eps=1e-6, mean=mean, rstd=rstd)
    assert (y == 0).all() and (mean == 3).all()
    near(rstd, torch.full((4,), 1e3, device="cuda").double(), 4 * U * 1e3 + 1e3 * U, "rstd")
    g = gen(N)
    x = 100 + torch.randn(50, N, device="cuda", generator=g)
    y, _, _, tol, _, _ = forward64(x, None, None, 1e-5)
    near(sg.layer_norm(x), y, tol, "y")
    # eps = 0 and no variance: 0 / 0 in that row only
    x[7] = 3.0
    y = sg.layer_norm(x, eps=0.0)
    assert y[7].isnan().all() and torch.isfinite(y[:7]).all() and torch.isfinite(y[8:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [30, 512, 3000, 9000, 17000])
def test_non_finite_values_stay_in_their_rows(N):
    g = gen(N + 1)
    M = 9
    x, dy = (torch.randn(M, N, device="cuda", generator=g) for _ in range(2))
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    want = sg.layer_norm(x, mean=mean, rstd=rstd).clone()
    dwant = sg.layer_norm_backward(dy, x, mean, rstd)[0]
    for bad in (float("nan"), float("inf"), -float("inf")):
        x2, dy2 = x.clone(), dy.clone()
        x2[4, N // 2] = bad
        y = sg.layer_norm(x2)
        rows = torch.arange(M, device="cuda") != 4
        assert torch.equal(y[rows], want[rows]) and y[4].isnan().all()
        dy2[4, N // 2] = bad
        dx, dw, db = sg.layer_norm_backward(dy2, x, mean, rstd)
        assert torch.equal(dx[rows], dwant[rows]) and not torch.isfinite(dx[4]).any()
        cols = torch.arange(N, device="cuda") != N // 2
        assert torch.isfinite(dw[cols]).all() and torch.isfinite(db[cols]).all()
        assert not torch.isfinite(dw[~cols]).any() and not torch.isfinite(db[~cols]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [70, 1500, 9000])
def test_gradients_against_differences(N):
    """The loss sum(y * C) moved along a direction: the 64-bit forward's central
    difference against the gradients from FP32 statistics."""
    g = gen(N)
    M = 23
    x, C = (torch.randn(M, N, device="cuda", generator=g) for _ in range(2))
    w, b = (torch.randn(N, device="cuda", generator=g) for _ in range(2))
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    sg.layer_norm(x, w, b, mean=mean, rstd=rstd)
    grads = sg.layer_norm_backward(C, x, mean, rstd, w)

    def loss(x, w, b):
        _, d, r = stats64(x, 1e-5)
        return ((d * r[:, None] * w + b) * C.double()).sum()

    base = [x.double(), w.double(), b.double()]
    for i, d in enumerate(grads):
        v = torch.randn(d.shape, device="cuda", generator=g).double()
        h, up, dn = 1e-5, list(base), list(base)
        up[i], dn[i] = base[i] + h * v, base[i] - h * v
        num = ((loss(*up) - loss(*dn)) / (2 * h)).item()
        terms = (d.double() * v).abs().sum().item()
        # sums of N and M terms, and the difference's own error
        assert abs((d.double() * v).sum().item() - num) <= (1e-5 + 1e-6) * terms


@pytest.mark.gpu
def test_sums_of_many_rows_keep_their_accuracy():
    M, N = 1 << 21, 40
    x = torch.rand(M, N, device="cuda", generator=gen(3))
    dy = torch.rand(M, N, device="cuda", generator=gen(4))
    mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    _, dw, db = sg.layer_norm_backward(dy, x, mean, rstd)
    terms = dy.double() * x.double()
    # 256 terms, then at most as many spans a part, then 64 parts and 16 rows by halves
    near(dw, terms.sum(0), (256 + 256 + 32) * U * terms.sum(0), "dw")
    near(db, dy.double().sum(0), (256 + 256 + 32) * U * dy.double().sum(0), "db")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 64), (300, 1024), (40, 5000), (6, 20000)])
def test_replays_from_a_graph_and_runs_on_a_stream(M, N):
    g = gen(M + N)
    x, dy = (torch.randn(M, N, device="cuda", generator=g) for _ in range(2))
    w, b = (torch.randn(N, device="cuda", generator=g) for _ in range(2))
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    ws = torch.empty(sg.sgemm_layer_norm_backward_workspace_bytes(M, N) // 4, device="cuda")

    def step(**kw):
        y = sg.layer_norm(x, w, b, mean=mean, rstd=rstd, **kw)
        return (y, *sg.layer_norm_backward(dy, x, mean, rstd, w, y, workspace=ws, **kw))

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
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for p, q in zip(got, step()):
            assert torch.equal(p, q), rep


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows 2^31 floats apart, checked from both ends."""
    M, N, ld = 3, 300, (1 << 31) - 4
    buf = torch.empty((M - 1) * ld + N, device="cuda")
    x = buf.as_strided((M, N), (ld, 1))
    g = gen(8)
    rows = torch.randn(M, N, device="cuda", generator=g)
    x.copy_(rows)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    want = sg.layer_norm(rows, mean=mean, rstd=rstd)
    grads = sg.layer_norm_backward(rows, rows, mean, rstd, None, rows)
    got = sg.layer_norm_backward(x, x, mean, rstd, None, x, out=x)
    for p, q in zip(got, grads):
        assert torch.equal(p, q)
    x.copy_(rows)
    assert torch.equal(sg.layer_norm(x, out=x), want)


# Refusals (CPU).

BIG = 1 << 33
FAR = BIG + (1 << 40)


@pytest.fixture(scope="module")
def lib():
    from tiled_fp32_gemm_amd import build
    build.ensure_built()
    return sg.load()


def forward(M=4, N=8, X=BIG, ldx=8, w=0, b=0, eps=1e-5, Y=FAR, ldy=8, mean=0, rstd=0):
    return sg.sgemm_layer_norm(M, N, X, ldx, w, b, eps, Y, ldy, mean, rstd, 0)


@pytest.mark.parametrize("args", [
    dict(M=-1), dict(N=-1), dict(ldx=7), dict(ldy=7), dict(eps=-1e-9), dict(eps=float("nan")),
    dict(X=0), dict(Y=0), dict(X=BIG + 2), dict(Y=FAR + 1), dict(w=BIG + (1 << 34) + 2),
    dict(b=BIG + (1 << 34) + 1), dict(mean=BIG + (1 << 34) + 3),
    dict(Y=BIG, ldy=9), dict(Y=BIG + 4), dict(w=FAR), dict(b=FAR + 64), dict(mean=BIG),
    dict(rstd=FAR), dict(mean=FAR * 2, rstd=FAR * 2 + 12), dict(w=FAR * 2, mean=FAR * 2)])
def test_norm_refuses(lib, args):
    assert forward(**args) == sg.ERR_INVALID_ARG


def backward(M=4, N=8, dY=BIG, lddy=8, X=BIG + (1 << 34), ldx=8, mean=BIG + (1 << 35),
             rstd=BIG + (1 << 36), w=0, res=0, ldr=8, dX=FAR, lddx=8, dw=FAR * 2, db=FAR * 3, ws=FAR * 4,
             ws_bytes=1 << 20):
    return sg.sgemm_layer_norm_backward(M, N, dY, lddy, X, ldx, mean, rstd, w, res, ldr, dX, lddx,
                                        dw, db, 0, ws, ws_bytes)


@pytest.mark.parametrize("args", [
    dict(M=-1), dict(N=-1), dict(lddy=7), dict(ldx=7), dict(lddx=7), dict(res=FAR * 5, ldr=7),
    dict(dY=0), dict(X=0), dict(mean=0), dict(rstd=0), dict(dY=BIG + 2), dict(dX=FAR + 2),
    dict(mean=BIG + (1 << 35) + 1), dict(dw=FAR * 2 + 2), dict(ws=0), dict(ws=FAR * 4 + 1),
    dict(ws_bytes=-4), dict(ws_bytes=8), dict(ws_bytes=0), dict(dX=BIG, lddx=9), dict(dX=BIG + 16),
    dict(dX=BIG + (1 << 35)), dict(dw=FAR), dict(db=FAR * 2 + 16), dict(dw=BIG), dict(ws=BIG),
    dict(ws=FAR), dict(ws=FAR * 2), dict(w=FAR), dict(w=FAR * 3), dict(res=FAR * 4)])
def test_norm_backward_refuses(lib, args):
    assert backward(**args) == sg.ERR_INVALID_ARG


def test_norm_unsupported_and_nothing_to_do(lib):
    assert forward(M=1 << 31) == sg.ERR_UNSUPPORTED
    assert forward(N=1 << 31, ldx=1 << 31, ldy=1 << 31) == sg.ERR_UNSUPPORTED
    assert forward(M=1 << 30, ldx=1 << 60, ldy=1 << 60) == sg.ERR_UNSUPPORTED
    assert forward(M=1 << 23, N=20000, ldx=20000, ldy=20000, Y=1 << 52) == sg.ERR_UNSUPPORTED
    assert backward(M=1 << 31, dw=0, db=0) == sg.ERR_UNSUPPORTED
    assert forward(M=0, X=0, Y=0) == sg.OK and forward(N=0, X=0, Y=0) == sg.OK
    assert backward(N=0, dY=0, X=0) == sg.OK
    assert backward(dX=0, dw=0, db=0) == sg.OK
    assert backward(M=0, dw=0, db=0, dY=0) == sg.OK
    for sizes in ((0, 8), (8, 0), (-1, 8), (8, -1), (1 << 31, 8)):
        assert sg.sgemm_layer_norm_backward_workspace_bytes(*sizes) == 0
    assert sg.sgemm_layer_norm_backward_workspace_bytes(1, 1) == 8


def test_the_header_declares_the_binding_names(lib):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "sgemm_norm.h")).read(),
                  flags=re.S)
    found = re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, re.M)
    assert sorted(found) == sorted(sg.NORM_SYMBOLS)
    for n in found:
        assert hasattr(lib, n) and hasattr(sg, n)


def test_the_binding_refuses_what_is_no_gpu_tensor():
    x = torch.randn(4, 8)
    with pytest.raises(ValueError, match="on a GPU"):
        sg.layer_norm(x)
    with pytest.raises(ValueError, match="on a GPU"):
        sg.layer_norm_backward(x, x, x[:, 0], x[:, 0])


@pytest.mark.gpu
def test_the_binding_refuses_bad_tensors():
    x, v, r = (torch.zeros(s, device="cuda") for s in ((4, 8), 8, 4))
    bad = [dict(weight=r), dict(bias=r), dict(weight=v.half()), dict(bias=v.cpu()),
           dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(mean=v),
           dict(rstd=r.double()), dict(out=torch.zeros(8, 4, device="cuda")),
           dict(out=x.t().contiguous().t()), dict(weight=torch.zeros(16, device="cuda")[::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            sg.layer_norm(x, **kw)
    with pytest.raises(ValueError):
        sg.layer_norm(x.half())
    with pytest.raises(ValueError):
        sg.layer_norm(v)
    for args in ((x, x[:3], r, r), (x, x, v, r), (x, x, r, v), (x, x, r, r, r),
                 (x, x, r, r, v, x[:, :4]), (x, x.half(), r, r)):
        with pytest.raises(ValueError):
            sg.layer_norm_backward(*args)
    with pytest.raises(ValueError, match="workspace"):
        sg.layer_norm_backward(x, x, r, r, workspace=torch.zeros(4))
    with pytest.raises(sg.SgemmError):      # too little room
        sg.layer_norm_backward(x, x, r, r, workspace=torch.zeros(4, device="cuda"))
    with pytest.raises(sg.SgemmError):      # overlapping, not the same
        base = torch.zeros(5, 8, device="cuda")
        sg.layer_norm(base[:4], out=base[1:])
    with pytest.raises(sg.SgemmError):      # rows on top of each other
        sg.layer_norm(torch.zeros(1, 8, device="cuda").expand(4, 8))
