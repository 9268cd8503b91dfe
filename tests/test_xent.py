"""Cross entropy of a product's rows and its gradients, against the definition in
64 bits.

Tolerances, from FP32 arithmetic (u = 2^-24; S(n) = min(1e-5, (n + 3) u)):
  z     S(H) (|A|·|B|), called e
  lse   moves by no more than the largest e of its row; an exponential is within 2 u
        and 1.22 u times its distance from its reference, twice (in its strip, and its
        strip's among the others), whose means under the softmax are at most ln V (the
        entropy) in sum; the sum of V of them goes by 4 columns, 4 steps over lanes,
        strips of 32 or 64 columns in 64 parts sixteen at a time, and 6 halves: with
        that (40 + V / 2048 + 8 + ln V) u, as 1.22 ln V <= ln V + 4 below 2^20; m and
        log s are rounded once each and added
  loss  the same, and e at the target
  dz    relative to |dloss| p, e at its place, and an exponential by a power of two:
        its argument (z - lse) log2 e is rounded twice, u |z - lse| each, log2 e is off
        by 0.22 u of it, the power by 2 u; 2 u of p and of the target's 1
  dA, dB   dz's error carried over, S of the products' lengths over |dz|·|B| and
        |A|·|dz|; a vocabulary in n pieces adds n roundings of dA's partial sums
FP32 has no normal number below 2^-126 (probabilities of 1e-305 that FP64 has are 0
there): an exponential, a dz and each term and sum of a product may be off by that.
"""
from __future__ import annotations

import math

import pytest

import tiled_fp32_gemm_amd as sg
from test_linear import U, gen, sum_tol, wide

torch = pytest.importorskip("torch")


def near(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, {(err / tol)[bad].max().item()} bounds"


def logits64(A, B, tb):
    a, b = A.double(), (B.t() if tb else B).double()
    return a @ b, sum_tol(A.shape[1]) * (a.abs() @ b.abs())


def check_loss(loss, lse, A, B, targets, tb):
    T, V = A.shape[0], B.shape[0 if tb else 1]
    kept = (targets >= 0) & (targets < V)
    assert (loss[~kept] == 0).all()
    assert lse is None or (lse[~kept] == 0).all()
    rows = kept.nonzero().squeeze(1)
    z, e = logits64(A[rows], B, tb)
    want = torch.logsumexp(z, 1)
    size = z.abs().amax(1) if rows.numel() else want
    tol = e.amax(1) if rows.numel() else want
    tol = tol + (40 + V / 2048 + 8 + math.log(V)) * U + 3 * U * (size + want.abs())
    if lse is not None:
        near(lse[rows], want, tol, "lse")
    at = targets[rows].long()[:, None]
    hit = z.gather(1, at).squeeze(1)
    near(loss[rows], want - hit, tol + e.gather(1, at).squeeze(1) + 2 * U * (want - hit), "loss")


def grads64(dloss, A, B, targets, lse, tb, pieces=64):
    """dA, dB and their bounds, from lse and dloss as given."""
    T, V = A.shape[0], B.shape[0 if tb else 1]
    kept = (targets >= 0) & (targets < V)
    a = torch.where(kept[:, None], A, 0.0)      # what it holds does not matter
    g = torch.where(kept, dloss, 0.0).double()[:, None]
    l = torch.where(kept, lse, 0.0).double()[:, None]
    z, e = logits64(a, B, tb)
    p = torch.where(kept[:, None], torch.exp(z - l), 0.0)
    hit = torch.zeros_like(p)
    hit[kept, targets[kept].long()] = 1.0
    dz = (p - hit) * g
    rel = e + 2.3 * U * (z - l).abs() + 10 * U
    tiny = 2.0 ** -126
    dtol = g.abs() * (p * (rel + rel * rel) + 2 * U * (p + hit) + tiny) + tiny
    a, b = a.double(), (B.t() if tb else B).double()
    dA, dB = dz @ b.t(), a.t() @ dz
    tA = dtol @ b.abs().t() + (sum_tol(V) + pieces * U) * (dz.abs() @ b.abs().t())
    tB = a.abs().t() @ dtol + sum_tol(T) * (a.abs().t() @ dz.abs())
    tA, tB = tA + 2 * V * tiny, tB + 2 * T * tiny
    return dA, dB.t() if tb else dB, tA, tB.t() if tb else tB


def make(T, H, V, tb, g, pad=0, off=0, ignored=0.0, dtype=torch.int64, scale=2.0):
    A = wide(T, H, pad, off, g)
    B = wide(*((V, H) if tb else (H, V)), pad, off, g, scale * max(H, 1) ** -0.5)
    targets = torch.randint(0, max(V, 1), (T,), device="cuda", generator=g).to(dtype)
    skip = torch.rand(T, device="cuda", generator=g) < ignored
    targets[skip] = -100
    return A, B, targets, skip


def run(T, H, V, tb=True, pad=0, off=0, ignored=0.0, dtype=torch.int64, seed=1, ws=None, scale=2.0):
    g = gen(seed)
    A, B, targets, skip = make(T, H, V, tb, g, pad, off, ignored, dtype, scale)
    lse, out = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    assert sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse, out=out) is out
    check_loss(out, lse, A, B, targets, tb)
    dloss = torch.randn(T, device="cuda", generator=g)
    room = None
    if ws is not None:
        room = torch.full((ws // 4,), float("nan"), device="cuda")
    dA, dB = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb,
                                              workspace=room)
    wA, wB, tA, tB = grads64(dloss, A, B, targets, lse, tb, max(64, V // 256 + 1))
    near(dA, wA, tA, "dA")
    near(dB, wB, tB, "dB")
    assert (dA[skip] == 0).all()
    return dA, dB


SHAPES = [(1, 1, 1), (1, 64, 100), (3, 5, 7), (2, 3, 1), (16, 256, 1000), (8, 1024, 4100),
          (33, 65, 130), (100, 128, 257), (7, 777, 5003), (130, 96, 3000), (64, 64, 64),
          (1000, 100, 500), (257, 512, 2050), (300, 33, 20000), (4000, 40, 1500), (31, 2000, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", SHAPES)
@pytest.mark.parametrize("tb", [False, True])
def test_loss_and_its_gradients(T, H, V, tb):
    run(T, H, V, tb)
    run(T, H, V, tb, pad=3, off=1, ignored=0.4, dtype=torch.int32, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(2048, 1024, 8200), (9000, 256, 7000), (1025, 2050, 9001)])
@pytest.mark.parametrize("tb", [False, True])
def test_many_rows_of_which_some_count(T, H, V, tb):
    """Large enough for the rows with a target to be gathered first."""
    for ignored in (0.0, 0.6):
        run(T, H, V, tb, ignored=ignored, seed=T)
    run(T, H, V, tb, pad=1, off=2, ignored=0.999, seed=T + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(1024, 512, 30000), (1000, 1030, 15001), (700, 1500, 15000)])
@pytest.mark.parametrize("tb", [False, True])
def test_up_to_1024_rows_gathered_for_the_loss(T, H, V, tb):
    """One launch numbers and copies the rows, here for a product of over 200 us."""
    assert 2 * T * H * V > 200e-6 * 150e12
    run(T, H, V, tb, ignored=0.4, seed=T)
    run(T, H, V, tb, pad=3, off=1, ignored=0.0, dtype=torch.int32, seed=V)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(19, 2894, 3306), (3, 2647, 111), (300, 4096, 500),
                                   (1, 1024, 32768), (8, 1030, 20001), (4, 1305, 142),
                                   (14, 1330, 2235), (1000, 4096, 300), (2, 5000, 3)])
@pytest.mark.parametrize("tb", [False, True])
def test_few_tiles_over_a_long_k_and_few_rows(T, H, V, tb):
    """The product is left in planes."""
    run(T, H, V, tb, seed=T + V)
    run(T, H, V, tb, pad=3, off=1, ignored=0.4, dtype=torch.int32, seed=T + V + 1)
    # in pieces, where a smaller one may have no planes
    least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
    run(T, H, V, tb, ignored=0.3, ws=least)
    run(T, H, V, tb, ignored=0.3, ws=least + 4 * T * 700)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(5, 30, 3000), (300, 64, 5000), (1500, 512, 2600)])
@pytest.mark.parametrize("tb", [False, True])
def test_a_vocabulary_in_pieces(T, H, V, tb):
    least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
    most = sg.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H)
    assert least < most
    run(T, H, V, tb, ignored=0.3, ws=least)
    run(T, H, V, tb, ignored=0.3, ws=least + 4 * T * 300)
    want = run(T, H, V, tb, ignored=0.3, ws=most)
    for x, y in zip(run(T, H, V, tb, ignored=0.3, ws=most + 12345 * 4), want):
        assert torch.equal(x, y)
    for x, y in zip(run(T, H, V, tb, ignored=0.3), want):     # a workspace of its own
        assert torch.equal(x, y)


FEW = [(1, 255, 1000), (2, 256, 4099), (3, 257, 513), (5, 1025, 2047), (6, 130, 1024),
       (8, 512, 1025), (8, 2049, 129), (7, 1, 3000), (4, 3000, 1), (8, 4, 70000), (1, 1030, 33000),
       (3, 5000, 700), (9, 300, 900), (16, 333, 2049), (13, 1024, 511), (16, 2, 5),
       (17, 90, 1030), (15, 4000, 600), (16, 60, 20000), (11, 129, 641)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", FEW)
@pytest.mark.parametrize("tb", [False, True])
def test_a_few_rows(T, H, V, tb):
    """Both gradients from one reading of B, and in pieces where there is no room for
    that; either alone; rows without a target in every place, whatever they hold."""
    run(T, H, V, tb, seed=H)
    run(T, H, V, tb, pad=5, off=3, ignored=0.5, dtype=torch.int32, seed=V)
    least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
    most = sg.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H)
    assert least <= most
    run(T, H, V, tb, ignored=0.3, ws=least, seed=T)
    g = gen(T * V)
    A, B, targets, _ = make(T, H, V, tb, g, pad=1, off=1)
    dloss, lse = torch.randn(T, device="cuda", generator=g), torch.empty(T, device="cuda")
    ws = torch.empty(most // 4, device="cuda")
    sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse)
    for none in [()] + [(t,) for t in range(T)] + [tuple(range(T))]:
        t2, A2, d2, l2 = targets.clone(), A.clone(), dloss.clone(), lse.clone()
        for t in none:
            t2[t], A2[t], d2[t], l2[t] = V + t, float("nan"), float("inf"), float("nan")
        ws.fill_(float("nan"))
        dA, dB = sg.linear_cross_entropy_backward(d2, A2, B, t2, l2, transpose_b=tb, workspace=ws)
        wA, wB, tA, tB = grads64(d2, A2, B, t2, l2, tb, max(64, V // 256 + 1))
        near(dA, wA, tA, "dA")
        near(dB, wB, tB, "dB")
        for a, b in ((True, False), (False, True)):
            got = sg.linear_cross_entropy_backward(d2, A2, B, t2, l2, transpose_b=tb, a_grad=a,
                                                   b_grad=b, workspace=ws)
            assert torch.equal(got[1 - a], (dA, dB)[1 - a]) and got[a] is None


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8])
def test_a_few_rows_over_a_large_weight(T):
    """B past the caches whose rows begin at any 4 bytes."""
    run(T, 1100, 70001, False, seed=T)
    run(T, 1100, 70001, False, pad=2, off=1, ignored=0.4, seed=T + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(5, 70, 900), (8, 300, 2000), (100, 70, 900)])
@pytest.mark.parametrize("tb", [False, True])
def test_gradients_into_wider_rows(T, H, V, tb):
    """Leading dimensions of the outputs: what lies between and behind their rows stays."""
    g = gen(H)
    A, B, targets, _ = make(T, H, V, tb, g, pad=2, ignored=0.3)
    dloss, lse = torch.randn(T, device="cuda", generator=g), torch.empty(T, device="cuda")
    sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse)
    want = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb)
    outs = [torch.full((w.shape[0] + 1, w.shape[1] + 3), 7.0, device="cuda") for w in want]
    ws = torch.empty(sg.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H), device="cuda",
                     dtype=torch.uint8)
    st = sg.sgemm_linear_xent_backward(
        tb, T, V, H, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0), targets.data_ptr(), 8,
        lse.data_ptr(), dloss.data_ptr(), outs[0].data_ptr(), H + 3, outs[1].data_ptr(),
        outs[1].shape[1], torch.cuda.current_stream().cuda_stream, ws.data_ptr(), ws.numel())
    assert st == sg.OK
    for o, w in zip(outs, want):
        assert torch.equal(o[:-1, :-3], w) and (o[:, -3:] == 7).all() and (o[-1] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 40, 2048])
def test_rows_without_a_target_reach_nothing(T):
    """Whatever they hold; and targets of every kind that is none."""
    H, V = {2048: 1024, 40: 50, 20: 3000}[T], 8200 if T > 20 else 300
    g = gen(T)
    for tb in (False, True):
        for dtype in (torch.int32, torch.int64):
            A, B, targets, skip = make(T, H, V, tb, g, ignored=0.5, dtype=dtype)
            none = skip.nonzero().squeeze(1)
            for i, bad in enumerate((-1, V, torch.iinfo(dtype).max, torch.iinfo(dtype).min)):
                targets[none[i::4]] = bad
            dloss = torch.randn(T, device="cuda", generator=g)
            lse = torch.empty(T, device="cuda")
            loss = sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse)
            want = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb)
            check_loss(loss, lse, A, B, targets, tb)
            for bad in (float("nan"), float("inf")):
                A2, d2, l2 = A.clone(), dloss.clone(), lse.clone()
                A2[skip], d2[skip], l2[skip] = bad, bad, bad
                got = torch.empty(T, device="cuda")
                assert torch.equal(sg.linear_cross_entropy(A2, B, targets, transpose_b=tb,
                                                           lse=got), loss)
                assert torch.equal(got, lse)
                for x, y in zip(sg.linear_cross_entropy_backward(d2, A2, B, targets, l2,
                                                                 transpose_b=tb), want):
                    assert torch.equal(x, y)
            # no row counts
            targets.fill_(-1)
            assert (sg.linear_cross_entropy(A, B, targets, transpose_b=tb) == 0).all()
            dA, dB = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb)
            assert (dA == 0).all() and (dB == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [17, 63, 64, 65, 256, 257, 511, 1023, 1024, 1025])
def test_rows_are_numbered(T):
    """Up to 1024 by a wave each."""
    for H, ignored in ((1030, 0.5), (3, 0.9), (2049, 0.0)):
        run(T, H, 60, H > 3, ignored=ignored, dtype=torch.int32 if H == 3 else torch.int64, seed=T)


@pytest.mark.gpu
def test_more_rows_than_one_workgroup_numbers_at_a_time():
    """Rows with a target in every pattern: 200000 tokens, 1024 a workgroup."""
    g = gen(55)
    T, H, V = 200000, 8, 40
    A, B, targets, _ = make(T, H, V, True, g, ignored=0.5)
    targets[3000:9000] = -1
    targets[20000:27000] = 3
    lse, dloss = torch.empty(T, device="cuda"), torch.randn(T, device="cuda", generator=g)
    loss = sg.linear_cross_entropy(A, B, targets, transpose_b=True, lse=lse)
    check_loss(loss, lse, A, B, targets, True)
    dA, dB = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=True)
    wA, wB, tA, tB = grads64(dloss, A, B, targets, lse, True)
    near(dA, wA, tA, "dA")
    near(dB, wB, tB, "dB")


@pytest.mark.gpu
def test_empty_sizes():
    for tb in (False, True):
        A, B = torch.randn(5, 8, device="cuda"), torch.randn(8, 6, device="cuda")
        B = B.t().contiguous() if tb else B
        none = torch.empty(0, dtype=torch.int64, device="cuda")
        f = torch.empty(0, device="cuda")
        assert sg.linear_cross_entropy(A[:0], B, none, transpose_b=tb).shape == (0,)
        dA, dB = sg.linear_cross_entropy_backward(f, A[:0], B, none, f, transpose_b=tb)
        assert dA.shape == (0, 8) and dB.shape == B.shape and (dB == 0).all()
        # no vocabulary
        t = torch.zeros(5, dtype=torch.int64, device="cuda")
        E = B[:0] if tb else B[:, :0]
        lse = torch.empty(5, device="cuda")
        assert (sg.linear_cross_entropy(A, E, t, transpose_b=tb, lse=lse) == 0).all()
        dA, dB = sg.linear_cross_entropy_backward(lse, A, E, t, lse, transpose_b=tb)
        assert (dA == 0).all() and dB.shape == E.shape
        # nothing to sum: equal logits
        E = B[:, :0] if tb else B[:0]
        loss = sg.linear_cross_entropy(A[:, :0], E, t, transpose_b=tb, lse=lse)
        near(loss, torch.full((5,), math.log(6)).double().cuda(), 16 * U, "loss")
        dA, dB = sg.linear_cross_entropy_backward(loss, A[:, :0], E, t, lse, transpose_b=tb)
        assert dA.shape == (5, 0) and dB.shape == E.shape


@pytest.mark.gpu
def test_one_gradient_alone():
    g = gen(4)
    for tb in (False, True):
        A, B, targets, _ = make(200, 70, 3000, tb, g, ignored=0.2)
        lse, dloss = torch.empty(200, device="cuda"), torch.randn(200, device="cuda", generator=g)
        sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse)
        want = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb)
        for a, b in ((True, False), (False, True), (False, False)):
            got = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb,
                                                   a_grad=a, b_grad=b)
            for w, x, asked in zip(want, got, (a, b)):
                assert torch.equal(w, x) if asked else x is None


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, 30.0, 2000.0])
def test_equal_and_far_logits(scale):
    run(50, 64, 1000, scale=scale, seed=3)
    run(50, 64, 1000, tb=False, scale=scale, seed=4)


@pytest.mark.gpu
def test_infinite_and_nan_logits():
    inf, nan = float("inf"), float("nan")
    g = gen(6)
    T, H, V = 6, 4, 300
    A = torch.zeros(T, H, device="cuda")
    A[:, 0] = torch.tensor([1.0, -1.0, 1.0, 1.0, 1.0, 0.5], device="cuda")
    B = torch.zeros(H, V, device="cuda")
    B[0] = torch.randn(V, device="cuda", generator=g)
    t = torch.tensor([3, 3, 290, 3, 3, 3], device="cuda")
    lse = torch.empty(T, device="cuda")
    base = sg.linear_cross_entropy(A, B, t, lse=lse).clone()
    for B2, tb in ((B.clone(), False), (B.t().contiguous(), True)):
        col = B2[290] if tb else B2[:, 290]
        col[0] = inf      # column 290: +inf where A is positive, -inf in row 1
        loss = sg.linear_cross_entropy(A, B2, t, transpose_b=tb, lse=lse)
        up = torch.tensor([0, 2, 3, 4, 5], device="cuda")
        assert (lse[up] == inf).all() and torch.isfinite(lse[1]) and torch.isfinite(loss[1])
        assert (loss[[0, 3, 4, 5]] == inf).all() and loss[2].isnan()
        z = (A[1:2, :1] * B[:1]).double()
        z[0, 290] = -inf
        near(lse[1:2], torch.logsumexp(z, 1), 80 * U * (1 + z[z > -inf].abs().max()), "lse")
        col[0] = nan
        loss = sg.linear_cross_entropy(A, B2, t, transpose_b=tb, lse=lse)
        assert lse.isnan().all() and loss.isnan().all()
    # a row's NaN stays in its row
    A[2, 1] = nan
    loss = sg.linear_cross_entropy(A, B, t, lse=lse)
    rows = torch.tensor([0, 1, 3, 4, 5], device="cuda")
    assert loss[2].isnan() and torch.equal(loss[rows], base[rows])


# Few rows, with their logits by tiles, by rows and in planes; a split K's planes; tiles.
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V", [(6, 4, 300), (1, 1024, 32768), (8, 300, 2000), (15, 4000, 600),
                                   (16, 256, 9001), (19, 2894, 3306), (200, 100, 3000),
                                   (1500, 512, 2600)])
@pytest.mark.parametrize("tb", [False, True])
def test_gradients_of_rows_with_an_infinite_logit(T, H, V, tb):
    """One infinite weight makes a logit of a row +inf (then lse is, p is 0 at the
    others and NaN there) or -inf (p is 0 there).  dB is NaN in that weight's column
    alone, dA in the rows whose p is, and where 0 meets the weight."""
    inf, col = float("inf"), min(V - 1, 290)
    g = gen(T + V)
    A, B, targets, skip = make(T, H, V, tb, g, ignored=0.3 if T > 6 else 0.0)
    targets[targets == col] = 0
    A[:, 0] = torch.where(torch.arange(T, device="cuda") % 3 == 1, -1.0, 1.0) + 0.1 * A[:, 0]
    (B[col] if tb else B[:, col])[0] = inf
    lse, dloss = torch.empty(T, device="cuda"), torch.randn(T, device="cuda", generator=g)
    sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse)
    up, kept = (A[:, 0] > 0) & ~skip, ~skip
    assert (lse[up] == inf).all() and torch.isfinite(lse[~up]).all()

    a = torch.where(kept[:, None], A, 0.0).double()
    b = (B.t() if tb else B).double()
    finite = b.clone()
    finite[0, col] = 0.0
    z = a @ finite
    z[:, col] = torch.where(up, inf, -inf)
    e = sum_tol(H) * (a.abs() @ finite.abs())
    l, d = torch.where(kept, lse, 0.0).double()[:, None], torch.where(kept, dloss, 0.0).double()
    p = torch.where(kept[:, None], torch.exp(z - l), 0.0)
    hit = torch.zeros_like(p)
    hit[kept, targets[kept].long()] = 1.0
    dz = (p - hit) * d[:, None]
    # as in grads64, where p is not 0
    rel = torch.where(p > 0, e + 2.3 * U * (z - l).abs() + 10 * U, 0.0)
    tiny = 2.0 ** -126
    dtol = d.abs()[:, None] * (p * (rel + rel * rel) + 2 * U * (p + hit) + tiny) + tiny
    wB, tB = a.t() @ dz, a.abs().t() @ dtol + sum_tol(T) * (a.abs().t() @ dz.abs()) + 2 * T * tiny
    pieces = max(64, V // 256 + 1)
    wA = dz @ finite.t()
    tA = dtol @ finite.abs().t() + (sum_tol(V) + pieces * U) * (dz.abs() @ finite.abs().t())
    tA = tA + 2 * V * tiny
    wA[kept & ~up, 0] = float("nan")      # 0 times the weight
    least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
    for ws in (None, torch.empty(least // 4, device="cuda")):
        dA, dB = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=tb,
                                                  workspace=ws)
        dB = dB.t() if tb else dB
        assert (dA[skip] == 0).all()
        assert torch.equal(dA.isnan(), wA.isnan()) and dA[up].isnan().all()
        near(dA.nan_to_num(0), wA.nan_to_num(0), tA.nan_to_num(0), "dA")
        here = torch.arange(V, device="cuda") == col
        if up.any():
            assert dB[:, here].isnan().all()
        assert torch.isfinite(dB[:, ~here]).all()
        near(dB[:, ~here], wB[:, ~here], tB[:, ~here], "dB")


@pytest.mark.gpu
@pytest.mark.parametrize("tb", [False, True])
def test_gradients_against_differences(tb):
    """The loss sum(loss * C) moved along a direction: the 64-bit forward's central
    difference against the gradients."""
    g = gen(12)
    T, H, V = 60, 48, 700
    A, B, targets, skip = make(T, H, V, tb, g, ignored=0.2)
    C = torch.randn(T, device="cuda", generator=g)
    lse = torch.empty(T, device="cuda")
    sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse)
    grads = sg.linear_cross_entropy_backward(C, A, B, targets, lse, transpose_b=tb)
    rows = (~skip).nonzero().squeeze(1)

    def loss(a, b):
        z = a[rows] @ (b.t() if tb else b)
        hit = z.gather(1, targets[rows][:, None]).squeeze(1)
        return ((torch.logsumexp(z, 1) - hit) * C[rows].double()).sum()

    base = [A.double(), B.double()]
    for i, d in enumerate(grads):
        v = torch.randn(d.shape, device="cuda", generator=g).double()
        h, up, dn = 1e-5, list(base), list(base)
        up[i], dn[i] = base[i] + h * v, base[i] - h * v
        num = ((loss(*up) - loss(*dn)) / (2 * h)).item()
        terms = (d.double() * v).abs().sum().item()
        assert abs((d.double() * v).sum().item() - num) <= (1e-5 + 1e-6) * terms


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V,tb", [(1, 64, 500, True), (200, 100, 3000, False),
                                      (19, 2894, 3306, False), (4, 1024, 32768, True),
                                      (12, 300, 5000, True), (16, 200, 9001, False),
                                      (2048, 1024, 8192, True)])
def test_replays_from_a_graph_with_other_targets(T, H, V, tb):
    g = gen(T + V)
    A, B, targets, _ = make(T, H, V, tb, g, ignored=0.3)
    dloss, lse = torch.randn(T, device="cuda", generator=g), torch.empty(T, device="cuda")
    ws = torch.empty(max(sg.sgemm_linear_xent_workspace_bytes(tb, T, V, H),
                         sg.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H)) // 4,
                     device="cuda")

    def step(**kw):
        loss = sg.linear_cross_entropy(A, B, targets, transpose_b=tb, lse=lse, workspace=ws, **kw)
        return (loss, lse, *sg.linear_cross_entropy_backward(dloss, A, B, targets, lse,
                                                             transpose_b=tb, workspace=ws, **kw))

    want = [o.clone() for o in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        A.normal_(generator=g)
        targets.random_(-V if rep % 2 else 0, V, generator=g)      # half of them none, or all
        for o in out:
            o.fill_(float("nan"))
        ws.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for x, y in zip(got, step()):
            assert torch.equal(x, y), rep


@pytest.mark.gpu
def test_operands_past_32_bits():
    g = gen(21)
    # T V logits and their strips past 2^32 bytes, of few values a row
    T, H, V = 70000, 16, 65000
    A, B, targets, _ = make(T, H, V, True, g, ignored=0.1)
    lse = torch.empty(T, device="cuda")
    loss = sg.linear_cross_entropy(A, B, targets, transpose_b=True, lse=lse)
    for part in (slice(0, 300), slice(T - 300, T)):
        check_loss(loss[part], lse[part], A[part], B, targets[part], True)
    dloss = torch.randn(T, device="cuda", generator=g)
    dA, dB = sg.linear_cross_entropy_backward(dloss, A, B, targets, lse, transpose_b=True)
    for part in (slice(0, 300), slice(T - 300, T)):
        wA, _, tA, _ = grads64(dloss[part], A[part], B, targets[part], lse[part], True)
        near(dA[part], wA, tA, "dA")
    del A, B, dA, dB
    # a weight past 4 GiB
    T, H, V = 5, 1100, 1 << 20
    A, B, targets, _ = make(T, H, V, True, g)
    targets[0], targets[1] = V - 1, V - 70000
    lse = torch.empty(T, device="cuda")
    loss = sg.linear_cross_entropy(A, B, targets, transpose_b=True, lse=lse)
    top = torch.stack([torch.logsumexp(A.double() @ B[i:i + 65536].double().t(), 1)
                       for i in range(0, V, 65536)])
    want = torch.logsumexp(top, 0)
    size = sum_tol(H) * (A.double().norm(dim=1) * B[:4096].double().norm(dim=1).max() * 1.5)
    near(lse, want, size + 700 * U * (1 + want.abs()), "lse")
    dA, dB = sg.linear_cross_entropy_backward(loss, A, B, targets, lse, transpose_b=True)
    for part in (slice(0, 2000), slice(V - 2000, V)):
        z = A.double() @ B[part].double().t()
        p = torch.exp(z - lse.double()[:, None])
        hit = torch.arange(part.start, part.stop, device="cuda") == targets[:, None]
        dz = (p - hit.double()) * loss.double()[:, None]
        # a part in 10^5 of the terms: the products' own bound and the exponential's
        tol = 3e-5 * ((p + hit.double()) * loss.double().abs()[:, None]).t() @ A.double().abs()
        near(dB[part], dz.t() @ A.double(), tol, "dB")


@pytest.mark.gpu
def test_two_streams_have_their_own_workspaces():
    g = gen(33)
    ins = [make(300, 256, 3000, tb, g, ignored=0.2) for tb in (True, False)]
    want, lses = [], []
    for (A, B, t, _), tb in zip(ins, (True, False)):
        lse = torch.empty(300, device="cuda")
        loss = sg.linear_cross_entropy(A, B, t, transpose_b=tb, lse=lse)
        lses.append(lse)
        want.append((loss, *sg.linear_cross_entropy_backward(loss, A, B, t, lse, transpose_b=tb)))
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (A, B, t, _), tb, s, lse in zip(ins, (True, False), streams, lses):
            loss = sg.linear_cross_entropy(A, B, t, transpose_b=tb, stream=s)
            got.append((loss, *sg.linear_cross_entropy_backward(loss, A, B, t, lse, transpose_b=tb,
                                                                stream=s)))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for x, y in zip(o, want[i % 2]):
            assert torch.equal(x, y)


# Refusals (CPU).

BIG = 1 << 33
FAR = BIG + (1 << 40)


@pytest.fixture(scope="module")
def lib():
    from tiled_fp32_gemm_amd import build
    build.ensure_built()
    return sg.load()


def forward(tb=0, T=4, V=16, H=8, X=BIG, ldx=None, B=BIG + (1 << 34), ldb=None, t=BIG + (1 << 35),
            b=8, loss=FAR, lse=FAR * 2, ws=FAR * 3, nb=1 << 20):
    ldx = max(H, 1) if ldx is None else ldx
    ldb = max(H if tb else V, 1) if ldb is None else ldb
    return sg.sgemm_linear_xent(tb, T, V, H, X, ldx, B, ldb, t, b, loss, lse, 0, ws, nb)


def backward(tb=0, T=4, V=16, H=8, X=BIG, ldx=None, B=BIG + (1 << 34), ldb=None,
             t=BIG + (1 << 35), b=8, lse=BIG + (1 << 36), d=BIG + (1 << 37), dX=FAR, lddx=None,
             dB=FAR * 2, lddb=None, ws=FAR * 3, nb=1 << 20):
    ldx = max(H, 1) if ldx is None else ldx
    lddx = max(H, 1) if lddx is None else lddx
    ldb = max(H if tb else V, 1) if ldb is None else ldb
    lddb = max(H if tb else V, 1) if lddb is None else lddb
    return sg.sgemm_linear_xent_backward(tb, T, V, H, X, ldx, B, ldb, t, b, lse, d, dX, lddx, dB,
                                         lddb, 0, ws, nb)


COMMON = [dict(tb=2), dict(tb=-1), dict(T=-1), dict(V=-1), dict(H=-1), dict(ldx=7), dict(ldb=15),
          dict(tb=1, ldb=7), dict(b=2), dict(b=0), dict(X=0), dict(B=0), dict(t=0),
          dict(X=BIG + 2), dict(B=BIG + (1 << 34) + 1), dict(t=BIG + (1 << 35) + 4),
          dict(b=4, t=BIG + (1 << 35) + 2), dict(nb=-4), dict(nb=16), dict(nb=0), dict(ws=0),
          dict(ws=FAR * 3 + 2), dict(ws=BIG), dict(ws=BIG + (1 << 34)), dict(ws=BIG + (1 << 35))]


@pytest.mark.parametrize("args", COMMON + [
    dict(loss=0), dict(loss=FAR + 1), dict(lse=FAR * 2 + 2), dict(lse=FAR), dict(loss=BIG),
    dict(lse=BIG + (1 << 34)), dict(loss=BIG + (1 << 35) + 16), dict(ws=FAR), dict(ws=FAR * 2)])
def test_loss_refuses(lib, args):
    assert forward(**args) == sg.ERR_INVALID_ARG


@pytest.mark.parametrize("args", COMMON + [
    dict(lse=0), dict(d=0), dict(lse=BIG + (1 << 36) + 1), dict(d=BIG + (1 << 37) + 2),
    dict(dX=FAR + 2), dict(dB=FAR * 2 + 1), dict(lddx=7), dict(lddb=15), dict(tb=1, lddb=7),
    dict(dX=BIG), dict(dX=BIG + (1 << 34)), dict(dB=BIG + (1 << 34)), dict(dB=BIG + (1 << 36)),
    dict(dX=BIG + (1 << 37)), dict(dB=FAR + 64), dict(ws=FAR), dict(ws=FAR * 2 + 4)])
def test_backward_refuses(lib, args):
    assert backward(**args) == sg.ERR_INVALID_ARG


def test_unsupported_and_nothing_to_do(lib):
    most = 1 << 20
    huge = dict(B=FAR * 5, X=FAR * 6, t=FAR * 7)
    for f in (forward, backward):
        assert f(T=1 << 31, **huge) == sg.ERR_UNSUPPORTED
        assert f(V=most + 1, **huge) == sg.ERR_UNSUPPORTED
        assert f(H=most + 1, **huge) == sg.ERR_UNSUPPORTED
        assert f(ldx=most + 1, **huge) == sg.ERR_UNSUPPORTED
        assert f(ldb=most + 1, **huge) == sg.ERR_UNSUPPORTED
    assert backward(lddb=most + 1) == sg.ERR_UNSUPPORTED
    assert forward(T=0, X=0, t=0, loss=0, lse=0, ws=0, nb=0) == sg.OK
    assert backward(dX=0, dB=0) == sg.OK
    assert backward(H=0, X=0, B=0) == sg.OK
    for sizes in ((2, 4, 4, 4), (0, -1, 4, 4), (0, 4, -1, 4), (0, 4, 4, -1), (0, 1 << 31, 4, 4),
                  (0, 4, most + 1, 4), (0, 4, 4, most + 1)):
        assert sg.sgemm_linear_xent_workspace_bytes(*sizes) == 0
        assert sg.sgemm_linear_xent_backward_workspace_bytes(*sizes) == 0
        assert sg.sgemm_linear_xent_backward_least_bytes(*sizes) == 0


def test_workspaces_hold_no_logits(lib):
    """Less than a tenth of T x V, and no less than is said to be enough."""
    T, V, H = 16384, 131072, 1024
    for tb in (0, 1):
        assert sg.sgemm_linear_xent_workspace_bytes(tb, T, V, H) < 4 * T * V // 10
        full = sg.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H)
        least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
        assert least < full < 4 * T * V // 10
        args = dict(tb=tb, T=T, V=V, H=H, X=FAR * 5, B=FAR * 6, t=FAR * 7, dX=FAR * 8, dB=FAR * 9)
        assert backward(nb=least - 4, **args) == sg.ERR_INVALID_ARG


ODD = [(17, 301, 64), (19, 333, 2894), (7, 1001, 30), (23, 517, 33), (1, 3, 5), (40, 263, 100)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
@pytest.mark.parametrize("T,V,H", ODD)
@pytest.mark.parametrize("tb", [0, 1])
def test_every_workspace_from_the_least_on_is_enough(lib, T, V, H, tb):
    """T V need not be a multiple of four floats.  (Accepted, a call fails at its launch.)"""
    least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
    most = sg.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H)
    piece = 4 * T * V      # the whole vocabulary's, and each plane's
    near = [n + d for n in range(least, most + 2 * piece, piece) for d in range(-64, 256, 4)]
    sizes = near + [most + d for d in range(-64, 64, 4)] + list(range(least, most + 64, 116))
    sizes += list(range(least, least + 40000, 4)) + [least + d for d in (1, 2, 3, 5, 17)]
    assert backward(tb, T, V, H, nb=least - 1) == sg.ERR_INVALID_ARG
    for nb in sizes:
        if nb >= least:
            assert backward(tb, T, V, H, nb=nb) == sg.ERR_LAUNCH, (nb, least, most)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", ODD)
@pytest.mark.parametrize("tb", [False, True])
def test_workspaces_around_a_whole_vocabulary(T, V, H, tb):
    least = sg.sgemm_linear_xent_backward_least_bytes(tb, T, V, H)
    whole = least + 4 * T * max(V - 256, 0)
    for ws in range(max(least, whole - 16), whole + 36, 4):
        run(T, H, V, tb, ignored=0.3, ws=ws, seed=T)
    for planes in (2, 3):
        for d in range(0, 16, 4):
            run(T, H, V, tb, ws=whole + 4 * (planes - 1) * T * V + d, seed=V)


@pytest.mark.parametrize("tb", [0, 1])
def test_rows_that_no_launch_copies_stay_where_they_are(lib, tb):
    """From 2^34 values on: the loss takes them without copying them together, the
    gradients refuse them before any launch."""
    T, V, H = 1 << 23, 1000, 2048
    assert sg.sgemm_linear_xent_workspace_bytes(tb, T - 1, V, H) > 4 * (T - 1) * H     # copied
    assert sg.sgemm_linear_xent_workspace_bytes(tb, T, V, H) < 4 * T * H // 20
    far = dict(X=FAR * 5, B=FAR * 6, t=FAR * 7, nb=1 << 45)
    assert backward(tb, T, V, H, lse=FAR * 8, d=FAR * 9, dX=FAR * 10, dB=FAR * 11, ws=FAR * 64,
                    **far) == sg.ERR_UNSUPPORTED


def test_the_header_declares_the_binding_names(lib):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "sgemm_xent.h")).read(),
                  flags=re.S)
    found = re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, re.M)
    assert sorted(found) == sorted(sg.XENT_SYMBOLS)
    for n in found:
        assert hasattr(lib, n) and hasattr(sg, n)


def test_the_binding_refuses_what_is_no_gpu_tensor():
    A, B, t = torch.randn(4, 8), torch.randn(8, 9), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="on a GPU"):
        sg.linear_cross_entropy(A, B, t)
    with pytest.raises(ValueError, match="on a GPU"):
        sg.linear_cross_entropy_backward(A[:, 0], A, B, t, A[:, 0])


@pytest.mark.gpu
def test_the_binding_refuses_bad_tensors():
    A, B = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 9, device="cuda")
    t, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    for args in ((A.half(), B, t), (A, B.double(), t), (A, B[:4], t), (A, B, t[:3]),
                 (A, B, t.float()), (A, B, t.short()), (A, B, t.cpu()), (A, B, t[None]),
                 (A[0], B, t), (A, B.t(), t), (A, B, None)):
        with pytest.raises(ValueError):
            sg.linear_cross_entropy(*args)
    with pytest.raises(ValueError):
        sg.linear_cross_entropy(A, B, t, transpose_b=True)
    for kw in (dict(lse=f[:3]), dict(lse=f.double()), dict(out=torch.zeros(5, device="cuda")),
               dict(workspace=torch.zeros(4))):
        with pytest.raises(ValueError):
            sg.linear_cross_entropy(A, B, t, **kw)
    for args in ((f[:3], A, B, t, f), (f, A, B, t, f[:3]), (f.half(), A, B, t, f),
                 (f.sum().expand(4), A, B, t, f), (f, A, B, t, None)):
        with pytest.raises(ValueError):
            sg.linear_cross_entropy_backward(*args)
    small = torch.zeros(2, device="cuda")
    with pytest.raises(sg.SgemmError):
        sg.linear_cross_entropy(A, B, t, workspace=small)
    with pytest.raises(sg.SgemmError):
        sg.linear_cross_entropy_backward(f, A, B, t, f, workspace=small)
