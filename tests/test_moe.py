"""Expert routing and the experts' products, against plain definitions: the
sort and the moves exactly (a weighted sum of `top` rows within top + 1
roundings), the products within the bounds of test_linear.py."""
from __future__ import annotations

import pytest

import tiled_fp32_gemm_amd as sg
from test_linear import ACTS, U, act64, gen, slope64, sum_tol, wide

torch = pytest.importorskip("torch")


def plain_sort(ids, E):
    flat = ids.reshape(-1).tolist()
    buckets = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            buckets[e].append(i)
    offsets, order, place = [0], [], [-1] * len(flat)
    for b in buckets:
        for i in b:
            place[i] = len(order)
            order.append(i)
        offsets.append(len(order))
    order += [-1] * (len(flat) - len(order))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(order, dtype=torch.int32),
            torch.tensor(place, dtype=torch.int32).reshape(ids.shape))


def check_sort(ids, E, **kw):
    got = sg.moe_sort(ids, E, **kw)
    for g, w in zip(got, plain_sort(ids.cpu(), E)):
        assert torch.equal(g.cpu(), w)
    return got


SORTS = [(1, 1, 1), (1, 2, 8), (16, 2, 8), (7, 3, 5), (64, 1, 64), (65, 1, 65), (1000, 2, 16),
         (4095, 2, 64), (4096, 2, 64), (4097, 2, 64), (8191, 4, 128), (5000, 8, 1000),
         (20000, 1, 1024), (100000, 2, 3), (300000, 4, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,top,E", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, top, E, dtype):
    g = gen(T + E)
    ids = torch.randint(0, E, (T, top), device="cuda", generator=g).to(dtype)
    check_sort(ids, E)
    # dropped choices of every kind, and a workspace of the caller's
    ids[torch.rand(T, top, device="cuda", generator=g) < 0.2] = -1
    ids[torch.rand(T, top, device="cuda", generator=g) < 0.1] = E
    ids[0, 0] = torch.iinfo(dtype).max
    ids[-1, -1] = torch.iinfo(dtype).min
    ws = torch.full((1 << 20,), -7, dtype=torch.int32, device="cuda")
    check_sort(ids, E, workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 63, 64, 1000, 8192, 8193, 70000])
def test_sort_of_one_expert_of_none_and_of_equal_ids(n):
    check_sort(torch.zeros(n, 1, dtype=torch.int64, device="cuda"), 1)
    check_sort(torch.full((n, 1), 4, dtype=torch.int32, device="cuda"), 9)
    check_sort(torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), 9)
    check_sort(torch.arange(n, device="cuda").flip(0).reshape(n, 1), min(n, 1024))
    check_sort(torch.arange(n, device="cuda", dtype=torch.int32) % 2 * 1023, 1024)   # 1-D


@pytest.mark.gpu
def test_sort_of_nothing():
    offsets, order, place = sg.moe_sort(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 5)
    assert offsets.tolist() == [0] * 6 and order.numel() == 0 and place.shape == (0, 2)


def route(T, top, E, drop, g):
    ids = torch.randint(0, E, (T, top), device="cuda", generator=g)
    if drop:
        ids[torch.rand(T, top, device="cuda", generator=g) < 0.3] = -1
        ids[0] = -1       # a token without any expert
    return ids


MOVES = [(1, 1, 1), (1, 2, 16), (3, 2, 5), (16, 2, 1024), (100, 3, 777), (33, 8, 130),
         (257, 1, 64), (50, 5, 4099), (1000, 2, 20), (300, 9, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,top,H", MOVES)
@pytest.mark.parametrize("drop", [False, True])
def test_moves_and_their_gradients(T, top, H, drop):
    g = gen(T * H)
    for pad, off in ((0, 0), (3, 1)):
        ids = route(T, top, 8, drop, g)
        offsets, order, place = sg.moe_sort(ids, 8)
        kept = int(offsets[-1])
        rows = order[:kept].long()
        tok = rows // top
        X = wide(T, H, pad, off, g)
        out = wide(T * top, H, pad, off, g, fill=7.0)
        before = out.clone()
        assert sg.moe_permute(X, place, out=out) is out
        assert torch.equal(out[:kept], X[tok])
        assert torch.equal(out[kept:], before[kept:])      # rows of no expert stay
        # back
        w = torch.rand(T, top, device="cuda", generator=g)
        Yp = wide(T * top, H, pad, off, g)
        Yp[kept:] = float("nan")                            # never read
        for weights in (w, None):
            Y = sg.moe_unpermute(Yp, place, weights, out=wide(T, H, pad, off, g))
            ww = torch.ones_like(w) if weights is None else w
            terms = ww.reshape(-1)[rows].double()[:, None] * Yp[:kept].double()
            want = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, tok, terms)
            size = torch.zeros_like(want).index_add_(0, tok, terms.abs())
            assert ((Y.double() - want).abs() <= (top + 1) * U * size).all()
            # its gradients
            dY = wide(T, H, pad, off, g)
            dyp = wide(T * top, H, pad, off, g, fill=7.0)
            before = dyp.clone()
            got, dw = sg.moe_unpermute_backward(dY, Yp, place, weights, out=dyp)
            assert torch.equal(got[:kept], ww.reshape(-1)[rows][:, None] * dY[tok])
            assert torch.equal(got[kept:], before[kept:])
            prod = dY[tok].double() * Yp[:kept].double()
            want = torch.zeros(T * top, dtype=torch.float64, device="cuda")
            size = torch.zeros_like(want)
            want[rows], size[rows] = prod.sum(1), prod.abs().sum(1)
            assert ((dw.reshape(-1).double() - want).abs() <= sum_tol(H) * size).all()
            assert (dw.reshape(-1)[place.reshape(-1) < 0] == 0).all()
            # in place over the rows
            over = Yp.clone()
            got2, dw2 = sg.moe_unpermute_backward(dY, over, place, weights, out=over)
            assert torch.equal(got2[:kept], got[:kept]) and torch.equal(dw2, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,H", [(1, 3, 5), (40, 4, 33), (9000, 16, 20)])
def test_one_choice_a_token_in_one_dimension(T, E, H):
    g = gen(T)
    ids = torch.randint(-1, E, (T,), device="cuda", generator=g)
    offsets, order, place = sg.moe_sort(ids, E)
    x, dy = (torch.randn(T, H, device="cuda", generator=g) for _ in range(2))
    w = torch.rand(T, device="cuda", generator=g)
    flat, column = [], []
    for out, p, weights in ((flat, place, w), (column, place[:, None], w[:, None])):
        xp = sg.moe_permute(x, p, out=torch.zeros(T, H, device="cuda"))
        dyp, dw = sg.moe_unpermute_backward(dy, xp, p, weights, out=torch.zeros_like(xp))
        out += [xp, sg.moe_unpermute(xp, p, weights), sg.moe_unpermute(xp, p), dyp, dw]
    assert flat[-1].shape == (T,)
    column[-1] = column[-1][:, 0]
    for a, b in zip(flat, column):
        assert torch.equal(a, b)
    kept = (ids >= 0).float()[:, None]
    assert torch.equal(flat[2], x * kept) and torch.equal(flat[1], w[:, None] * x * kept)
    for bad in (w[:, None], w[: T - 1]):
        with pytest.raises(ValueError):
            sg.moe_unpermute(flat[0], place, bad)
    with pytest.raises(ValueError):
        sg.moe_permute(x, place.reshape(1, T, 1))


@pytest.mark.gpu
def test_places_outside_the_rows_count_as_dropped():
    g = gen(2)
    place = torch.tensor([[0, 1], [6, -5], [2, 1 << 30], [-(1 << 31), 3]], dtype=torch.int32,
                         device="cuda")
    place[1, 0] = 8     # T·top
    X, Yp = torch.randn(4, 33, device="cuda", generator=g), torch.randn(8, 33, device="cuda",
                                                                        generator=g)
    out = sg.moe_permute(X, place, out=torch.zeros(8, 33, device="cuda"))
    assert torch.equal(out[:4], X[[0, 0, 2, 3]]) and (out[4:] == 0).all()
    Y = sg.moe_unpermute(Yp, place)
    assert torch.equal(Y[1], torch.zeros(33, device="cuda")) and torch.equal(Y[2], Yp[2])
    dyp, dw = sg.moe_unpermute_backward(X, Yp, place, out=torch.zeros(8, 33, device="cuda"))
    assert torch.equal(dyp[:4], X[[0, 0, 2, 3]]) and (dyp[4:] == 0).all()
    assert dw[1].tolist() == [0, 0] and dw[2, 1] == 0 and dw[3, 0] == 0


# Grouped products.

def offsets_of(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32,
                        device="cuda")


GROUPS = [([1], 8, 8), ([5], 33, 17), ([0, 3, 0], 20, 9), ([1, 1, 1, 1], 64, 100),
          ([4, 0, 7, 2, 0, 0, 1, 9], 130, 70), ([33, 64, 1, 0, 95], 96, 65),
          ([130, 0, 200], 200, 128), ([16] * 8, 512, 256), ([2, 9, 0, 300, 1, 17], 257, 1000),
          ([0, 0], 10, 10), ([3] * 70, 40, 30), ([1000, 5], 72, 0), ([7] + [0] * 200 + [1], 65, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", GROUPS)
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("behind", [0, 6])
def test_grouped_linear_and_its_gradients(counts, N, K, tb, behind):
    g = gen(sum(counts) + N)
    G, kept = len(counts), sum(counts)
    M = kept + behind
    offsets = offsets_of(counts)
    of = torch.repeat_interleave(torch.arange(G, device="cuda"),
                                 torch.tensor(counts, device="cuda"))
    for i, (act, pad, ws_bytes) in enumerate((("gelu", 0, 0), ("silu", 3, 1 << 23),
                                              ("none", 1, 1 << 23))):
        A = wide(M, K, pad, i, g)
        A[kept:] = float("nan")
        r, c = (N, K) if tb else (K, N)
        B = wide(G * (r + 1), c, pad, i, g, max(K, 1) ** -0.5).unflatten(0, (G, r + 1))[:, :r]
        bias = wide(G, N, pad, i, g) if i != 2 else None
        R = wide(M, N, pad, i, g) if i != 0 else None
        out, Z = wide(M, N, pad, i, g, fill=7.0), wide(M, N, pad, i, g, fill=7.0)
        before = out.clone(), Z.clone()
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
        sg.grouped_linear(A, B, offsets, bias, act, R, transpose_b=tb, out=out, preact=Z,
                          workspace=ws)
        b64 = (B.transpose(1, 2) if tb else B).double().contiguous()
        z = torch.zeros(kept, N, dtype=torch.float64, device="cuda")
        T = torch.zeros_like(z)
        for e in range(G):
            s = slice(*offsets[e:e + 2].tolist())
            z[s] = A[s].double() @ b64[e]
            T[s] = A[s].double().abs() @ b64[e].abs()
        if bias is not None:
            z, T = z + bias.double()[of], T + bias.double().abs()[of]
        ztol = sum_tol(K) * T
        assert ((Z[:kept].double() - z).abs() <= ztol).all()
        y = act64(act, z) + (R[:kept].double() if R is not None else 0)
        tol = 1.13 * ztol + 32 * U * z.abs() + U * y.abs()
        assert ((out[:kept].double() - y).abs() <= 1.001 * tol).all()
        assert torch.equal(out[kept:], before[0][kept:]) and torch.equal(Z[kept:], before[1][kept:])

        dC = wide(M, N, pad, i, g)
        dC[kept:] = float("nan")
        Z[kept:] = float("nan")
        dA, dB, db = sg.grouped_linear_backward(dC, A, B, offsets, act,
                                                None if act == "none" else Z, transpose_b=tb,
                                                workspace=ws)
        dz = dC[:kept].double() * slope64(act, Z[:kept].double())
        dtol = 64 * U * dC[:kept].double().abs()
        assert dB.shape == B.shape and db.shape == (G, N) and dA.shape == (M, K)
        for e in range(G):
            s = slice(*offsets[e:e + 2].tolist())
            n = counts[e]
            a, d, t = A[s].double(), dz[s], dtol[s]
            bt = b64[e].t()
            assert ((dA[s].double() - d @ bt).abs()
                    <= sum_tol(N) * (d.abs() @ bt.abs()) + t @ bt.abs()).all()
            got = (dB[e].t() if tb else dB[e]).double()
            assert ((got - a.t() @ d).abs()
                    <= sum_tol(n) * (a.abs().t() @ d.abs()) + a.abs().t() @ t).all()
            assert ((db[e].double() - d.sum(0)).abs()
                    <= sum_tol(n) * d.abs().sum(0) + t.sum(0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tb", [False, True])
def test_grouped_integers_are_exact_and_the_same_every_time(tb):
    g = gen(4)
    for counts, N, K in (([300, 0, 5, 700], 300, 200), ([4, 4, 1, 0, 3, 9], 512, 128),
                         ([20, 31, 64, 2], 128, 1024)):
        M, G = sum(counts), len(counts)
        draw = lambda *s: torch.randint(-8, 9, s, device="cuda", generator=g).float()  # noqa: E731
        A, B, b = draw(M, K), draw(G, *((N, K) if tb else (K, N))), draw(G, N)
        offsets = offsets_of(counts)
        of = torch.repeat_interleave(torch.arange(G, device="cuda"),
                                     torch.tensor(counts, device="cuda"))
        b64 = (B.transpose(1, 2) if tb else B).double().contiguous()
        edges = offsets.tolist()
        want = torch.cat([A[i:j].double() @ b64[e] for e, (i, j) in
                          enumerate(zip(edges, edges[1:]))]) + b.double()[of]
        ws = torch.empty(1 << 22, device="cuda")
        for w in (None, ws):
            for _ in range(2):
                assert torch.equal(sg.grouped_linear(A, B, offsets, b, transpose_b=tb,
                                                     workspace=w).double(), want)
        dC = draw(M, N)
        dA, dB, db = sg.grouped_linear_backward(dC, A, B, offsets, transpose_b=tb, workspace=ws)
        for e, (i, j) in enumerate(zip(edges, edges[1:])):
            d = dC[i:j].double()
            assert torch.equal(dA[i:j].double(), d @ b64[e].t().contiguous())
            w = A[i:j].double().t() @ d
            assert torch.equal(dB[e].double(), w.t() if tb else w)
            assert torch.equal(db[e].double(), d.sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,G,N,K", [(9000, 9, 2100, 64), (17000, 7, 4000, 100),
                                        (20000, 70, 2000, 64)])
def test_large_tiles_over_uneven_groups_are_exact(rows, G, N, K):
    """The 128- and 256-row tiles: whole ones first, partial ones by length (up
    to 64 groups), waves without rows."""
    g = gen(rows)
    draw = lambda *s: torch.randint(-8, 9, s, device="cuda", generator=g).float()  # noqa: E731
    p = torch.softmax(torch.randn(G, device="cuda", generator=g), 0)
    p[1] = 0
    counts = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g),
                            minlength=G).tolist()
    offsets = offsets_of(counts)
    edges = offsets.tolist()
    A, b, dC = draw(rows, K), draw(G, N), draw(rows, N)
    R = draw(rows, N)
    ws = torch.empty(1 << 24, device="cuda")
    for tb in (False, True):
        B = draw(G, *((N, K) if tb else (K, N)))
        C = sg.grouped_linear(A, B, offsets, b, "relu", R, transpose_b=tb, workspace=ws)
        dA, dB, db = sg.grouped_linear_backward(dC, A, B, offsets, transpose_b=tb, workspace=ws)
        for e, (i, j) in enumerate(zip(edges, edges[1:])):
            m = (B[e].t() if tb else B[e]).double()
            a, d = A[i:j].double(), dC[i:j].double()
            assert torch.equal(C[i:j].double(), (a @ m + b[e].double()).clamp(min=0) + R[i:j])
            assert torch.equal(dA[i:j].double(), d @ m.t())
            w = a.t() @ d
            assert torch.equal(dB[e].double(), w.t() if tb else w)
            assert torch.equal(db[e].double(), d.sum(0))


# Few rows a group through an N x K stack over a long K: chunks of four and eight
# rows, more rows than a chunk, columns by fours (N = 300) and by sixteens.
@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1, 3, 0, 2, 0, 0, 4, 1], [3, 8, 0, 1, 5, 2], [11, 1, 4, 0],
                                    [9, 1, 0, 1, 0, 2]])
@pytest.mark.parametrize("N", [300, 2100])
@pytest.mark.parametrize("K", [2048, 2051, 4099])
def test_few_rows_a_group_over_a_long_k(counts, N, K):
    g = gen(N + K)
    G, kept = len(counts), sum(counts)
    offsets = offsets_of(counts)
    of = torch.repeat_interleave(torch.arange(G, device="cuda"),
                                 torch.tensor(counts, device="cuda"))
    for pad, off, act in ((0, 0, "none"), (1, 1, "silu")):
        A = wide(kept + 2, K, pad, off, g)
        A[kept:] = float("nan")
        B = wide(G * (N + 1), K, pad, off, g, K ** -0.5).unflatten(0, (G, N + 1))[:, :N]
        bias, R = wide(G, N, pad, off, g), wide(kept + 2, N, pad, off, g)
        out, Z = (wide(kept + 2, N, pad, off, g, fill=7.0) for _ in range(2))
        before = out.clone(), Z.clone()
        sg.grouped_linear(A, B, offsets, bias, act, R, transpose_b=True, out=out, preact=Z)
        z = torch.empty(kept, N, dtype=torch.float64, device="cuda")
        T = torch.empty_like(z)
        for e in range(G):
            s, b = slice(*offsets[e:e + 2].tolist()), B[e].double().t().contiguous()
            z[s], T[s] = A[s].double() @ b, A[s].double().abs() @ b.abs()
        z, T = z + bias.double()[of], T + bias.double().abs()[of]
        ztol = sum_tol(K) * T
        assert ((Z[:kept].double() - z).abs() <= ztol).all()
        y = act64(act, z) + R[:kept].double()
        tol = 1.13 * ztol + 32 * U * z.abs() + U * y.abs()
        assert ((out[:kept].double() - y).abs() <= 1.001 * tol).all()
        assert torch.equal(out[kept:], before[0][kept:]) and torch.equal(Z[kept:], before[1][kept:])


# Weight gradients whose sum over a group's rows is split: one group with nearly
# all rows, empty ones, some shorter than a slab (so that splits are empty), more
# than sixteen (which go out in order) and more than a wave's.
SPLIT_SUMS = [([16000, 0, 5, 379], 64, 64), ([16000, 0, 5, 379], 128, 128),
              ([5990, 3, 7], 70, 36), ([1, 8900, 0, 2, 0, 97], 33, 65),
              ([0, 31, 32, 33, 1, 0, 38000, 64, 65, 5, 0, 700, 2, 3, 0, 900, 164, 0, 0, 0], 100, 60),
              ([2, 0] * 34 + [59000, 932], 20, 20)]


def test_sums_over_groups_are_split(lib):
    for counts, N, K in SPLIT_SUMS:
        for tb in (0, 1):
            size = 4 * N * K * len(counts)
            need = sg.sgemm_grouped_wgrad_workspace_bytes(tb, sum(counts), N, K, len(counts))
            assert need >= 2 * size and need % size == 0, (counts, N, K, tb)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", SPLIT_SUMS)
@pytest.mark.parametrize("tb", [False, True])
def test_split_sums_over_uneven_groups_are_exact_and_replay(counts, N, K, tb):
    g = gen(N)
    M, G = sum(counts), len(counts)
    draw = lambda *s: torch.randint(-8, 9, s, device="cuda", generator=g).float()  # noqa: E731
    # 60000 products of at most 64 stay below 2^24
    A, dC, B = draw(M + 3, K), draw(M + 3, N), draw(G, *((N, K) if tb else (K, N)))
    A[M:], dC[M:] = float("nan"), float("nan")
    need = sg.sgemm_grouped_wgrad_workspace_bytes(tb, M + 3, N, K, G)
    assert need > 0

    def want(offsets):
        edges = offsets.tolist()
        w = torch.stack([A[i:j].double().t().contiguous() @ dC[i:j].double()
                         for i, j in zip(edges, edges[1:])])
        return w.transpose(1, 2) if tb else w

    offsets = offsets_of(counts)
    exact = want(offsets)
    for room in (need, need // 2, 0):
        ws = torch.full((room // 4,), float("nan"), device="cuda") if room else None
        for _ in range(2):
            dB = sg.grouped_linear_backward(dC, A, B, offsets, transpose_b=tb, workspace=ws)[1]
            assert torch.equal(dB.double(), exact), room
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    run = lambda: sg.grouped_linear_backward(dC, A, B, offsets, transpose_b=tb,  # noqa: E731
                                             workspace=ws)[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for other in (counts[::-1], counts, [M] + [0] * (G - 1), [0] * G):
        offsets.copy_(offsets_of(other))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.double(), want(offsets)), other
        assert torch.equal(run(), out)


def grouped_act(dC, Z, act, dZ, db, offsets, room, N):
    """sgemm_grouped_act_backward over every row of dC, in `room` floats."""
    ws = torch.full((room,), float("nan"), device="cuda") if room else None
    lead = lambda t: t.stride(0) if t is not None else 1  # noqa: E731
    ptr = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
    st = sg.sgemm_grouped_act_backward(
        dC.shape[0], N, offsets.numel() - 1, offsets.data_ptr(), ptr(dC), lead(dC), ptr(Z),
        lead(Z), sg.ACTIVATIONS[act], ptr(dZ), lead(dZ), ptr(db), lead(db),
        torch.cuda.current_stream().cuda_stream, ptr(ws), 4 * room)
    assert st == sg.OK


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N", [
    ([0, 0, 0], 40), ([5], 3), ([0, 2000, 0, 1, 37], 130), ([4000, 0, 16, 17], 33),
    ([3, 0, 9000, 200, 0, 0, 800], 300), ([64, 65, 0, 63, 128, 1], 1500),
    ([1, 0, 40] * 30 + [30000], 5), ([0] * 100 + [700, 0, 70000] + [0, 1] * 50, 64)])
def test_the_activation_pass_over_uneven_groups(counts, N):
    """Integers, so exactly: spans of the rows that end inside groups and with
    them, groups of no row and of nearly all, with every amount of room."""
    g = gen(N)
    G, kept = len(counts), sum(counts)
    offsets = offsets_of(counts)
    edges = offsets.tolist()
    need = sg.sgemm_grouped_act_backward_workspace_bytes(kept + 7, N, G) // 4
    for pad, off in ((0, 0), (3, 1)):
        dC, Z = wide(kept + 7, N, pad, off, g, 4.0), wide(kept + 7, N, pad, off, g)
        dC.round_()
        dC[kept:] = Z[kept:] = float("nan")
        want = dC[:kept].double() * (Z[:kept] > 0)
        sums = torch.stack([want[i:j].sum(0) for i, j in zip(edges, edges[1:])])
        plain = torch.stack([dC[i:j].double().sum(0) for i, j in zip(edges, edges[1:])])
        for room in {need, need // 2, (G + 2) * N, 0}:
            dZ, db = wide(kept + 7, N, pad, off, g, fill=7.0), wide(G, N, pad, off, g, fill=7.0)
            before = dZ.clone()
            grouped_act(dC, Z, "relu", dZ, db, offsets, room, N)
            assert torch.equal(dZ[:kept].double(), want) and torch.equal(db.double(), sums), room
            assert torch.equal(dZ[kept:], before[kept:])
            db.fill_(7.0)
            grouped_act(dC, Z, "relu", None, db, offsets, room, N)       # the sums alone
            assert torch.equal(db.double(), sums), room
            grouped_act(dC, None, "none", None, db, offsets, room, N)
            assert torch.equal(db.double(), plain), room
            over = dC.clone()                                            # in place, without them
            grouped_act(over, Z, "relu", over, None, offsets, room, N)
            assert torch.equal(over[:kept], dZ[:kept])


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N", [([0, 2000, 0, 1, 37], 130), ([3, 0, 9000, 200, 0, 0, 800], 300),
                                      ([1, 0, 40] * 30 + [30000], 5), ([9000] * 3 + [1], 1)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_grouped_sums_are_the_same_whatever_the_room(counts, N, act):
    g = gen(N)
    G, M = len(counts), sum(counts)
    offsets = offsets_of(counts)
    need = sg.sgemm_grouped_act_backward_workspace_bytes(M, N, G) // 4
    dC, Z = wide(M, N, 0, 0, g), wide(M, N, 0, 0, g)
    B, A = torch.empty(G, 0, N, device="cuda"), torch.empty(M, 0, device="cuda")
    db = sg.grouped_linear_backward(dC, A, B, offsets, act, Z)[2]
    for room in (need, need - 1, G * N, 1, 0):
        for dZ in (torch.empty(M, N, device="cuda") if act != "none" else None, None):
            got = torch.full((G, N), 7.0, device="cuda")
            grouped_act(dC, Z, act, dZ, got, offsets, room, N)
            assert torch.equal(got, db), room


@pytest.mark.gpu
def test_sums_of_a_group_with_nearly_all_rows_keep_their_accuracy():
    """A column's 262144 equal values in one of 64 groups: a lane adds at most 64
    of them one after another, a span's lanes and the spans fewer than 32 more, so
    fewer than 128 roundings of at most U of the sum meet."""
    M, N, G = 1 << 18, 256, 64
    counts = [3] * G
    counts[5] = M - 3 * (G - 1)
    dC = torch.full((M, N), 0.1, device="cuda")
    db = torch.empty(G, N, device="cuda")
    room = sg.sgemm_grouped_act_backward_workspace_bytes(M, N, G) // 4
    grouped_act(dC, None, "none", None, db, offsets_of(counts), room, N)
    want = dC[0, 0].double() * torch.tensor(counts, device="cuda", dtype=torch.float64)[:, None]
    assert ((db.double() - want).abs() <= 128 * U * want).all()


@pytest.mark.gpu
def test_the_activation_pass_with_bad_offsets_stays_inside_its_operands():
    g = gen(3)
    M, N = 5000, 24
    dC = torch.randn(M, N, device="cuda", generator=g)
    guard = torch.full((M + 40, N), 7.0, device="cuda")
    sums = torch.full((3 + 40, N), 7.0, device="cuda")
    for off in ([-5, 4, 10, 1 << 30], [0, 4900, 3, 4999], [6000, 7000, 8000, 9000],
                [(1 << 31) - 1, -(1 << 31), (1 << 31) - 1, 0]):
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        need = sg.sgemm_grouped_act_backward_workspace_bytes(M, N, 3) // 4
        for room in (need, 0):
            guard.fill_(7.0)
            sums.fill_(7.0)
            grouped_act(dC, None, "none", guard[20:M + 20], sums[20:23], offsets, room, N)
            for t in (guard, sums):
                assert (t[:20] == 7).all() and (t[-20:] == 7).all()
            if off[0] == -5:
                assert torch.equal(guard[20:M + 20], dC)


@pytest.mark.gpu
def test_moves_past_32_bits():
    g = gen(12)
    T, top, H = 310000, 4, 1000
    ids = torch.randint(-1, 20, (T, top), device="cuda", generator=g)
    offsets, order, place = sg.moe_sort(ids, 20)
    kept = int(offsets[-1])
    X = torch.randn(T, H, device="cuda", generator=g)
    xp = sg.moe_permute(X, place, out=torch.zeros(T * top, H, device="cuda"))
    for s in (slice(0, 5000), slice(kept - 5000, kept)):
        assert torch.equal(xp[s], X[order[s].long() // top])
    assert (xp[kept:] == 0).all()
    w = torch.rand(T, top, device="cuda", generator=g)
    y = sg.moe_unpermute(xp, place, w)
    ws = (w * (place >= 0)).double().sum(1, keepdim=True)
    for s in (slice(0, 5000), slice(T - 5000, T)):
        want = ws[s] * X[s].double()
        assert ((y[s].double() - want).abs() <= (top + 1) * U * want.abs()).all()
    dyp, dw = sg.moe_unpermute_backward(X, xp, place, w, out=xp)
    for s in (slice(0, 5000), slice(kept - 5000, kept)):
        c = order[s].long()
        assert torch.equal(dyp[s], w.reshape(-1)[c][:, None] * X[c // top])
    for s in (slice(0, 5000), slice(T - 5000, T)):
        size = X[s].double().square().sum(1, keepdim=True)
        want = size * (place[s] >= 0)
        assert ((dw[s].double() - want).abs() <= sum_tol(H) * size).all()


@pytest.mark.gpu
def test_a_stack_of_matrices_past_32_bits():
    g = gen(14)
    E, K, N = 300, 1900, 2000
    B = torch.randn(E, K, N, device="cuda", generator=g)     # 4.5 GB
    for per in (1, 40):
        counts = [0] * E
        for e in (0, 1, 150, 298, 299):
            counts[e] = per
        offsets, M = offsets_of(counts), 5 * per
        A, dC = torch.randn(M, K, device="cuda", generator=g), torch.randn(M, N, device="cuda",
                                                                           generator=g)
        C = sg.grouped_linear(A, B, offsets)
        dA, dB, _ = sg.grouped_linear_backward(dC, A, B, offsets)
        for i, e in enumerate((0, 1, 150, 298, 299)):
            s = slice(i * per, (i + 1) * per)
            a, b, d = A[s].double(), B[e].double(), dC[s].double()
            assert ((C[s].double() - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all()
            assert ((dA[s].double() - d @ b.t()).abs() <= 1e-5 * (d.abs() @ b.t().abs())).all()
            assert ((dB[e].double() - a.t() @ d).abs() <= 1e-5 * (a.t().abs() @ d.abs())).all()
        assert (dB[2:150] == 0).all() and (dB[151:298] == 0).all()


@pytest.mark.gpu
def test_bad_offsets_stay_inside_the_operands():
    """Offsets past the rows, negative or falling: clamped, so the rows they
    still describe are right and nothing outside is touched."""
    g = gen(6)
    A, B = torch.randn(20, 16, device="cuda", generator=g), torch.randn(3, 16, 24, device="cuda",
                                                                        generator=g)
    guard = torch.full((60, 24), 7.0, device="cuda")
    for off in ([-5, 4, 10, 1 << 30], [0, 25, 3, 20], [0, 0, 0, 0], [30, 40, 50, 60]):
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        guard.fill_(7.0)
        sg.grouped_linear(A, B, offsets, out=guard[20:40])
        assert (guard[:20] == 7).all() and (guard[40:] == 7).all()
        if off[0] == -5:
            want = torch.cat([A[:4] @ B[0], A[4:10] @ B[1], A[10:] @ B[2]])
            assert torch.allclose(guard[20:40], want, atol=1e-4)
        sg.grouped_linear_backward(torch.randn(20, 24, device="cuda"), A, B, offsets)
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_layer_of_experts_end_to_end():
    """Sort, gather, two products and back, against each token's own experts,
    and every gradient against the definition's."""
    g = gen(8)
    T, top, E, H, F = 150, 2, 6, 72, 100
    x = torch.randn(T, H, device="cuda", generator=g)
    W1 = torch.randn(E, H, F, device="cuda", generator=g) * H ** -0.5
    W2 = torch.randn(E, H, F, device="cuda", generator=g) * F ** -0.5    # out x in
    b1, b2 = torch.randn(E, F, device="cuda", generator=g), torch.randn(E, H, device="cuda",
                                                                        generator=g)
    scores, ids = torch.topk(torch.randn(T, E, device="cuda", generator=g), top)
    w = torch.softmax(scores, 1)
    ids[5] = -1
    ids[9, 1] = E
    dy = torch.randn(T, H, device="cuda", generator=g)
    ws = torch.empty(1 << 22, device="cuda")

    def ours():
        offsets, _, place = sg.moe_sort(ids, E, workspace=ws)
        xp = sg.moe_permute(x, place)
        z = torch.empty(T * top, F, device="cuda")
        h = sg.grouped_linear(xp, W1, offsets, b1, "silu", preact=z, workspace=ws)
        yp = sg.grouped_linear(h, W2, offsets, b2, transpose_b=True, workspace=ws)
        y = sg.moe_unpermute(yp, place, w)
        dyp, dw = sg.moe_unpermute_backward(dy, yp, place, w)
        dh, dW2, db2 = sg.grouped_linear_backward(dyp, h, W2, offsets, transpose_b=True,
                                                  workspace=ws)
        dxp, dW1, db1 = sg.grouped_linear_backward(dh, xp, W1, offsets, "silu", z, workspace=ws)
        return y, sg.moe_unpermute(dxp, place), dw, dW1, db1, dW2, db2

    leaves = [t.double().requires_grad_() for t in (x, w, W1, b1, W2, b2)]
    X, Wt, V1, c1, V2, c2 = leaves
    kept = ((ids >= 0) & (ids < E)).double()
    rows = []
    for j in range(top):
        parts = []
        for e in range(E):
            h = X @ V1[e] + c1[e]
            y = (h * torch.sigmoid(h)) @ V2[e].t() + c2[e]
            parts.append(y * (ids[:, j] == e).double()[:, None])
        rows.append(sum(parts) * (Wt[:, j] * kept[:, j])[:, None])
    want = sum(rows)
    grads = torch.autograd.grad((want * dy.double()).sum(), leaves)
    dX, dWt, dV1, dc1, dV2, dc2 = grads
    got = ours()
    # Two products, two moves and their activations in FP32: a thousand
    # roundings of the output's size bound every one of these sums.
    for name, a, b in zip(("y", "dx", "dw", "dW1", "db1", "dW2", "db2"), got,
                          (want, dX, dWt, dV1, dc1, dV2, dc2)):
        assert ((a.double() - b).abs().max() <= 1000 * U * b.abs().max()), name

    # captured and replayed with other inputs, the same as eager
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ours()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ours()
    for rep in range(4):
        x.normal_(generator=g)
        ids.copy_(torch.randint(-1, E, (T, top), device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        kept_out = [o.clone() for o in out]
        for a, b in zip(kept_out, ours()):
            assert torch.equal(a, b), rep


@pytest.mark.gpu
@pytest.mark.parametrize("own_room", [False, True])
def test_routing_of_many_tokens_replays_from_a_graph(own_room):
    g = gen(16)
    T, top, E, H = 6000, 3, 40, 100       # more choices than one workgroup sorts
    x, w = torch.randn(T, H, device="cuda", generator=g), torch.rand(T, top, device="cuda",
                                                                     generator=g)
    ids = torch.randint(-1, E + 1, (T, top), device="cuda", generator=g)
    ws = torch.empty(1 << 20, device="cuda") if own_room else None
    xp = torch.zeros(T * top, H, device="cuda")

    def step():
        offsets, order, place = sg.moe_sort(ids, E, workspace=ws)
        sg.moe_permute(x, place, out=xp)
        return offsets, order, place, sg.moe_unpermute(xp, place, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        ids.copy_(torch.randint(-1, E + 1, (T, top), device="cuda", generator=g))
        x.normal_(generator=g)
        for o in out:
            o.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, plain_sort(ids.cpu(), E)):
            assert torch.equal(a.cpu(), b), rep
        for a, b in zip(got, step()):
            assert torch.equal(a, b), rep


# Refusals (CPU).

BIG = 1 << 33
FAR = BIG + (1 << 40)


@pytest.fixture(scope="module")
def lib():
    from tiled_fp32_gemm_amd import build
    build.ensure_built()
    return sg.load()


def sort_args(n=16, E=4, ids=BIG, bytes_=4, off=FAR, order=FAR * 2, place=FAR * 3, ws=FAR * 4,
              ws_bytes=1 << 20):
    return n, E, ids, bytes_, off, order, place, 0, ws, ws_bytes


@pytest.mark.parametrize("args", [
    dict(n=-1), dict(E=0), dict(E=-3), dict(bytes_=2), dict(bytes_=0), dict(ids=0),
    dict(ids=BIG + 2), dict(bytes_=8, ids=BIG + 4), dict(off=0), dict(off=FAR + 2),
    dict(order=0), dict(order=FAR + 1), dict(place=0), dict(place=FAR * 3 + 2),
    dict(off=BIG), dict(order=BIG + 32), dict(place=FAR * 2 + 60), dict(order=FAR + 16),
    dict(ws_bytes=-4), dict(n=100000, ws_bytes=64), dict(n=100000, ws=0),
    dict(n=100000, ws=FAR * 4 + 2), dict(n=100000, ws=FAR * 2)])
def test_sort_refuses(lib, args):
    assert sg.sgemm_moe_sort(*sort_args(**args)) == sg.ERR_INVALID_ARG


def test_sort_unsupported_and_workspace(lib):
    assert sg.sgemm_moe_sort(*sort_args(E=1025)) == sg.ERR_UNSUPPORTED
    assert sg.sgemm_moe_sort(*sort_args(n=(1 << 31) - 1023, order=FAR * 20, place=FAR * 40,
                                        ws_bytes=1 << 40)) == sg.ERR_UNSUPPORTED
    f = sg.sgemm_moe_sort_workspace_bytes
    assert f(16, 8) == 0 and f(-1, 8) == 0 and f(100000, 0) == 0 and f(100000, 1025) == 0
    assert f(100000, 8) > 0
    # bounded whatever the number of choices
    assert f((1 << 31) - 1024, 1024) <= 513 * 1024 * 4


MOVE = dict(T=4, top=2, H=8, a=BIG, lda=8, place=FAR, b=FAR * 2, ldb=8)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(top=-1), 1), (dict(H=-1), 1), (dict(lda=7), 1), (dict(ldb=7), 1),
    (dict(a=0), 1), (dict(b=0), 1), (dict(place=0), 1), (dict(a=BIG + 2), 1),
    (dict(b=FAR * 2 + 1), 1), (dict(place=FAR + 3), 1), (dict(b=BIG + 64), 1), (dict(b=FAR), 1),
    (dict(T=1 << 20, top=1 << 12), 2), (dict(H=(1 << 31) - 1023, lda=1 << 31, ldb=1 << 31), 2),
    (dict(lda=1 << 62), 2)])
def test_moves_refuse(lib, change, status):
    m = {**MOVE, **change}
    assert sg.sgemm_moe_permute(m["T"], m["top"], m["H"], m["a"], m["lda"], m["place"], m["b"],
                                m["ldb"], 0) == status
    assert sg.sgemm_moe_unpermute(m["T"], m["top"], m["H"], m["a"], m["lda"], m["place"], 0,
                                  m["b"], m["ldb"], 0) == status


def test_unpermute_backward_refuses(lib):
    f, far = sg.sgemm_moe_unpermute_backward, FAR
    good = [4, 2, 8, BIG, 8, far, 8, far * 2, far * 3, far * 4, 8, far * 5, 0]
    for i, v in ((0, -1), (1, -1), (2, -1), (3, 0), (3, BIG + 2), (4, 7), (5, 0), (6, 7), (7, 0),
                 (8, far * 3 + 2), (9, BIG), (9, far + 32), (9, far * 2), (9, far * 3), (10, 7),
                 (11, BIG), (11, far), (11, far * 2), (11, far * 3), (11, far * 4)):
        bad = list(good)
        bad[i] = v
        assert f(*bad) == sg.ERR_INVALID_ARG, (i, v)
    assert f(4, 2, 8, BIG, 8, 0, 8, far * 2, 0, 0, 8, 0, 0) == sg.OK      # nothing wanted
    assert f(0, 2, 8, 0, 8, 0, 8, 0, 0, 0, 8, 0, 0) == sg.OK


def grouped(tb=0, M=16, N=8, K=4, G=2, off=BIG, A=FAR, lda=4, B=FAR * 2, ldb=8, sb=32, C=FAR * 3,
            ldc=8, ws=0, ws_bytes=0, **ep):
    e = None
    if ep:
        e = sg.Epilogue()
        for k, v in ep.items():
            setattr(e, k, v)
    return sg.sgemm_grouped(tb, M, N, K, G, off, A, lda, B, ldb, sb, C, ldc, e, 0, ws, ws_bytes)


@pytest.mark.parametrize("args,status", [
    (dict(tb=2), 1), (dict(M=-1), 1), (dict(G=-1), 1), (dict(G=1025), 2), (dict(off=0), 1),
    (dict(off=BIG + 2), 1), (dict(A=0), 1), (dict(lda=3), 1), (dict(ldb=7), 1), (dict(sb=31), 1),
    (dict(tb=1, ldb=3), 1), (dict(ldc=7), 1), (dict(C=FAR), 1), (dict(C=FAR * 2 + 200), 1),
    (dict(C=BIG), 1), (dict(bias=FAR * 4, ldbias=7), 1), (dict(bias=FAR * 3, ldbias=8), 1),
    (dict(preact=FAR * 3, ldp=8), 1), (dict(residual=FAR * 3 + 4, ldr=8), 1),
    (dict(sb=1 << 62), 2), (dict(ws=0, ws_bytes=8), 1), (dict(M=0, A=0, C=0), 0),
    (dict(N=0, B=0, C=0), 0), (dict(G=0, off=0, B=0), 0)])
def test_grouped_refuses(lib, args, status):
    assert grouped(**args) == status


def test_grouped_gradients_refuse(lib):
    f = sg.sgemm_grouped_wgrad
    good = [0, 16, 8, 4, 2, BIG, FAR, 4, FAR * 2, 8, FAR * 3, 8, 32, 0, 0, 0]
    for i, v in ((0, 2), (1, -1), (2, -1), (3, -1), (4, -1), (5, 0), (5, BIG + 2), (6, 0), (7, 3),
                 (8, 0), (9, 7), (10, 0), (10, FAR), (10, FAR * 2), (10, BIG), (11, 7), (12, 31),
                 (14, 2), (15, -4), (15, 64)):
        bad = list(good)
        bad[i] = v
        assert f(*bad) == sg.ERR_INVALID_ARG, (i, v)
    f = sg.sgemm_grouped_act_backward
    good = [16, 8, 2, BIG, FAR, 8, FAR * 2, 8, 1, FAR * 3, 8, FAR * 4, 8, 0, 0, 0]
    for i, v in ((0, -1), (1, -1), (2, -1), (3, 0), (4, 0), (5, 7), (6, 0), (7, 7), (8, 9),
                 (9, FAR + 16), (9, BIG), (10, 7), (11, FAR), (11, BIG), (12, 7), (15, -4)):
        bad = list(good)
        bad[i] = v
        assert f(*bad) == sg.ERR_INVALID_ARG, (i, v)


@pytest.mark.gpu
def test_the_binding_refuses_bad_tensors():
    f = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    i32 = torch.int32
    A, B, off = f(6, 4), f(2, 4, 8), f(3, dtype=i32)
    place, X = f(3, 2, dtype=i32), f(3, 5)
    for call in (lambda: sg.moe_sort(f(3, 2), 4), lambda: sg.moe_sort(f(3, 2, dtype=i32), 0),
                 lambda: sg.moe_sort(f(3, 2, dtype=i32).t(), 4),
                 lambda: sg.moe_sort(torch.zeros(3, dtype=i32), 4),
                 lambda: sg.moe_permute(f(4, 5), place), lambda: sg.moe_permute(X, place.long()),
                 lambda: sg.moe_permute(X, place, out=f(5, 5)),
                 lambda: sg.moe_unpermute(f(5, 5), place),
                 lambda: sg.moe_unpermute(f(6, 5), place, f(3, 3)),
                 lambda: sg.moe_unpermute(f(6, 5), place, f(2, 3).t()),
                 lambda: sg.moe_unpermute_backward(f(3, 4), f(6, 5), place),
                 lambda: sg.grouped_linear(A, B, f(2, dtype=i32)),
                 lambda: sg.grouped_linear(A, B, off.long()),
                 lambda: sg.grouped_linear(A, B[0], off),
                 lambda: sg.grouped_linear(A, f(2, 5, 8), off),
                 lambda: sg.grouped_linear(A, B, off, f(8)),
                 lambda: sg.grouped_linear(A, B, off, residual=f(6, 7)),
                 lambda: sg.grouped_linear_backward(f(6, 7), A, B, off),
                 lambda: sg.grouped_linear_backward(f(6, 8), A, B, off, "gelu")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sg.SgemmError):
        sg.moe_sort(f(30000, dtype=i32), 4, workspace=f(1))
