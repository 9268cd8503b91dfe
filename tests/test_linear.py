"""Products with an epilogue and their gradients, against the definition in 64
bits.

Tolerances, from FP32 arithmetic (u = 2^-24, half a step):
  Z   any order of summing K products and a bias: (K + 3) u (|A|·|B| + |bias|),
      and never more than the library's 1e-5 of the same.
  C   |act'| <= 1.13 carries Z's error over; the activation itself is z times a
      factor of at most 1 made in fewer than 32 roundings, the residual's sum
      one rounding more.
  dZ  act' is made in fewer than 64 roundings of values of at most 1.13.
  sums and products of dZ   as for Z, over |dZ|, with dZ's error carried over.
"""
from __future__ import annotations

import itertools

import pytest

import tiled_fp32_gemm_amd as sg

torch = pytest.importorskip("torch")
U = 2.0 ** -24
ACTS = sorted(sg.ACTIVATIONS)


def act64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / 2 ** 0.5)
    if name == "silu":
        return z * torch.sigmoid(z)
    return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))


def slope64(name, z):
    z = z.clone().requires_grad_()
    with torch.enable_grad():
        act64(name, z).sum().backward()
    return z.grad if name != "relu" else (z > 0).double()


def sum_tol(K):
    return min(1e-5, (K + 3) * U)


def wide(rows, cols, pad=0, off=0, gen=None, scale=1.0, fill=float("nan")):
    """rows x cols normals inside a buffer of `fill`: `pad` more columns, the
    first element `off` floats from an aligned address."""
    buf = torch.full((off + rows * (cols + pad) + 8,), fill, device="cuda")
    view = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(scale * torch.randn(rows, cols, device="cuda", generator=gen))
    return view


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def run_case(M, N, K, ta=False, tb=False, act="none", bias=True, residual=True, preact=True,
             pad=0, off=0, ws_bytes=0, seed=1, in_place=False):
    g = gen(seed)
    A = wide(*((K, M) if ta else (M, K)), pad, off, g)
    B = wide(*((N, K) if tb else (K, N)), pad, off, g, max(K, 1) ** -0.5)
    b = torch.randn(N, device="cuda", generator=g) if bias else None
    C = wide(M, N, pad, off, g, fill=7.0)
    R = (C if in_place else wide(M, N, pad, off, g)) if residual else None
    R0 = R.clone() if residual else None
    Z = wide(M, N, pad, off, g, fill=7.0) if preact else None
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
    out = sg.linear(A, B, b, act, R, transpose_a=ta, transpose_b=tb, out=C, preact=Z,
                    workspace=ws)
    assert out is C
    torch.cuda.synchronize()
    a64, b64 = (A.t() if ta else A).double(), (B.t() if tb else B).double()
    z = a64 @ b64
    T = a64.abs() @ b64.abs()
    if bias:
        z, T = z + b.double(), T + b.double().abs()
    ztol = sum_tol(K) * T
    if preact:
        assert ((Z.double() - z).abs() <= ztol).all(), "preact"
    y = act64(act, z)
    tol = 1.13 * ztol + 32 * U * z.abs()
    if residual:
        y = y + R0.double()
        tol = tol + U * y.abs() + U * tol
    err = (C.double() - y).abs()
    assert (err <= tol).all(), f"C: {err.max().item()} at {(err - tol).argmax().item()}"
    for t in (C, Z):   # nothing beside the matrix is written
        if t is not None and pad and M > 1:
            base = t.as_strided((M - 1, pad), (t.stride(0), 1), t.storage_offset() + N)
            assert (base == 7.0).all()
    return C


SHAPES = [(1, 1, 1), (1, 7, 5), (3, 1, 33), (5, 9, 0), (1, 130, 300), (1, 512, 2048),
          (2, 63, 64), (4, 100, 31), (7, 257, 515), (8, 64, 128), (9, 1000, 70), (16, 48, 1000),
          (17, 33, 65), (31, 65, 129), (33, 64, 32), (64, 64, 64), (65, 129, 97),
          (100, 300, 200), (257, 130, 40), (300, 260, 190), (128, 512, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
def test_linear_shapes(M, N, K, ta, tb):
    run_case(M, N, K, ta, tb, "gelu", pad=0)
    run_case(M, N, K, ta, tb, "silu", pad=3, off=1, ws_bytes=1 << 22)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 300, 100), (40, 72, 50), (130, 200, 64)])
def test_linear_epilogues(act, M, N, K):
    for bias, residual, preact in itertools.product((False, True), repeat=3):
        run_case(M, N, K, act=act, bias=bias, residual=residual, preact=preact)
        run_case(M, N, K, tb=True, act=act, bias=bias, residual=residual, preact=preact, pad=1)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 200, 64), (6, 64, 128), (70, 90, 30), (256, 256, 256)])
def test_linear_residual_in_place(M, N, K):
    for pad in (0, 5):
        run_case(M, N, K, act="relu", in_place=True, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 16384), (64, 64, 16384), (130, 70, 5001),
                                   (256, 256, 8192), (20, 36, 4097), (33, 65, 65537)])
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False)])
def test_linear_long_k_with_and_without_workspace(M, N, K, ta, tb):
    need = sg.sgemm_linear_workspace_bytes(ta, tb, M, N, K)
    for ws in {0, need, need // 2 // 4 * 4, 1 << 26}:
        run_case(M, N, K, ta, tb, "gelu_tanh", ws_bytes=ws)


@pytest.mark.gpu
def test_linear_integers_are_exact():
    g = gen(3)
    for M, N, K in [(1, 100, 64), (5, 33, 100), (70, 80, 90), (300, 200, 64), (1000, 1500, 777)]:
        A = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float()
        B = torch.randint(-8, 9, (K, N), generator=g, device="cuda").float()
        b = torch.randint(-8, 9, (N,), generator=g, device="cuda").float()
        R = torch.randint(-8, 9, (M, N), generator=g, device="cuda").float()
        ws = torch.empty(1 << 24, device="cuda")
        want = ((A.double() @ B.double() + b).clamp(min=0) + R).float()
        assert torch.equal(sg.linear(A, B, b, "relu", R, workspace=ws), want)
        At, Bt = A.t().contiguous(), B.t().contiguous()
        assert torch.equal(sg.linear(A, Bt, b, "relu", R, transpose_b=True), want)
        assert torch.equal(sg.linear(At, B, b, "relu", R, transpose_a=True), want)
        assert torch.equal(sg.linear(At, Bt, b, "relu", R, transpose_a=True, transpose_b=True),
                           want)


# A shape of odd sizes for every tile, whatever the layouts.
TILES = [("256x256x32", 7461, 3931, 45), ("128x128x32", 7208, 389, 47),
         ("64x128x32", 513, 6694, 49), ("64x128x32_ks2", 8553, 69, 47),
         ("64x64x32", 8663, 16, 45), ("32x64x32_ks2", 9098, 69, 47),
         ("32x64x64_ks4", 33, 16, 163), ("32x64x32_ks2_s4", 35, 17, 45)]


@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("tile,M,N,K", TILES)
def test_shapes_of_every_tile(lib, tile, M, N, K, ta, tb):
    kernel = sg.sgemm_linear_plan_query(ta, tb, M, N, K)[1].kernel.decode()
    assert kernel == f"product_{'sf'[not ta]}{'sf'[tb]}_{tile}"


@pytest.mark.gpu
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("tile,M,N,K", TILES)
def test_linear_every_tile(tile, M, N, K, ta, tb):
    run_case(M, N, K, ta, tb, "gelu", pad=3, off=1)
    run_case(M, N, K, ta, tb, "none", bias=False, residual=False, preact=False)


# Both kernels for a few rows, every width of theirs, short and long K.
ROWS = [(True, 37, 300, "fast_%dx4"), (True, 37, 2051, "fast_%dx4"), (True, 61, 5000, "fast_%dx4"),
        (True, 4100, 301, "fast_%dx16"), (True, 4100, 2051, "fast_%dx16"),
        (False, 243, 301, "slow_%dx16"), (False, 5203, 130, "slow_%dx32"),
        (False, 10501, 99, "slow_%dx64"), (False, 33001, 77, "slow_%dx64")]


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("tb,N,K,kernel", ROWS)
def test_shapes_of_the_rows_kernels(lib, tb, N, K, kernel, M):
    plan = sg.sgemm_linear_plan_query(0, tb, M, N, K)[1]
    assert plan.kernel.decode() == "rows_" + kernel % {3: 4, 5: 8}.get(M, M)
    assert plan.threads == (512 if not tb and N < 32768 else 256)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("tb,N,K,kernel", ROWS)
def test_linear_by_rows(tb, N, K, kernel, M):
    run_case(M, N, K, tb=tb, act="silu", pad=3, off=1)
    run_case(M, N, K, tb=tb, act="none", bias=False, residual=False, preact=False)


# Cut in two launches: by rows (one, a few by the vector kernels, many), by columns.
CUTS = [(2049, 4096, 1000), (2053, 4096, 1024), (2100, 4096, 4001), (2048, 4104, 1024),
        (4096, 4097, 1000), (4200, 4096, 1500)]


@pytest.mark.gpu
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("M,N,K", CUTS)
def test_linear_in_two_launches(M, N, K, ta, tb):
    assert "+" in sg.sgemm_linear_plan_query(ta, tb, M, N, K, 1 << 26)[1].kernel.decode()
    run_case(M, N, K, ta, tb, "silu", ws_bytes=1 << 26, in_place=True)
    run_case(M, N, K, ta, tb, "gelu", pad=3, off=1)


@pytest.mark.gpu
def test_linear_in_two_launches_is_exact_and_replays():
    g = gen(8)
    M, N, K = 4700, 4096, 4096   # the second launch splits K
    A = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float()
    B = torch.randint(-8, 9, (K, N), generator=g, device="cuda").float()
    b = torch.randint(-8, 9, (N,), generator=g, device="cuda").float()
    need = sg.sgemm_linear_workspace_bytes(0, 0, M, N, K)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = (A.double() @ B.double() + b).clamp(min=0).float()
    assert torch.equal(sg.linear(A, B, b, "relu", workspace=ws), want)
    assert torch.equal(sg.linear(A, B, b, "relu"), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sg.linear(A, B, b, "relu", workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_activations_at_the_extremes():
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 0.5, -0.5, 4.0, -4.0, 9.0, -9.0,
                      13.0, -13.0, 40.0, -40.0, 88.0, -88.0, 120.0, -120.0, 1e20, -1e20, 3e38,
                      -3e38, inf, -inf, nan], device="cuda")
    A, B = torch.zeros(1, 4, device="cuda"), torch.zeros(4, x.numel(), device="cuda")
    for act in ACTS:
        y = sg.linear(A, B, x, act)[0]
        dz, _ = sg.activation_backward(torch.ones(1, x.numel(), device="cuda"), act, x[None],
                                       out=torch.empty(1, x.numel(), device="cuda"))
        z = x[:24].double()
        want, slope = act64(act, z), slope64(act, z)
        slope = torch.where(slope.isnan(), (z > 0).double(), slope)   # 0 * inf in the formula
        assert ((y[:24].double() - want).abs() <= 32 * U * z.abs() + 1e-37).all(), act
        assert ((dz[0, :24].double() - slope).abs() <= 64 * U).all(), act
        limits = [inf, -inf if act == "none" else 0.0]
        assert y[24:26].tolist() == limits, (act, y[24:26])
        assert dz[0, 24:26].tolist() == [1.0, 1.0 if act == "none" else 0.0], act
        assert y[26].isnan() and (act == "none" or dz[0, 26].isnan())
        # The lower tail keeps its relative accuracy: the exponential's argument
        # is off by fewer than 8 roundings, the fit of the normal distribution
        # function by 1.2e-7 of values above 0.03, the rest is 64 roundings.
        t = torch.linspace(-12, -1, 500, device="cuda")
        y = sg.linear(A, torch.zeros(4, 500, device="cuda"), t, act)[0].double()
        t = t.double()
        want = act64(act, t)
        arg = torch.maximum(t * t / 2, 1.6 * t.abs() * (1 + 0.044715 * t * t))
        assert ((y - want).abs() <= (128 + 8 * arg) * U * want.abs() + 1e-37).all(), act


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (3, 5), (100, 64), (33, 257), (2000, 130),
                                 (0, 40), (5000, 3)])
def test_activation_backward(act, M, N):
    g = gen(5)
    for pad, ws_bytes in ((0, 0), (2, 1 << 20), (0, 5 * N * 4)):
        dC, Z = wide(M, N, pad, pad, g), wide(M, N, pad, pad, g, 2.0)
        out = wide(M, N, pad, pad, g, fill=7.0)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
        dz, db = sg.activation_backward(dC, act, Z, out=out, workspace=ws)
        want = dC.double() * slope64(act, Z.double())
        tol = 64 * U * dC.double().abs()
        assert ((dz.double() - want).abs() <= tol).all()
        btol = sum_tol(M) * want.abs().sum(0) + tol.sum(0)
        assert ((db.double() - want.sum(0)).abs() <= btol).all()
        # in place over dC, over preact, and the sums alone
        c, z = dC.clone(), Z.clone()
        assert torch.equal(sg.activation_backward(c, act, Z, out=c, workspace=ws)[0], dz)
        assert torch.equal(sg.activation_backward(dC, act, z, out=z, workspace=ws)[0], dz)
        only = torch.empty(N, device="cuda")
        assert sg.sgemm_act_backward(M, N, dC.data_ptr(), N + pad, Z.data_ptr(), N + pad,
                                     sg.ACTIVATIONS[act], 0, 1, only.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream,
                                     ws.data_ptr() if ws_bytes else 0, ws_bytes) == sg.OK
        assert torch.equal(only, db)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1 << 18, 256), (1 << 19, 3), (300000, 130), (40000, 1030)])
def test_sums_of_tall_matrices_keep_their_accuracy_without_room(M, N):
    """Equal values of one sign: a lane adds at most 256 of them one after another
    (and at most 16 such runs), a span's lanes at most 256, the spans at most 1024
    / 64 and 6 halvings, so fewer than 600 roundings of at most U of the sum meet."""
    dC = torch.full((M, N), 0.1, device="cuda")
    want = float(dC[0, 0]) * M
    stream = torch.cuda.current_stream().cuda_stream
    need = sg.sgemm_act_backward_workspace_bytes(M, N)
    assert need > 0
    sums = []
    for room in (0, 16, need - 4, need):
        ws = torch.full((need // 4,), float("nan"), device="cuda")
        db = torch.empty(N, device="cuda")
        assert sg.sgemm_act_backward(M, N, dC.data_ptr(), N, 0, 1, 0, 0, 1, db.data_ptr(), stream,
                                     ws.data_ptr() if room else 0, room) == sg.OK
        assert ((db.double() - want).abs() <= 600 * U * want).all(), room
        sums.append(db)
    sums.append(sg.activation_backward(dC)[1])
    for db in sums[1:]:      # the same whatever the room
        assert torch.equal(db, sums[0])


@pytest.mark.gpu
def test_gradients_without_a_workspace_replay_from_a_graph():
    g = gen(21)
    M, N, K = 9000, 130, 40
    A, B, Z = (torch.randn(*s, device="cuda", generator=g) for s in ((M, K), (K, N), (M, N)))
    dC = torch.randn(M, N, device="cuda", generator=g)
    sums = torch.empty(N, device="cuda")

    def step():
        assert sg.sgemm_act_backward(M, N, dC.data_ptr(), N, Z.data_ptr(), N, 4, 0, 1,
                                     sums.data_ptr(), torch.cuda.current_stream().cuda_stream,
                                     0, 0) == sg.OK
        return (*sg.linear_backward(dC, A, B, "silu", Z), sums)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        for t in (A, B, Z, dC):
            t.normal_(generator=g)
        for o in out:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), rep
        assert torch.equal(got[2], got[3])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(70, 5), (1000, 17), (5000, 300), (20001, 1), (9000, 1500)])
def test_the_activation_pass_is_the_same_whatever_the_room(act, M, N):
    g = gen(M)
    for pad in (0, 3):
        dC, Z = wide(M, N, pad, pad, g), wide(M, N, pad, pad, g, 2.0)
        z = None if act == "none" else Z
        need = sg.sgemm_act_backward_workspace_bytes(M, N)
        room = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        dz, db = sg.activation_backward(dC, act, z, out=wide(M, N, pad, pad, g))
        for ws in (room(4), room(max(need - 4, 4)), room(max(need, 4)), room(need + 400)):
            for out in (wide(M, N, pad, pad, g), dC.clone(), Z.clone()):
                src = out if torch.equal(out, dC) else dC
                pre = z if z is None or not torch.equal(out, Z) else out
                got = sg.activation_backward(src, act, pre, out=out, workspace=ws)
                assert torch.equal(got[0], dz) and torch.equal(got[1], db)
            A, B = torch.empty(M, 0, device="cuda"), torch.empty(0, N, device="cuda")
            assert torch.equal(sg.linear_backward(dC, A, B, act, z, workspace=ws)[2], db)
        assert torch.equal(sg.linear_backward(dC, A, B, act, z)[2], db)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 30, 50), (5, 64, 40), (130, 70, 200), (257, 100, 64),
                                   (2000, 24, 36), (0, 20, 30)])
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
def test_linear_backward(M, N, K, ta, tb):
    g = gen(7)
    for act, pad in (("gelu", 0), ("none", 3), ("silu", 1)):
        A = wide(*((K, M) if ta else (M, K)), pad, 0, g)
        B = wide(*((N, K) if tb else (K, N)), pad, 0, g)
        Z, dC = wide(M, N, pad, 0, g), wide(M, N, pad, 0, g)
        ws = torch.empty(1 << 20, device="cuda")
        dA, dB, db = sg.linear_backward(dC, A, B, act, None if act == "none" else Z,
                                        transpose_a=ta, transpose_b=tb, workspace=ws)
        assert dA.shape == A.shape and dB.shape == B.shape
        a, b = (A.t() if ta else A).double(), (B.t() if tb else B).double()
        dz = dC.double() * slope64(act, Z.double())
        dtol = 64 * U * dC.double().abs()
        got_a, got_b = (dA.t() if ta else dA).double(), (dB.t() if tb else dB).double()
        assert ((got_a - dz @ b.t()).abs()
                <= sum_tol(N) * (dz.abs() @ b.abs().t()) + dtol @ b.abs().t()).all()
        assert ((got_b - a.t() @ dz).abs()
                <= sum_tol(M) * (a.abs().t() @ dz.abs()) + a.abs().t() @ dtol).all()
        assert ((db.double() - dz.sum(0)).abs() <= sum_tol(M) * dz.abs().sum(0) + dtol.sum(0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(act):
    """The loss sum(C * W) moved along a direction: the 64-bit forward's central
    difference (step 1e-5, whose own error is below 1e-8 of the terms' size)
    against the gradients."""
    g = gen(9)
    M, N, K = 37, 50, 41
    A, B = torch.randn(M, K, device="cuda", generator=g), torch.randn(K, N, device="cuda",
                                                                      generator=g)
    b, W = torch.randn(N, device="cuda", generator=g), torch.randn(M, N, device="cuda",
                                                                   generator=g)
    Z = torch.empty(M, N, device="cuda")
    sg.linear(A, B, b, act, preact=Z)
    dA, dB, db = sg.linear_backward(W, A, B, act, Z)

    def loss(a, bb, c):
        return (act64(act, a @ bb + c) * W.double()).sum()

    base = [A.double(), B.double(), b.double()]
    for i, d in enumerate((dA, dB, db)):
        v = torch.randn(d.shape, device="cuda", generator=g).double()
        h, up, dn = 1e-5, list(base), list(base)
        up[i], dn[i] = base[i] + h * v, base[i] - h * v
        num = ((loss(*up) - loss(*dn)) / (2 * h)).item()
        terms = (d.double() * v).abs().sum().item()
        assert abs((d.double() * v).sum().item() - num) <= 1e-5 * terms + 1e-6 * terms


@pytest.mark.gpu
def test_linear_runs_on_the_given_stream_and_is_the_same_every_time():
    g = gen(11)
    A, B = torch.randn(200, 3000, device="cuda", generator=g), torch.randn(3000, 150,
                                                                           device="cuda",
                                                                           generator=g)
    ws = torch.empty(1 << 22, device="cuda")
    want = sg.linear(A, B, None, "silu", workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sg.linear(A, B, None, "silu", stream=s, workspace=ws)
    grads = sg.linear_backward(got, A, B, "none", stream=s, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    for x, y in zip(grads, sg.linear_backward(want, A, B, "none", workspace=ws)):
        assert torch.equal(x, y)
    for _ in range(3):
        assert torch.equal(sg.linear(A, B, None, "silu", workspace=ws), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (256, 256, 4096), (100, 70, 33)])
def test_linear_and_its_gradients_replay_from_a_graph(M, N, K):
    g = gen(13)
    A, B = torch.randn(M, K, device="cuda", generator=g), torch.randn(K, N, device="cuda",
                                                                      generator=g)
    b, dC = torch.randn(N, device="cuda", generator=g), torch.randn(M, N, device="cuda",
                                                                    generator=g)
    Z, ws = torch.empty(M, N, device="cuda"), torch.empty(1 << 22, device="cuda")

    def step():
        y = sg.linear(A, B, b, "gelu", preact=Z, workspace=ws)
        return (y, Z, *sg.linear_backward(dC, A, B, "gelu", Z, workspace=ws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        A.normal_(generator=g)
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for x, y in zip(got, step()):
            assert torch.equal(x, y), rep


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Operands of more than 4 GiB, checked on rows from both ends."""
    g = gen(17)
    M, N, K = (1 << 20) + 3, 1100, 20
    A = torch.randn(M, K, device="cuda", generator=g)
    B = torch.randn(K, N, device="cuda", generator=g)
    b = torch.randn(N, device="cuda", generator=g)
    R, Z = torch.randn(M, N, device="cuda", generator=g), torch.empty(M, N, device="cuda")
    rows = torch.tensor([0, 1, M // 2, M - 130, M - 2, M - 1], device="cuda")
    C = sg.linear(A, B, b, "relu", R, preact=Z)
    z = A[rows].double() @ B.double() + b.double()
    tol = sum_tol(K) * (A[rows].double().abs() @ B.double().abs() + b.double().abs())
    assert ((Z[rows].double() - z).abs() <= tol).all()
    y = z.clamp(min=0) + R[rows].double()
    assert ((C[rows].double() - y).abs() <= tol + 2 * U * y.abs()).all()
    # the sums over all its rows, K slow in both operands
    ws = torch.empty(1 << 24, device="cuda")
    dz, db = sg.activation_backward(R, "relu", Z, out=C, workspace=ws)
    assert torch.equal(dz[rows], torch.where(Z[rows] > 0, R[rows], 0.0))
    dB = sg.linear(A, dz, transpose_a=True, workspace=ws)
    # The same in 64 bits by parts, with the bounds of their sizes: 1e-5 as M is long.
    want = torch.zeros(K, N, dtype=torch.float64, device="cuda")
    size, sums, ssize = want.clone(), want[0].clone(), want[0].clone()
    for i in range(0, M, 1 << 17):
        a, d = A[i:i + (1 << 17)].double(), dz[i:i + (1 << 17)].double()
        want += a.t() @ d
        size += a.abs().t() @ d.abs()
        sums += d.sum(0)
        ssize += d.abs().sum(0)
    assert ((dB.double() - want).abs() <= 1e-5 * size).all()
    assert ((db.double() - sums).abs() <= 1e-5 * ssize).all()
    # rows of a long k
    T = dz.view(-1)[:(1 << 29) + 4].view(2, -1)[:, :(1 << 28) + 1]
    W = torch.randn(3, T.shape[1], device="cuda", generator=g)
    got = sg.linear(T, W, transpose_b=True, workspace=ws)
    for j in range(3):
        terms = T.double() * W[j].double()
        assert ((got[:, j].double() - terms.sum(1)).abs() <= 1e-5 * terms.abs().sum(1)).all()


@pytest.mark.gpu
def test_a_single_row_has_no_leading_dimension():
    g = gen(23)
    far, s = 1 << 40, torch.cuda.current_stream().cuda_stream
    for M, N, K, lda, ldb, ldc in ((1, 70, 90, far, 70, far), (50, 70, 1, 1, far, 70),
                                   (300, 200, 1, 1, far, 200)):
        A, B = torch.randn(M, K, device="cuda", generator=g), torch.randn(K, N, device="cuda",
                                                                          generator=g)
        C = torch.empty(M, N, device="cuda")
        assert sg.sgemm_linear(0, 0, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, C.data_ptr(),
                               ldc, None, s) == sg.OK
        a, b = A.double(), B.double()
        assert ((C.double() - a @ b).abs() <= sum_tol(K) * (a.abs() @ b.abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K", [(3, 37, 70), (40, 37, 70), (70, 131, 64)])
def test_every_alignment(off, M, N, K):
    for pad in range(4):
        run_case(M, N, K, act="silu", pad=pad, off=off)
        run_case(M, N, K, tb=True, act="silu", pad=pad, off=off)


@pytest.mark.gpu
def test_non_finite_values_stay_in_their_rows_and_columns():
    g = gen(19)
    for M, N, K in ((5, 70, 100), (100, 130, 77), (300, 300, 64)):
        A, B = torch.randn(M, K, device="cuda", generator=g), torch.randn(K, N, device="cuda",
                                                                          generator=g)
        clean = sg.linear(A, B)
        A[M // 2, K - 1], B[0, N // 3] = float("nan"), float("inf")
        for a, b, ta, tb in ((A, B, 0, 0), (A, B.t().contiguous(), 0, 1),
                             (A.t().contiguous(), B, 1, 0)):
            C = sg.linear(a, b, transpose_a=ta, transpose_b=tb)
            assert C[M // 2].isnan().all() and not C[:, N // 3].isfinite().any()
            keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
            keep[M // 2], keep[:, N // 3] = False, False
            tol = 2 * sum_tol(K) * (A.nan_to_num(0).abs() @ B.nan_to_num(0, 0, 0).abs())
            assert ((C - clean).abs()[keep] <= tol[keep]).all()


@pytest.mark.gpu
def test_two_graphs_share_a_workspace_and_two_streams_have_their_own():
    g = gen(29)
    shapes = [(256, 256, 4096), (64, 300, 8000)]
    ins = [(torch.randn(M, K, device="cuda", generator=g),
            torch.randn(K, N, device="cuda", generator=g)) for M, N, K in shapes]
    shared = torch.empty(1 << 22, device="cuda")
    for (A, B), (M, N, K) in zip(ins, shapes):
        assert sg.sgemm_linear_plan_query(0, 0, M, N, K, 1 << 24)[1].splits > 1
    want = [sg.linear(A, B, None, "gelu", workspace=shared) for A, B in ins]
    graphs, outs = [], []
    for A, B in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(sg.linear(A, B, None, "gelu", workspace=shared))
    for rep in range(4):
        for o in outs:
            o.fill_(float("nan"))
        for i in ((0, 1), (1, 0))[rep % 2]:
            graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
    streams = [torch.cuda.Stream() for _ in ins]
    rooms = [torch.empty(1 << 22, device="cuda") for _ in ins]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for (A, B), s, ws in zip(ins, streams, rooms):
            got.append(sg.linear(A, B, None, "gelu", stream=s, workspace=ws))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


# Plans (CPU).

@pytest.fixture(scope="module")
def lib():
    from tiled_fp32_gemm_amd import build
    build.ensure_built()
    return sg.load()


@pytest.mark.parametrize("ta,tb,M,N,K,kernel", [
    (0, 0, 4096, 4096, 4096, "product_fs_256x256x32"),
    (0, 1, 4096, 4096, 4096, "product_ff_256x256x32"),
    (1, 0, 4096, 4096, 4096, "product_ss_256x256x32"),
    (1, 1, 8192, 8192, 8192, "product_sf_256x256x32"),
    (0, 0, 1000, 1500, 777, "product_fs_32x64x32_ks2"),
    (0, 0, 65536, 128, 256, "product_fs_128x128x32"),
    (0, 1, 1, 4096, 4096, "rows_fast_1x16"), (0, 1, 1, 1024, 4096, "rows_fast_1x4"),
    (0, 1, 12, 4096, 4096, "rows_fast_8x16"), (0, 0, 5, 4096, 4096, "rows_slow_8x16"),
    (0, 0, 2, 32768, 1024, "rows_slow_2x64"), (0, 0, 9, 4096, 4096, "rows_slow_8x32"),
    (0, 0, 17, 4096, 4096, "product_fs_32x64x64_ks4"),
    (1, 0, 1, 4096, 4096, "product_ss_32x64x64_ks4")])
def test_plans_without_workspace(lib, ta, tb, M, N, K, kernel):
    st, plan = sg.sgemm_linear_plan_query(ta, tb, M, N, K)
    assert st == sg.OK and plan.kernel.decode() == kernel
    assert plan.splits == 1 and plan.workspace_bytes == 0 and plan.workgroups > 0


def test_split_plans_fit_their_workspace(lib):
    for ta, tb in itertools.product((0, 1), repeat=2):
        for M, N, K in ((256, 256, 8192), (64, 64, 65536), (512, 512, 2048), (256, 128, 65536)):
            need = sg.sgemm_linear_workspace_bytes(ta, tb, M, N, K)
            st, plan = sg.sgemm_linear_plan_query(ta, tb, M, N, K, need)
            assert st == sg.OK and plan.splits > 1
            assert plan.workspace_bytes == need == plan.splits * M * N * 4
            assert sg.sgemm_linear_plan_query(ta, tb, M, N, K, 1 << 40)[1].as_dict() \
                == plan.as_dict()
            less = sg.sgemm_linear_plan_query(ta, tb, M, N, K, need - 4)[1]
            assert less.workspace_bytes <= need - 4
            assert sg.sgemm_linear_plan_query(ta, tb, M, N, K)[1].splits == 1
    for args in ((0, 0, 4096, 4096, 4096), (0, 1, 1, 4096, 4096), (0, 0, 256, 256, 0)):
        assert sg.sgemm_linear_workspace_bytes(*args) == 0


@pytest.mark.parametrize("ta,tb,M,N,K,kernel", [
    (0, 0, 4097, 4096, 4096, "product_fs_256x256x32+1rows"),
    (0, 1, 8200, 4096, 4096, "product_ff_256x256x32+8rows"),
    (1, 0, 2100, 4096, 4096, "product_ss_128x128x32+52rows"),
    (0, 0, 4096, 4200, 4096, "product_fs_256x256x32+104cols"),
    (0, 0, 4096, 4096, 4096, "product_fs_256x256x32"),
    (0, 0, 5000, 4096, 4096, "product_fs_128x128x32"),
    (0, 0, 1000, 1500, 777, "product_fs_32x64x32_ks2")])
def test_plans_in_two_launches(lib, ta, tb, M, N, K, kernel):
    assert sg.sgemm_linear_plan_query(ta, tb, M, N, K)[1].kernel.decode() == kernel


def test_two_launches_fit_their_workspace(lib):
    for ta, tb in itertools.product((0, 1), repeat=2):
        for M, N, K in ((4700, 4096, 4096), (4096, 4700, 4096), (4097, 4096, 4096),
                        (2100, 4096, 4096), (9000, 2048, 4096)):
            need = sg.sgemm_linear_workspace_bytes(ta, tb, M, N, K)
            st, plan = sg.sgemm_linear_plan_query(ta, tb, M, N, K, need)
            assert st == sg.OK and plan.workspace_bytes == need
            assert sg.sgemm_linear_plan_query(ta, tb, M, N, K, 1 << 40)[1].as_dict() \
                == plan.as_dict()
            if need:
                less = sg.sgemm_linear_plan_query(ta, tb, M, N, K, need - 4)[1]
                assert less.workspace_bytes <= need - 4


def test_plan_query_refuses(lib):
    for args in ((2, 0, 4, 4, 4), (0, 0, -1, 4, 4), (0, 0, 4, 4, 4, -1)):
        assert sg.sgemm_linear_plan_query(*args)[0] == sg.ERR_INVALID_ARG
    assert sg.sgemm_linear_plan_query(0, 0, (1 << 31) - 1023, 4, 4)[0] == sg.ERR_UNSUPPORTED
    assert lib.sgemm_linear_plan_query(0, 0, 4, 4, 4, 0, None) == sg.ERR_INVALID_ARG
    assert sg.sgemm_linear_plan_query(0, 0, 0, 4, 4)[0] == sg.OK


# Refusals (CPU).

BIG = 1 << 33


def test_the_headers_declare_the_binding_names(lib):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for header, names in (("sgemm_linear.h", sg.LINEAR_SYMBOLS), ("sgemm_moe.h", sg.MOE_SYMBOLS)):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", header)).read(),
                      flags=re.S)
        found = re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, re.M)
        assert sorted(found) == sorted(names)
        for n in names:
            assert hasattr(lib, n) and hasattr(sg, n)


def test_the_package_imports_torch_only_when_it_is_needed():
    import os
    import subprocess
    import sys
    code = ("import sys, tiled_fp32_gemm_amd as sg, tiled_fp32_gemm_amd.build; "
            "assert 'torch' not in sys.modules; sg.linear; assert 'torch' in sys.modules; "
            "assert all(hasattr(sg, n) for n in sg.__all__); "
            "assert not hasattr(sg, 'no_such_name')")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)


def call(ta=0, tb=0, M=4, N=8, K=16, A=BIG, lda=None, B=BIG + (1 << 31), ldb=None,
         C=BIG + (1 << 32), ldc=None, ws=0, ws_bytes=0, **ep):
    lda = max(M if ta else K, 1) if lda is None else lda
    ldb = max(K if tb else N, 1) if ldb is None else ldb
    ldc = max(N, 1) if ldc is None else ldc
    e = None
    if ep:
        e = sg.Epilogue()
        for k, v in ep.items():
            setattr(e, k, v)
    return sg.sgemm_linear(ta, tb, M, N, K, A, lda, B, ldb, C, ldc, e, 0, ws, ws_bytes)


FAR = BIG + (1 << 40)


@pytest.mark.parametrize("args", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(ta=2), dict(tb=-1),
    dict(lda=15), dict(ta=1, lda=3), dict(ldb=7), dict(tb=1, ldb=15), dict(ldc=7),
    dict(A=0), dict(B=0), dict(C=0), dict(A=BIG + 2), dict(B=BIG + 1), dict(C=FAR + 3),
    dict(C=BIG + 16), dict(C=BIG + (1 << 31) + 64),
    dict(act=5), dict(act=-1), dict(bias=FAR + 2), dict(bias=BIG + (1 << 32) + 8),
    dict(residual=FAR, ldr=7), dict(residual=FAR + 1, ldr=8),
    dict(residual=BIG + (1 << 32), ldr=9),            # C with another row pitch
    dict(residual=BIG + (1 << 32) + 16, ldr=8),       # overlapping C
    dict(preact=FAR, ldp=7), dict(preact=BIG + (1 << 32), ldp=8), dict(preact=BIG, ldp=8),
    dict(preact=BIG + (1 << 31), ldp=8), dict(preact=FAR, ldp=8, residual=FAR, ldr=8),
    dict(preact=FAR, ldp=8, bias=FAR),
    dict(ws=0, ws_bytes=64), dict(ws=FAR, ws_bytes=-4), dict(ws=FAR + 2, ws_bytes=64)])
def test_linear_refuses(lib, args):
    assert call(**args) == sg.ERR_INVALID_ARG


@pytest.mark.parametrize("args", [
    dict(M=(1 << 31) - 1023, C=FAR * 2, B=FAR), dict(K=(1 << 31) - 1023, C=FAR, B=FAR * 2),
    dict(lda=1 << 62), dict(K=1 << 29, ldb=8, B=FAR, C=FAR * 2),
    dict(M=64, lda=1 << 25, B=FAR, C=FAR * 2),
    dict(M=64, N=64, K=64, ldb=1 << 26, B=FAR, C=FAR * 2),
    dict(M=64, ldc=1 << 26, B=FAR, C=FAR * 2), dict(M=64, residual=FAR * 3, ldr=1 << 26),
    dict(M=64, preact=FAR * 3, ldp=1 << 26), dict(ldb=1 << 31, B=FAR, C=FAR * 2)])
def test_linear_unsupported(lib, args):
    assert call(**args) == sg.ERR_UNSUPPORTED


def test_linear_with_nothing_to_do(lib):
    for a in (dict(M=0), dict(N=0)):
        assert call(A=0, B=0, C=0, **a) == sg.OK
    assert sg.sgemm_act_backward(4, 0, 0, 1, 0, 1, 1, 0, 1) == sg.OK
    assert sg.sgemm_act_backward(4, 8, BIG, 8, 0, 1, 0, 0, 1) == sg.OK   # nothing wanted
    for f in (sg.sgemm_linear_workspace_bytes,):
        assert f(0, 0, -1, 4, 4) == f(0, 0, 0, 4, 4) == f(0, 0, 4, 4, -1) == 0
    assert sg.sgemm_act_backward_workspace_bytes(-1, 4) == 0
    assert sg.sgemm_act_backward_workspace_bytes(4, 0) == 0


@pytest.mark.parametrize("args", [
    (-1, 8, BIG, 8, FAR, 8, 1, FAR * 2, 8, 0), (4, -1, BIG, 8, FAR, 8, 1, FAR * 2, 8, 0),
    (4, 8, BIG, 7, FAR, 8, 1, FAR * 2, 8, 0), (4, 8, BIG, 8, FAR, 7, 1, FAR * 2, 8, 0),
    (4, 8, BIG, 8, FAR, 8, 1, FAR * 2, 7, 0), (4, 8, BIG, 8, FAR, 8, 5, FAR * 2, 8, 0),
    (4, 8, 0, 8, FAR, 8, 1, FAR * 2, 8, 0), (4, 8, BIG, 8, 0, 8, 1, FAR * 2, 8, 0),
    (4, 8, BIG + 2, 8, FAR, 8, 1, FAR * 2, 8, 0), (4, 8, BIG, 8, FAR, 8, 1, FAR * 2 + 1, 8, 0),
    (4, 8, BIG, 8, FAR, 8, 1, FAR * 2, 8, 2), (4, 8, BIG, 8, FAR, 8, 1, BIG + 16, 8, 0),
    (4, 8, BIG, 8, FAR, 8, 1, BIG, 9, 0), (4, 8, BIG, 8, FAR, 8, 1, FAR + 16, 8, 0),
    (4, 8, BIG, 8, FAR, 8, 1, FAR * 2, 8, BIG), (4, 8, BIG, 8, FAR, 8, 1, FAR * 2, 8, FAR),
    (4, 8, BIG, 8, FAR, 8, 1, FAR * 2, 8, FAR * 2)])
def test_act_backward_refuses(lib, args):
    assert sg.sgemm_act_backward(*args) == sg.ERR_INVALID_ARG


def test_act_backward_refuses_a_bad_workspace(lib):
    a = (400000, 8, BIG, 8, FAR, 8, 1, FAR * 2, 8, FAR * 3)
    for ws, n in ((0, 4096), (FAR * 4 + 2, 4096), (FAR * 4, -4), (BIG, 4096), (FAR, 4096),
                  (FAR * 2, 4096), (FAR * 3, 4096)):
        assert sg.sgemm_act_backward(*a, 0, ws, n) == sg.ERR_INVALID_ARG, (ws, n)


def test_the_binding_refuses_what_is_no_gpu_tensor():
    x, y = torch.zeros(4, 4), torch.zeros(4, 4)
    for f in (lambda: sg.linear(x, y), lambda: sg.linear(None, y),
              lambda: sg.linear_backward(x, x, y), lambda: sg.activation_backward(x),
              lambda: sg.linear(x, y, activation="swish"),
              lambda: sg.linear(x, y, activation=["silu"])):
        with pytest.raises(ValueError):
            f()


@pytest.mark.gpu
def test_the_binding_refuses_bad_tensors():
    f = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    A, B = f(4, 6), f(6, 8)
    bad = [lambda: sg.linear(A, f(5, 8)), lambda: sg.linear(A, B, transpose_b=True),
           lambda: sg.linear(A.double(), B), lambda: sg.linear(A, B.half()),
           lambda: sg.linear(A, B.cpu()), lambda: sg.linear(A.t(), B, transpose_a=True),
           lambda: sg.linear(A, B, f(7)), lambda: sg.linear(A, B, f(16)[::2]),
           lambda: sg.linear(A, B, f(1, 8)), lambda: sg.linear(A, B, residual=f(4, 9)),
           lambda: sg.linear(A, B, preact=f(3, 8)), lambda: sg.linear(A, B, out=f(8, 4).t()),
           lambda: sg.linear(A, B, out=f(4, 7)), lambda: sg.linear(A, B, workspace=f(4, 8).t()),
           lambda: sg.linear(A, B, workspace=torch.zeros(4)),
           lambda: sg.linear_backward(f(4, 7), A, B),
           lambda: sg.linear_backward(f(4, 8), A, B, "silu"),
           lambda: sg.linear_backward(f(4, 8), A, B, "silu", f(4, 9))]
    for call_ in bad:
        with pytest.raises(ValueError):
            call_()
    with pytest.raises(sg.SgemmError):     # the result over an operand
        sg.linear(f(6, 6), A[:, :6].new_zeros(6, 6), out=(x := f(6, 6)), preact=x)
