"""Mixture-of-experts routing and the experts' products
(``include/sgemm_moe.h``), over torch tensors.

    offsets, order, place = moe_sort(experts, E)          # experts: T x top ids
    xp = moe_permute(x, place)                            # T·top rows, by expert
    hp = grouped_linear(xp, W1, offsets, b1, "silu")
    yp = grouped_linear(hp, W2, offsets, b2)
    y = moe_unpermute(yp, place, weights)                 # T rows

How many rows an expert has stays on the GPU.  Choices outside 0 .. E-1 are
dropped; rows from ``offsets[E]`` on belong to no expert, and no call reads or
writes them (in a tensor that a call makes they hold anything).
"""
from __future__ import annotations

import ctypes

import torch

import tiled_fp32_gemm_amd as sg

from .epilogue import (Epilogue, _act, _check, _device, _epilogue, _float, _matrix, _on, _own,
                       _sized, _workspace)

MOE_SYMBOLS = ("sgemm_moe_sort", "sgemm_moe_sort_workspace_bytes", "sgemm_moe_permute",
               "sgemm_moe_unpermute", "sgemm_moe_unpermute_backward", "sgemm_grouped",
               "sgemm_grouped_workspace_bytes", "sgemm_grouped_wgrad",
               "sgemm_grouped_wgrad_workspace_bytes", "sgemm_grouped_act_backward",
               "sgemm_grouped_act_backward_workspace_bytes")
MOE_MAX_EXPERTS = 1024     # SGEMM_MOE_MAX_EXPERTS


def prototypes(lib) -> None:
    i64, ptr, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    ep = ctypes.POINTER(Epilogue)
    for name, args in {
            "sgemm_moe_sort": [i64, i64, ptr, i32, ptr, ptr, ptr, ptr, ptr, i64],
            "sgemm_moe_permute": [i64, i64, i64, ptr, i64, ptr, ptr, i64, ptr],
            "sgemm_moe_unpermute": [i64, i64, i64, ptr, i64, ptr, ptr, ptr, i64, ptr],
            "sgemm_moe_unpermute_backward": [i64, i64, i64, ptr, i64, ptr, i64, ptr, ptr, ptr,
                                             i64, ptr, ptr],
            "sgemm_grouped": [i32, i64, i64, i64, i64, ptr, ptr, i64, ptr, i64, i64, ptr, i64,
                              ep, ptr, ptr, i64],
            "sgemm_grouped_wgrad": [i32, i64, i64, i64, i64, ptr, ptr, i64, ptr, i64, ptr, i64,
                                    i64, ptr, ptr, i64],
            "sgemm_grouped_act_backward": [i64, i64, i64, ptr, ptr, i64, ptr, i64, i32, ptr, i64,
                                           ptr, i64, ptr, ptr, i64]}.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, i32
    for name, args in {"sgemm_moe_sort_workspace_bytes": [i64, i64],
                       "sgemm_grouped_workspace_bytes": [i32, i64, i64, i64, i64],
                       "sgemm_grouped_wgrad_workspace_bytes": [i32, i64, i64, i64, i64],
                       "sgemm_grouped_act_backward_workspace_bytes": [i64, i64, i64]}.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, i64


def _caller(name: str):
    def call(*args) -> int:
        return getattr(sg.load(), name)(*args)
    call.__name__ = call.__qualname__ = name
    call.__doc__ = f"``{name}`` with the C arguments (see the C header)."
    return call


(sgemm_moe_sort, sgemm_moe_sort_workspace_bytes, sgemm_moe_permute, sgemm_moe_unpermute,
 sgemm_moe_unpermute_backward, sgemm_grouped, sgemm_grouped_workspace_bytes,
 sgemm_grouped_wgrad, sgemm_grouped_wgrad_workspace_bytes, sgemm_grouped_act_backward,
 sgemm_grouped_act_backward_workspace_bytes) = map(_caller, MOE_SYMBOLS)


def _index(t, name: str, dev: int, shape=None) -> int:
    """The address of a contiguous int32 tensor on GPU `dev`."""
    try:
        good = t.dtype is torch.int32 and t.get_device() == dev and t.is_contiguous()
    except AttributeError:
        good = False
    if not good or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous int32 tensor on cuda:{dev}"
                         + ("" if shape is None else f" of shape {shape}"))
    return t.data_ptr()


def _place(place, dev: int) -> tuple[int, int, int]:
    """T, top and the address of a place tensor."""
    p = _index(place, "place", dev)
    if place.dim() not in (1, 2):
        raise ValueError("place must be 2-D (tokens x choices) or 1-D (one choice a token)")
    return place.shape[0], place.shape[1] if place.dim() == 2 else 1, p


def _weights(weights, dev: int, place):
    if weights is None:
        return None
    if _float(weights, "weights", dev).shape != place.shape or not weights.is_contiguous():
        raise ValueError(f"weights must be contiguous and shaped like place: {tuple(place.shape)}")
    return weights.data_ptr()


def moe_sort(experts, num_experts, *, stream=None, workspace=None):
    """``(offsets, order, place)`` of a T x top tensor of expert ids (1-D: one a
    token), int32 or int64: expert e's rows are ``offsets[e]`` to ``offsets[e+1]-1``,
    row r holds choice ``order[r]`` (-1 behind the last row), choice c is in
    row ``place`` [c] (-1: dropped; shaped like ``experts``).  Equal experts
    keep their order.  Without a ``workspace`` one is made for the call.
    """
    dev = _device(experts, "experts")
    if experts.dtype not in (torch.int32, torch.int64) or not experts.is_contiguous():
        raise ValueError("experts must be a contiguous int32 or int64 tensor")
    E, n = int(num_experts), experts.numel()
    if E < 1:
        raise ValueError("num_experts must be positive")
    lib = sg.load()
    need = 0 if workspace is not None else lib.sgemm_moe_sort_workspace_bytes(n, E)
    ws, ws_bytes = _workspace(workspace, dev)

    def call(s):
        own, room, size = _own(experts, need, ws, ws_bytes)  # noqa: F841
        offsets = experts.new_empty(E + 1, dtype=torch.int32)
        order = experts.new_empty(n, dtype=torch.int32)
        place = experts.new_empty(experts.shape, dtype=torch.int32)
        st = lib.sgemm_moe_sort(n, E, experts.data_ptr(), experts.element_size(),
                                offsets.data_ptr(), order.data_ptr(), place.data_ptr(), s, room,
                                size)
        _check(st, "sgemm_moe_sort")
        return offsets, order, place
    return _on(dev, stream, call)


def moe_permute(X, place, *, out=None, stream=None):
    """Each token's row of X (T x H) at the rows ``place`` gives it: T·top x H.
    Its gradient is ``moe_unpermute(dXp, place)``."""
    dev = _device(X, "X")
    T, top, p = _place(place, dev)
    rows, H, ldx = _matrix(X, "X", dev)
    if rows != T:
        raise ValueError(f"X has {rows} rows, place {T}")
    ld = max(H, 1) if out is None else _sized(out, "out", dev, T * top, H)

    def call(s):
        xp = X.new_empty(T * top, H) if out is None else out
        _check(sg.load().sgemm_moe_permute(T, top, H, X.data_ptr(), ldx, p, xp.data_ptr(), ld, s),
               "sgemm_moe_permute")
        return xp
    return _on(dev, stream, call)


def moe_unpermute(Yp, place, weights=None, *, out=None, stream=None):
    """T x H: each token's rows of Yp (T·top x H) times their ``weights``
    (shaped like ``place``; None: 1), summed; 0 for a token without rows."""
    dev = _device(Yp, "Yp")
    T, top, p = _place(place, dev)
    rows, H, ldyp = _matrix(Yp, "Yp", dev)
    if rows != T * top:
        raise ValueError(f"Yp has {rows} rows, place {T} x {top}")
    w = _weights(weights, dev, place)
    ld = max(H, 1) if out is None else _sized(out, "out", dev, T, H)

    def call(s):
        y = Yp.new_empty(T, H) if out is None else out
        _check(sg.load().sgemm_moe_unpermute(T, top, H, Yp.data_ptr(), ldyp, p, w, y.data_ptr(),
                                             ld, s), "sgemm_moe_unpermute")
        return y
    return _on(dev, stream, call)


def moe_unpermute_backward(dY, Yp, place, weights=None, *, out=None, stream=None):
    """``(dYp, dweights)`` of ``moe_unpermute`` for the gradient dY (T x H) of
    its result; dweights is shaped like ``place``.  ``out`` receives dYp and may
    be ``Yp``."""
    dev = _device(dY, "dY")
    T, top, p = _place(place, dev)
    rows, H, lddy = _matrix(dY, "dY", dev)
    if rows != T:
        raise ValueError(f"dY has {rows} rows, place {T}")
    ldyp = _sized(Yp, "Yp", dev, T * top, H)
    w = _weights(weights, dev, place)
    ld = max(H, 1) if out is None else _sized(out, "out", dev, T * top, H)

    def call(s):
        dyp = dY.new_empty(T * top, H) if out is None else out
        dw = dY.new_empty(place.shape)
        _check(sg.load().sgemm_moe_unpermute_backward(
            T, top, H, dY.data_ptr(), lddy, Yp.data_ptr(), ldyp, p, w, dyp.data_ptr(), ld,
            dw.data_ptr(), s), "sgemm_moe_unpermute_backward")
        return dyp, dw
    return _on(dev, stream, call)


def _groups(A, B, offsets, dev: int, transposed: bool):
    """M, N, K, groups and the operands' leading dimensions and stride, for
    rows of A and a stack of matrices."""
    M, K, lda = _matrix(A, "A", dev)
    if _float(B, "B", dev).dim() != 3:
        raise ValueError("B must be 3-D (one matrix per group)")
    G, r, c = B.shape
    stride, ldb, unit = B.stride()
    if unit != 1 and c > 1:
        raise ValueError("B must have unit column stride (row-major)")
    if r <= 1:
        ldb = max(c, 1)
    if G <= 1:
        stride = r * ldb
    K2, N = (c, r) if transposed else (r, c)
    if K2 != K:
        raise ValueError(f"shape mismatch: A is {M} x {K}, op(B[g]) is {K2} x {N}")
    return M, N, K, G, lda, ldb, stride, _index(offsets, "offsets", dev, (G + 1,))


def grouped_linear(A, B, offsets, bias=None, activation="none", residual=None, *,
                   transpose_b=False, out=None, preact=None, stream=None, workspace=None):
    """``linear`` for each group g's rows ``offsets[g]`` to ``offsets[g+1]-1``
    of A (M x K) with that group's matrix ``B[g]`` (K x N; N x K with
    ``transpose_b``) and bias ``bias[g]``."""
    act = _act(activation)
    dev = _device(A, "A")
    M, N, K, G, lda, ldb, stride, off = _groups(A, B, offsets, dev, transpose_b)
    ld_bias = 1 if bias is None else _sized(bias, "bias", dev, G, N)
    ldr = 1 if residual is None else _sized(residual, "residual", dev, M, N)
    ldp = 1 if preact is None else _sized(preact, "preact", dev, M, N)
    epilogue = _epilogue(act, bias, ld_bias, residual, ldr, preact, ldp)
    ws, ws_bytes = _workspace(workspace, dev)
    ldc = max(N, 1) if out is None else _sized(out, "out", dev, M, N)

    def call(s):
        c = A.new_empty(M, N) if out is None else out
        _check(sg.load().sgemm_grouped(bool(transpose_b), M, N, K, G, off, A.data_ptr(), lda,
                                       B.data_ptr(), ldb, stride, c.data_ptr(), ldc, epilogue, s,
                                       ws, ws_bytes), "sgemm_grouped")
        return c
    return _on(dev, stream, call)


def grouped_linear_backward(dC, A, B, offsets, activation="none", preact=None, *,
                            transpose_b=False, bias_grad=True, stream=None, workspace=None):
    """``(dA, dB, dbias)`` of ``grouped_linear``: dA for the groups' rows, dB
    stored like B and dbias (groups x N; None without ``bias_grad``) 0 for a
    group without rows.  The residual's gradient is ``dC``.  Without a
    ``workspace`` one is made for dbias, and the products' sums are not split."""
    act = _act(activation)
    dev = _device(dC, "dC")
    M, N, K, G, lda, ldb, stride, off = _groups(A, B, offsets, dev, transpose_b)
    lddc = _sized(dC, "dC", dev, M, N)
    z, ldz = 0, 1
    if act:
        if preact is None:
            raise ValueError(f"activation {activation!r} needs preact")
        ldz = _sized(preact, "preact", dev, M, N)
        z = preact.data_ptr()
    ws, ws_bytes = _workspace(workspace, dev)
    lib = sg.load()
    need = 0
    if workspace is None and bias_grad:
        need = lib.sgemm_grouped_act_backward_workspace_bytes(M, N, G)

    def call(s):
        dZ, lddz = (dC.new_empty(M, N), max(N, 1)) if act else (dC, lddc)
        dbias = dC.new_empty(G, N) if bias_grad else None
        own, *sums = _own(dC, need, ws, ws_bytes)  # noqa: F841
        _check(lib.sgemm_grouped_act_backward(
            M, N, G, off, dC.data_ptr(), lddc, z, ldz, act, dZ.data_ptr() if act else None, lddz,
            dbias.data_ptr() if bias_grad else None, max(N, 1), s, *sums),
            "sgemm_grouped_act_backward")
        dA, dB = A.new_empty(M, K), B.new_empty(B.shape)
        _check(lib.sgemm_grouped(not transpose_b, M, K, N, G, off, dZ.data_ptr(), lddz,
                                 B.data_ptr(), ldb, stride, dA.data_ptr(), max(K, 1), None, s, ws,
                                 ws_bytes), "sgemm_grouped")
        r, c = B.shape[1:]
        _check(lib.sgemm_grouped_wgrad(
            bool(transpose_b), M, N, K, G, off, A.data_ptr(), lda, dZ.data_ptr(), lddz,
            dB.data_ptr(), max(c, 1), r * max(c, 1), s, ws, ws_bytes), "sgemm_grouped_wgrad")
        return dA, dB, dbias
    return _on(dev, stream, call)
