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

import tiled_fp32_gemm_amd as sg

from .epilogue import (Epilogue, _act, _check, _epilogue, _float, _gpu, _on, _op_shape,
                       _workspace)

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


def _index(t, name: str, device, shape=None) -> int:
    """The address of a contiguous int32 tensor on `device`."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise ValueError(f"{name} must be an int32 tensor on {device}")
    if not t.is_contiguous() or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name} must be contiguous"
                         + ("" if shape is None else f" and of shape {shape}"))
    return t.data_ptr()


def _place(place, device) -> tuple[int, int]:
    """T and top of a place tensor."""
    _index(place, "place", device)
    if place.dim() != 2:
        raise ValueError("place must be 2-D (tokens x choices)")
    return tuple(place.shape)


def _weights(weights, device, shape) -> int:
    if weights is None:
        return 0
    _float(weights, "weights", device, shape)
    if not weights.is_contiguous():
        raise ValueError("weights must be contiguous")
    return weights.data_ptr()


def moe_sort(experts, num_experts, *, stream=None, workspace=None):
    """``(offsets, order, place)`` of a T x top (or 1-D) tensor of expert ids,
    int32 or int64: expert e's rows are ``offsets[e]`` to ``offsets[e+1]-1``,
    row r holds choice ``order[r]`` (-1 behind the last row), choice c is in
    row ``place`` [c] (-1: dropped; shaped like ``experts``).  Equal experts
    keep their order.  Without a ``workspace`` one is made for the call.
    """
    import torch
    dev = _gpu(experts, "experts")
    if experts.dtype not in (torch.int32, torch.int64) or not experts.is_contiguous():
        raise ValueError("experts must be a contiguous int32 or int64 tensor")
    E, n = int(num_experts), experts.numel()
    if E < 1:
        raise ValueError("num_experts must be positive")
    with _on(dev, stream) as s:
        need = sgemm_moe_sort_workspace_bytes(n, E)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws, ws_bytes = _workspace(workspace, dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        order = torch.empty(n, dtype=torch.int32, device=dev)
        place = torch.empty(experts.shape, dtype=torch.int32, device=dev)
        st = sgemm_moe_sort(n, E, experts.data_ptr(), experts.element_size(),
                            offsets.data_ptr(), order.data_ptr(), place.data_ptr(), s, ws,
                            ws_bytes)
    _check(st, "sgemm_moe_sort")
    return offsets, order, place


def moe_permute(X, place, *, out=None, stream=None):
    """Each token's row of X (T x H) at the rows ``place`` gives it: T·top x H.
    Its gradient is ``moe_unpermute(dXp, place)``."""
    import torch
    dev = _gpu(X, "X")
    T, top = _place(place, dev)
    _, H = _op_shape(_float(X, "X", dev), "X", False)
    if X.shape[0] != T:
        raise ValueError(f"X has {X.shape[0]} rows, place {T}")
    if out is not None:
        _float(out, "out", dev, (T * top, H))
    ldx = sg._ld(X, "X")
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((T * top, H), dtype=torch.float32, device=dev)
        st = sgemm_moe_permute(T, top, H, X.data_ptr(), ldx, place.data_ptr(), out.data_ptr(),
                               sg._ld(out, "out"), s)
    _check(st, "sgemm_moe_permute")
    return out


def moe_unpermute(Yp, place, weights=None, *, out=None, stream=None):
    """T x H: each token's rows of Yp (T·top x H) times their ``weights``
    (T x top; None: 1), summed; 0 for a token without rows."""
    import torch
    dev = _gpu(Yp, "Yp")
    T, top = _place(place, dev)
    _, H = _op_shape(_float(Yp, "Yp", dev), "Yp", False)
    if Yp.shape[0] != T * top:
        raise ValueError(f"Yp has {Yp.shape[0]} rows, place {T} x {top}")
    w = _weights(weights, dev, (T, top))
    if out is not None:
        _float(out, "out", dev, (T, H))
    ldyp = sg._ld(Yp, "Yp")
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((T, H), dtype=torch.float32, device=dev)
        st = sgemm_moe_unpermute(T, top, H, Yp.data_ptr(), ldyp, place.data_ptr(), w,
                                 out.data_ptr(), sg._ld(out, "out"), s)
    _check(st, "sgemm_moe_unpermute")
    return out


def moe_unpermute_backward(dY, Yp, place, weights=None, *, out=None, stream=None):
    """``(dYp, dweights)`` of ``moe_unpermute`` for the gradient dY (T x H) of
    its result.  ``out`` receives dYp and may be ``Yp``."""
    import torch
    dev = _gpu(dY, "dY")
    T, top = _place(place, dev)
    _, H = _op_shape(_float(dY, "dY", dev), "dY", False)
    if dY.shape[0] != T:
        raise ValueError(f"dY has {dY.shape[0]} rows, place {T}")
    _float(Yp, "Yp", dev, (T * top, H))
    w = _weights(weights, dev, (T, top))
    if out is not None:
        _float(out, "out", dev, (T * top, H))
    lddy, ldyp = sg._ld(dY, "dY"), sg._ld(Yp, "Yp")
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((T * top, H), dtype=torch.float32, device=dev)
        dw = torch.empty((T, top), dtype=torch.float32, device=dev)
        st = sgemm_moe_unpermute_backward(T, top, H, dY.data_ptr(), lddy, Yp.data_ptr(), ldyp,
                                          place.data_ptr(), w, out.data_ptr(),
                                          sg._ld(out, "out"), dw.data_ptr(), s)
    _check(st, "sgemm_moe_unpermute_backward")
    return out, dw


def _groups(B, offsets, device, transposed: bool):
    """Groups, K, N, leading dimension and stride of a stack of matrices."""
    if _float(B, "B", device).dim() != 3:
        raise ValueError("B must be 3-D (one matrix per group)")
    G, K, N = B.shape
    if transposed:
        K, N = N, K
    ldb = sg._ld(B[0], "B") if G else max(B.shape[2], 1)
    stride = B.stride(0) if G > 1 else B.shape[1] * ldb
    _index(offsets, "offsets", device, (G + 1,))
    return G, K, N, ldb, stride


def grouped_linear(A, B, offsets, bias=None, activation="none", residual=None, *,
                   transpose_b=False, out=None, preact=None, stream=None, workspace=None):
    """``linear`` for each group g's rows ``offsets[g]`` to ``offsets[g+1]-1``
    of A (M x K) with that group's matrix ``B[g]`` (K x N; N x K with
    ``transpose_b``) and bias ``bias[g]``."""
    import torch
    act = _act(activation)
    dev = _gpu(A, "A")
    M, K = _op_shape(_float(A, "A", dev), "A", False)
    G, K2, N, ldb, stride = _groups(B, offsets, dev, transpose_b)
    if K2 != K:
        raise ValueError(f"shape mismatch: A is {M} x {K}, op(B[g]) is {K2} x {N}")
    lda, ld_bias = sg._ld(A, "A"), N
    if bias is not None:
        ld_bias = sg._ld(_float(bias, "bias", dev, (G, N)), "bias")
    if residual is not None:
        _float(residual, "residual", dev, (M, N))
    if preact is not None:
        _float(preact, "preact", dev, (M, N))
    epilogue = _epilogue(act, bias, max(ld_bias, 1), residual, preact)
    ws, ws_bytes = _workspace(workspace, dev)
    if out is not None:
        _float(out, "out", dev, (M, N))
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=dev)
        st = sgemm_grouped(transpose_b, M, N, K, G, offsets.data_ptr(), A.data_ptr(), lda,
                           B.data_ptr(), ldb, stride, out.data_ptr(), sg._ld(out, "out"),
                           epilogue, s, ws, ws_bytes)
    _check(st, "sgemm_grouped")
    return out


def grouped_linear_backward(dC, A, B, offsets, activation="none", preact=None, *,
                            transpose_b=False, bias_grad=True, stream=None, workspace=None):
    """``(dA, dB, dbias)`` of ``grouped_linear``: dA for the groups' rows, dB
    stored like B and dbias (groups x N; None without ``bias_grad``) 0 for a
    group without rows.  The residual's gradient is ``dC``."""
    import torch
    act = _act(activation)
    dev = _gpu(dC, "dC")
    M, K = _op_shape(_float(A, "A", dev), "A", False)
    G, K2, N, _, _ = _groups(B, offsets, dev, transpose_b)
    if K2 != K:
        raise ValueError(f"shape mismatch: A is {M} x {K}, op(B[g]) is {K2} x {N}")
    lddc = sg._ld(_float(dC, "dC", dev, (M, N)), "dC")
    z, ldz = 0, 1
    if act:
        if preact is None:
            raise ValueError(f"activation {activation!r} needs preact")
        z, ldz = _float(preact, "preact", dev, (M, N)).data_ptr(), sg._ld(preact, "preact")
    lda = sg._ld(A, "A")
    ws, ws_bytes = _workspace(workspace, dev)
    with _on(dev, stream) as s:
        dZ, lddz = dC, lddc
        if act:
            dZ, lddz = torch.empty((M, N), dtype=torch.float32, device=dev), max(N, 1)
        dbias = torch.empty((G, N), dtype=torch.float32, device=dev) if bias_grad else None
        _check(sgemm_grouped_act_backward(
            M, N, G, offsets.data_ptr(), dC.data_ptr(), lddc, z, ldz, act,
            dZ.data_ptr() if act else 0, lddz, dbias.data_ptr() if bias_grad else 0, max(N, 1), s,
            ws, ws_bytes), "sgemm_grouped_act_backward")
        dA = grouped_linear(dZ, B, offsets, transpose_b=not transpose_b, workspace=workspace)
        dB = torch.empty(B.shape, dtype=torch.float32, device=dev)
        _check(sgemm_grouped_wgrad(
            transpose_b, M, N, K, G, offsets.data_ptr(), A.data_ptr(), lda, dZ.data_ptr(), lddz,
            dB.data_ptr(), max(B.shape[2], 1), B.shape[1] * max(B.shape[2], 1), s, ws, ws_bytes),
            "sgemm_grouped_wgrad")
    return dA, dB, dbias
