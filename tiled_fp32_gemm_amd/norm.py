"""Layer norm and its gradients (``include/sgemm_norm.h``), over torch tensors.

``layer_norm`` and ``layer_norm_backward`` follow ``linear``: float32 GPU
tensors, row-major with any row stride, the current stream unless one is given,
nothing differentiated automatically.
"""
from __future__ import annotations

import ctypes

import tiled_fp32_gemm_amd as sg

from .epilogue import _check, _device, _matrix, _on, _own, _sized, _vector, _workspace

NORM_SYMBOLS = ("sgemm_layer_norm", "sgemm_layer_norm_backward",
                "sgemm_layer_norm_backward_workspace_bytes")


def prototypes(lib) -> None:
    i64, ptr, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    lib.sgemm_layer_norm.argtypes = [i64, i64, ptr, i64, ptr, ptr, f32, ptr, i64, ptr, ptr, ptr]
    lib.sgemm_layer_norm.restype = ctypes.c_int
    lib.sgemm_layer_norm_backward.argtypes = [i64, i64, ptr, i64, ptr, i64, ptr, ptr, ptr, ptr,
                                              i64, ptr, i64, ptr, ptr, ptr, ptr, i64]
    lib.sgemm_layer_norm_backward.restype = ctypes.c_int
    lib.sgemm_layer_norm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.sgemm_layer_norm_backward_workspace_bytes.restype = i64


def sgemm_layer_norm(*args) -> int:
    """``sgemm_layer_norm`` with the C arguments; returns the status code."""
    return sg.load().sgemm_layer_norm(*args)


def sgemm_layer_norm_backward(*args) -> int:
    """``sgemm_layer_norm_backward`` with the C arguments; returns the status code."""
    return sg.load().sgemm_layer_norm_backward(*args)


def sgemm_layer_norm_backward_workspace_bytes(M, N) -> int:
    return sg.load().sgemm_layer_norm_backward_workspace_bytes(M, N)


def _optional(t, name: str, dev: int, n: int):
    return None if t is None else _vector(t, name, dev, n)


def layer_norm(X, weight=None, bias=None, eps=1e-5, *, out=None, mean=None, rstd=None,
               stream=None):
    """``(X - mean) * rstd * weight + bias`` for each row of X (M x N), where
    ``rstd = 1 / sqrt(variance + eps)``.

    ``weight`` and ``bias`` have N values.  ``mean`` and ``rstd`` (M values)
    receive the rows' statistics, which ``layer_norm_backward`` needs.  ``out``
    may be ``X``.
    """
    dev = _device(X, "X")
    M, N, ldx = _matrix(X, "X", dev)
    eps = float(eps)
    if not 0 <= eps < float("inf"):
        raise ValueError(f"eps must be 0 or more: got {eps}")
    w, b = _optional(weight, "weight", dev, N), _optional(bias, "bias", dev, N)
    m, r = _optional(mean, "mean", dev, M), _optional(rstd, "rstd", dev, M)
    ldy = max(N, 1) if out is None else _sized(out, "out", dev, M, N)

    def call(s):
        y = X.new_empty(M, N) if out is None else out
        _check(sg.load().sgemm_layer_norm(M, N, X.data_ptr(), ldx, w, b, eps, y.data_ptr(), ldy,
                                          m, r, s), "sgemm_layer_norm")
        return y
    return _on(dev, stream, call)


def layer_norm_backward(dY, X, mean, rstd, weight=None, residual=None, *, weight_grad=True,
                        out=None, stream=None, workspace=None):
    """``(dX, dweight, dbias)`` of ``layer_norm`` for the gradient ``dY`` of its
    result, with the X, mean and rstd of that call; dweight and dbias are None
    without ``weight_grad``.

    ``residual`` (M x N), the gradient that reaches X by another way, is added
    to dX.  ``out`` receives dX and may be ``dY``, ``X`` or ``residual``.
    Without a ``workspace`` one is made for the sums.
    """
    dev = _device(dY, "dY")
    M, N, lddy = _matrix(dY, "dY", dev)
    ldx = _sized(X, "X", dev, M, N)
    m, r = _vector(mean, "mean", dev, M), _vector(rstd, "rstd", dev, M)
    w = _optional(weight, "weight", dev, N)
    ldr, res = 1, None
    if residual is not None:
        ldr, res = _sized(residual, "residual", dev, M, N), residual.data_ptr()
    ld = max(N, 1) if out is None else _sized(out, "out", dev, M, N)
    ws, ws_bytes = _workspace(workspace, dev)
    lib = sg.load()
    need = 0
    if workspace is None and weight_grad:
        need = lib.sgemm_layer_norm_backward_workspace_bytes(M, N)

    def call(s):
        dx = dY.new_empty(M, N) if out is None else out
        dw, db = (dY.new_empty(N), dY.new_empty(N)) if weight_grad else (None, None)
        own, room, size = _own(dY, need, ws, ws_bytes)  # noqa: F841
        _check(lib.sgemm_layer_norm_backward(
            M, N, dY.data_ptr(), lddy, X.data_ptr(), ldx, m, r, w, res, ldr,
            dx.data_ptr(), ld, dw.data_ptr() if weight_grad else None,
            db.data_ptr() if weight_grad else None, s, room, size), "sgemm_layer_norm_backward")
        return dx, dw, db
    return _on(dev, stream, call)
