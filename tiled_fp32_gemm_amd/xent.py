"""Softmax cross entropy of a product's rows, without the product in memory, and
its gradients (``include/sgemm_xent.h``), over torch tensors.

``linear_cross_entropy`` is ``linear`` into a vocabulary with its loss: float32 GPU
tensors, row-major with any row stride, the current stream unless one is given,
nothing differentiated automatically.
"""
from __future__ import annotations

import ctypes

import torch

import tiled_fp32_gemm_amd as sg

from .epilogue import _check, _device, _inner, _on, _own, _vector, _workspace

XENT_SYMBOLS = ("sgemm_linear_xent", "sgemm_linear_xent_workspace_bytes",
                "sgemm_linear_xent_backward", "sgemm_linear_xent_backward_workspace_bytes",
                "sgemm_linear_xent_backward_least_bytes")


def prototypes(lib) -> None:
    i64, ptr, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    sizes = [i32, i64, i64, i64]
    operands = [*sizes, ptr, i64, ptr, i64, ptr, i32]
    lib.sgemm_linear_xent.argtypes = [*operands, ptr, ptr, ptr, ptr, i64]
    lib.sgemm_linear_xent.restype = i32
    lib.sgemm_linear_xent_backward.argtypes = [*operands, ptr, ptr, ptr, i64, ptr, i64, ptr, ptr,
                                               i64]
    lib.sgemm_linear_xent_backward.restype = i32
    for name in XENT_SYMBOLS:
        if name.endswith("_bytes"):
            f = getattr(lib, name)
            f.argtypes, f.restype = sizes, i64


def _caller(name: str):
    def call(*args) -> int:
        return getattr(sg.load(), name)(*args)
    call.__name__ = call.__qualname__ = name
    call.__doc__ = f"``{name}`` with the C arguments (see the C header)."
    return call


(sgemm_linear_xent, sgemm_linear_xent_workspace_bytes, sgemm_linear_xent_backward,
 sgemm_linear_xent_backward_workspace_bytes,
 sgemm_linear_xent_backward_least_bytes) = map(_caller, XENT_SYMBOLS)


def _targets(targets, dev: int, T: int) -> tuple[int, int]:
    try:
        good = (targets.dtype in (torch.int32, torch.int64) and targets.get_device() == dev
                and targets.shape == (T,) and targets.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        raise ValueError(f"targets must be {T} contiguous int32 or int64 ids on cuda:{dev}")
    return targets.data_ptr(), targets.element_size()


def linear_cross_entropy(A, B, targets, *, transpose_b=False, out=None, lse=None, stream=None,
                         workspace=None):
    """The T losses ``log(sum(exp(z))) - z[target]`` of the rows z of ``A @
    op(B)``: A is T x H, B is H x V (V x H with ``transpose_b``), ``targets`` T
    ids, int32 or int64.

    A row whose target is outside 0 .. V-1 has loss 0 and no gradient.  ``lse`` (T
    values) receives the logarithms, which ``linear_cross_entropy_backward``
    needs.  Without a ``workspace`` (``sgemm_linear_xent_workspace_bytes``) one is
    made for the call.
    """
    dev = _device(A, "A")
    T, V, H, ldx, ldb = _inner(A, B, dev, False, transpose_b)
    ids, id_bytes = _targets(targets, dev, T)
    log = None if lse is None else _vector(lse, "lse", dev, T)
    if out is not None:
        _vector(out, "out", dev, T)
    tb = bool(transpose_b)
    ws, ws_bytes = _workspace(workspace, dev)
    lib = sg.load()
    need = 0 if workspace is not None else lib.sgemm_linear_xent_workspace_bytes(tb, T, V, H)

    def call(s):
        loss = A.new_empty(T) if out is None else out
        own, room, size = _own(A, need, ws, ws_bytes)  # noqa: F841
        _check(lib.sgemm_linear_xent(tb, T, V, H, A.data_ptr(), ldx, B.data_ptr(), ldb, ids,
                                     id_bytes, loss.data_ptr(), log, s, room, size),
               "sgemm_linear_xent")
        return loss
    return _on(dev, stream, call)


def linear_cross_entropy_backward(dloss, A, B, targets, lse, *, transpose_b=False, a_grad=True,
                                  b_grad=True, stream=None, workspace=None):
    """``(dA, dB)`` of ``linear_cross_entropy`` for the gradients ``dloss`` of
    its T losses, with the operands of that call and the ``lse`` it gave: dA 0 in
    rows without a target, dB stored like B; None without ``a_grad`` or
    ``b_grad``.

    ``workspace`` is room for a piece of the logits' gradient and the rows it is
    made of (``sgemm_linear_xent_backward_workspace_bytes``; with less, down to
    ``sgemm_linear_xent_backward_least_bytes``, there are more pieces).  Without
    one it is made for the call.
    """
    dev = _device(A, "A")
    T, V, H, ldx, ldb = _inner(A, B, dev, False, transpose_b)
    ids, id_bytes = _targets(targets, dev, T)
    log, grad = _vector(lse, "lse", dev, T), _vector(dloss, "dloss", dev, T)
    tb = bool(transpose_b)
    ws, ws_bytes = _workspace(workspace, dev)
    lib = sg.load()
    need = 0
    if workspace is None:
        need = lib.sgemm_linear_xent_backward_workspace_bytes(tb, T, V, H)

    def call(s):
        da = A.new_empty(T, H) if a_grad else None
        db = B.new_empty(B.shape) if b_grad else None
        own, room, size = _own(A, need, ws, ws_bytes)  # noqa: F841
        _check(lib.sgemm_linear_xent_backward(
            tb, T, V, H, A.data_ptr(), ldx, B.data_ptr(), ldb, ids, id_bytes, log, grad,
            da.data_ptr() if a_grad else None, max(H, 1), db.data_ptr() if b_grad else None,
            max(B.shape[1], 1), s, room, size), "sgemm_linear_xent_backward")
        return da, db
    return _on(dev, stream, call)
