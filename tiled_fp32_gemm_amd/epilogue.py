"""Products with a bias, an activation and a residual, and their gradients
(``include/sgemm_linear.h``), over torch tensors.

``linear`` and ``linear_backward`` follow ``matmul``: float32 GPU tensors,
row-major with any row stride, the current stream unless one is given, a
caller's workspace where sums may be split.  Nothing is differentiated
automatically: ``linear_backward`` is a call of its own.
"""
from __future__ import annotations

import ctypes
from contextlib import contextmanager

import tiled_fp32_gemm_amd as sg

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LINEAR_SYMBOLS = ("sgemm_linear", "sgemm_linear_workspace_bytes", "sgemm_linear_plan_query",
                  "sgemm_act_backward", "sgemm_act_backward_workspace_bytes")


class Epilogue(ctypes.Structure):
    """``sgemm_epilogue``."""
    _fields_ = [("act", ctypes.c_int), ("bias", ctypes.c_void_p), ("ldbias", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("preact", ctypes.c_void_p), ("ldp", ctypes.c_int64)]


def prototypes(lib) -> None:
    i64, ptr, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.sgemm_linear.argtypes = [i32, i32, i64, i64, i64, ptr, i64, ptr, i64, ptr, i64,
                                 ctypes.POINTER(Epilogue), ptr, ptr, i64]
    lib.sgemm_linear.restype = i32
    lib.sgemm_linear_workspace_bytes.argtypes = [i32, i32, i64, i64, i64]
    lib.sgemm_linear_workspace_bytes.restype = i64
    lib.sgemm_linear_plan_query.argtypes = [i32, i32, i64, i64, i64, i64,
                                            ctypes.POINTER(sg.SgemmPlan)]
    lib.sgemm_linear_plan_query.restype = i32
    lib.sgemm_act_backward.argtypes = [i64, i64, ptr, i64, ptr, i64, i32, ptr, i64, ptr, ptr,
                                       ptr, i64]
    lib.sgemm_act_backward.restype = i32
    lib.sgemm_act_backward_workspace_bytes.argtypes = [i64, i64]
    lib.sgemm_act_backward_workspace_bytes.restype = i64


def sgemm_linear(trans_a, trans_b, M, N, K, A, lda, B, ldb, C, ldc, epilogue=None, stream=0,
                 workspace=0, workspace_bytes=0) -> int:
    """C = act(op(A)·op(B) + bias) + residual; returns the status code."""
    return sg.load().sgemm_linear(trans_a, trans_b, M, N, K, A, lda, B, ldb, C, ldc, epilogue,
                                  stream, workspace, workspace_bytes)


def sgemm_linear_workspace_bytes(trans_a, trans_b, M, N, K) -> int:
    """Workspace bytes for ``sgemm_linear``'s fastest plan (0: none)."""
    return sg.load().sgemm_linear_workspace_bytes(trans_a, trans_b, M, N, K)


def sgemm_linear_plan_query(trans_a, trans_b, M, N, K, workspace_bytes=0):
    """``(status, SgemmPlan)`` for what ``sgemm_linear`` would launch."""
    plan = sg.SgemmPlan()
    st = sg.load().sgemm_linear_plan_query(trans_a, trans_b, M, N, K, workspace_bytes,
                                           ctypes.byref(plan))
    return st, plan


def sgemm_act_backward(M, N, dC, lddc, preact, ldp, act, dZ, lddz, dbias=0, stream=0,
                       workspace=0, workspace_bytes=0) -> int:
    """dZ = dC * act'(preact) and its column sums; returns the status code."""
    return sg.load().sgemm_act_backward(M, N, dC, lddc, preact, ldp, act, dZ, lddz, dbias,
                                        stream, workspace, workspace_bytes)


def sgemm_act_backward_workspace_bytes(M, N) -> int:
    return sg.load().sgemm_act_backward_workspace_bytes(M, N)


# Checks and marshalling shared with the grouped products.

def _act(activation) -> int:
    try:
        return ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}: "
                         f"got {activation!r}") from None


def _float(t, name: str, device, shape=None):
    """A float32 tensor on `device`, of `shape` where one is given."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a float32 tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}: got {tuple(t.shape)}")
    return t


def _gpu(t, name: str):
    """The device of an operand that has to be on a GPU."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a tensor on a GPU")
    return t.device


def _unit(t, name: str) -> int:
    """The address of a 1-D tensor with unit stride."""
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be 1-D with unit stride")
    return t.data_ptr()


def _workspace(workspace, device) -> tuple[int, int]:
    import torch
    if workspace is None:
        return 0, 0
    if (not isinstance(workspace, torch.Tensor) or workspace.device != device
            or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    n = workspace.numel() * workspace.element_size()
    return (workspace.data_ptr(), n) if n else (0, 0)


@contextmanager
def _on(device, stream):
    """`device` current, and `stream` (default: the device's current one) the
    stream that tensors made inside belong to; yields the stream's handle."""
    import torch
    if stream is None:
        if torch.cuda.current_device() == device.index:
            yield torch.cuda.current_stream().cuda_stream
            return
        with torch.cuda.device(device):
            yield torch.cuda.current_stream().cuda_stream
        return
    if stream.device != device:
        raise ValueError(f"stream must be of {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield stream.cuda_stream


def _check(status: int, what: str) -> None:
    if status != sg.OK:
        raise sg.SgemmError(status, what)


def _op_shape(t, name: str, transposed: bool) -> tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = t.shape
    return (c, r) if transposed else (r, c)


def _epilogue(act, bias, ld_bias, residual, preact):
    """``Epilogue`` of checked tensors, or None for an empty one."""
    if not act and bias is None and residual is None and preact is None:
        return None
    e = Epilogue()
    e.act = act
    if bias is not None:
        e.bias, e.ldbias = bias.data_ptr(), ld_bias
    if residual is not None:
        e.residual, e.ldr = residual.data_ptr(), sg._ld(residual, "residual")
    if preact is not None:
        e.preact, e.ldp = preact.data_ptr(), sg._ld(preact, "preact")
    return e


def linear(A, B, bias=None, activation="none", residual=None, *, transpose_a=False,
           transpose_b=False, out=None, preact=None, stream=None, workspace=None):
    """``out = act(op(A) @ op(B) + bias) + residual``.

    ``op`` is the transpose where ``transpose_a`` / ``transpose_b`` say so (B
    stored out x in: ``transpose_b``).  ``bias`` has N values; ``residual`` is
    M x N and may be ``out`` itself; ``preact`` (M x N) receives
    ``op(A) @ op(B) + bias``, which ``linear_backward`` needs for an
    activation.  ``workspace`` (any contiguous GPU tensor) is room for K to be
    split, see ``sgemm_linear_workspace_bytes``.  Raises ``ValueError`` on bad
    tensors and ``SgemmError`` on a library error.
    """
    import torch
    act = _act(activation)
    dev = _gpu(A, "A")
    M, K = _op_shape(_float(A, "A", dev), "A", transpose_a)
    K2, N = _op_shape(_float(B, "B", dev), "B", transpose_b)
    if K2 != K:
        raise ValueError(f"shape mismatch: op(A) is {M} x {K}, op(B) is {K2} x {N}")
    lda, ldb = sg._ld(A, "A"), sg._ld(B, "B")
    if bias is not None:
        _unit(_float(bias, "bias", dev, (N,)), "bias")
    if residual is not None:
        _float(residual, "residual", dev, (M, N))
    if preact is not None:
        _float(preact, "preact", dev, (M, N))
    epilogue = _epilogue(act, bias, N, residual, preact)
    ws, ws_bytes = _workspace(workspace, dev)
    if out is not None:
        _float(out, "out", dev, (M, N))
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=dev)
        st = sgemm_linear(transpose_a, transpose_b, M, N, K, A.data_ptr(), lda, B.data_ptr(),
                          ldb, out.data_ptr(), sg._ld(out, "out"), epilogue, s, ws, ws_bytes)
    _check(st, "sgemm_linear")
    return out


def activation_backward(dC, activation="none", preact=None, *, bias_grad=True, out=None,
                        stream=None, workspace=None):
    """``(dZ, dbias)``: ``dZ = dC * act'(preact)`` and its column sums (None
    without ``bias_grad``).

    ``out`` receives dZ and may be ``dC`` or ``preact``.  For activation
    "none" dZ is dC: unless ``out`` asks for a copy, dC itself is returned.
    """
    import torch
    act = _act(activation)
    dev = _gpu(dC, "dC")
    M, N = _op_shape(_float(dC, "dC", dev), "dC", False)
    lddc, z, ldz = sg._ld(dC, "dC"), 0, 1
    if act:
        if preact is None:
            raise ValueError(f"activation {activation!r} needs preact")
        z, ldz = _float(preact, "preact", dev, (M, N)).data_ptr(), sg._ld(preact, "preact")
    if out is not None:
        _float(out, "out", dev, (M, N))
    ws, ws_bytes = _workspace(workspace, dev)
    with _on(dev, stream) as s:
        dz = out
        if dz is None and act:
            dz = torch.empty((M, N), dtype=torch.float32, device=dev)
        dbias = torch.empty(N, dtype=torch.float32, device=dev) if bias_grad else None
        st = sgemm_act_backward(M, N, dC.data_ptr(), lddc, z, ldz, act,
                                0 if dz is None else dz.data_ptr(),
                                1 if dz is None else sg._ld(dz, "out"),
                                dbias.data_ptr() if bias_grad else 0, s, ws, ws_bytes)
    _check(st, "sgemm_act_backward")
    return (dC if dz is None else dz), dbias


def linear_backward(dC, A, B, activation="none", preact=None, *, transpose_a=False,
                    transpose_b=False, bias_grad=True, stream=None, workspace=None):
    """``(dA, dB, dbias)`` of ``linear`` for the gradient ``dC`` of its output:
    dA and dB in the shapes A and B are stored in, dbias None without
    ``bias_grad``.  ``preact`` is what ``linear`` stored (not needed for
    activation "none").  The residual's gradient is ``dC``.
    """
    dev = _gpu(dC, "dC")
    M, K = _op_shape(_float(A, "A", dev), "A", transpose_a)
    K2, N = _op_shape(_float(B, "B", dev), "B", transpose_b)
    if K2 != K:
        raise ValueError(f"shape mismatch: op(A) is {M} x {K}, op(B) is {K2} x {N}")
    _float(dC, "dC", dev, (M, N))
    with _on(dev, stream):   # dZ, when it is made here, belongs to the stream
        dZ, dbias = activation_backward(dC, activation, preact, bias_grad=bias_grad,
                                        workspace=workspace)
        if transpose_a:
            dA = linear(B, dZ, transpose_a=transpose_b, transpose_b=True, workspace=workspace)
        else:
            dA = linear(dZ, B, transpose_b=not transpose_b, workspace=workspace)
        if transpose_b:
            dB = linear(dZ, A, transpose_a=True, transpose_b=transpose_a, workspace=workspace)
        else:
            dB = linear(A, dZ, transpose_a=not transpose_a, workspace=workspace)
    return dA, dB, dbias
