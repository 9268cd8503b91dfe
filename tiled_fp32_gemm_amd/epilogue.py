"""Products with a bias, an activation and a residual, and their gradients
(``include/sgemm_linear.h``), over torch tensors.

``linear`` and ``linear_backward`` follow ``matmul``: float32 GPU tensors,
row-major with any row stride, the current stream unless one is given (what a
call makes then belongs to that stream), a caller's workspace where sums may be
split.  Nothing is differentiated automatically: ``linear_backward`` is a call
of its own.
"""
from __future__ import annotations

import ctypes

import torch

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


# Checks and marshalling shared with the routing calls.  They run before every
# launch and cost as much as a small kernel, so each tensor is asked once for
# what is needed of it.

def _act(activation) -> int:
    try:
        return ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}: "
                         f"got {activation!r}") from None


def _device(t, name: str) -> int:
    """The index of the GPU an operand is on."""
    try:
        dev = t.get_device()
    except AttributeError:
        dev = -1
    if dev < 0:
        raise ValueError(f"{name} must be a tensor on a GPU")
    return dev


def _float(t, name: str, dev: int):
    """A float32 tensor on GPU `dev`."""
    try:
        good = t.dtype is torch.float32 and t.get_device() == dev
    except AttributeError:
        good = False
    if not good:
        raise ValueError(f"{name} must be a float32 tensor on cuda:{dev}")
    return t


def _matrix(t, name: str, dev: int) -> tuple[int, int, int]:
    """Rows, columns and leading dimension of a row-major float32 matrix."""
    _float(t, name, dev)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = t.shape
    ld, unit = t.stride()
    if unit != 1 and c > 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    return r, c, ld if r > 1 else max(c, 1)


def _sized(t, name: str, dev: int, rows: int, cols: int) -> int:
    """The leading dimension of a rows x cols float32 matrix."""
    r, c, ld = _matrix(t, name, dev)
    if r != rows or c != cols:
        raise ValueError(f"{name} must be {rows} x {cols}: got {r} x {c}")
    return ld


def _vector(t, name: str, dev: int, n: int) -> int:
    """The address of n floats with unit stride."""
    _float(t, name, dev)
    if t.dim() != 1 or t.numel() != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be 1-D of {n} with unit stride")
    return t.data_ptr()


def _workspace(workspace, dev: int) -> tuple[int, int]:
    if workspace is None:
        return 0, 0
    try:
        good = workspace.get_device() == dev and workspace.is_contiguous()
    except AttributeError:
        good = False
    if not good:
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    n = workspace.numel() * workspace.element_size()
    return (workspace.data_ptr(), n) if n else (0, 0)


def _own(like, need: int, ws: int, ws_bytes: int):
    """A workspace of `need` bytes made for a call (0: the caller's), its address
    and size.  It has to be held until the last launch that uses it."""
    if not need:
        return None, ws, ws_bytes
    own = like.new_empty(need, dtype=torch.uint8)
    return own, own.data_ptr(), need


def _on(dev: int, stream, body):
    """``body(handle)`` with GPU `dev` current and `stream` (default: its
    current one) the stream that tensors made inside belong to."""
    if stream is None:
        if torch._C._cuda_getDevice() == dev:
            return body(torch._C._cuda_getCurrentRawStream(dev))
        with torch.cuda.device(dev):
            return body(torch._C._cuda_getCurrentRawStream(dev))
    if stream.device.index != dev:
        raise ValueError(f"stream must be of cuda:{dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _check(status: int, what: str) -> None:
    if status != sg.OK:
        raise sg.SgemmError(status, what)


def _epilogue(act, bias, ld_bias, residual, ldr, preact, ldp):
    """``Epilogue`` of checked tensors, or None for an empty one."""
    if not act and bias is None and residual is None and preact is None:
        return None
    return Epilogue(act, None if bias is None else bias.data_ptr(), ld_bias,
                    None if residual is None else residual.data_ptr(), ldr,
                    None if preact is None else preact.data_ptr(), ldp)


def _inner(A, B, dev: int, transpose_a, transpose_b):
    """M, N, K and the leading dimensions of op(A) and op(B)."""
    M, K, lda = _matrix(A, "A", dev)
    K2, N, ldb = _matrix(B, "B", dev)
    if transpose_a:
        M, K = K, M
    if transpose_b:
        K2, N = N, K2
    if K2 != K:
        raise ValueError(f"shape mismatch: op(A) is {M} x {K}, op(B) is {K2} x {N}")
    return M, N, K, lda, ldb


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
    act = _act(activation)
    dev = _device(A, "A")
    M, N, K, lda, ldb = _inner(A, B, dev, transpose_a, transpose_b)
    if bias is not None:
        _vector(bias, "bias", dev, N)
    ldr = 1 if residual is None else _sized(residual, "residual", dev, M, N)
    ldp = 1 if preact is None else _sized(preact, "preact", dev, M, N)
    epilogue = _epilogue(act, bias, N, residual, ldr, preact, ldp)
    ws, ws_bytes = _workspace(workspace, dev)
    ldc = max(N, 1) if out is None else _sized(out, "out", dev, M, N)

    def call(s):
        c = A.new_empty(M, N) if out is None else out
        st = sg.load().sgemm_linear(bool(transpose_a), bool(transpose_b), M, N, K, A.data_ptr(),
                                    lda, B.data_ptr(), ldb, c.data_ptr(), ldc, epilogue, s, ws,
                                    ws_bytes)
        _check(st, "sgemm_linear")
        return c
    return _on(dev, stream, call)


def activation_backward(dC, activation="none", preact=None, *, bias_grad=True, out=None,
                        stream=None, workspace=None):
    """``(dZ, dbias)``: ``dZ = dC * act'(preact)`` and its column sums (None
    without ``bias_grad``).

    ``out`` receives dZ and may be ``dC`` or ``preact``.  For activation
    "none" dZ is dC: unless ``out`` asks for a copy, dC itself is returned.
    Without a ``workspace`` one is made for the sums.
    """
    act = _act(activation)
    dev = _device(dC, "dC")
    M, N, lddc = _matrix(dC, "dC", dev)
    z, ldz = 0, 1
    if act:
        if preact is None:
            raise ValueError(f"activation {activation!r} needs preact")
        ldz = _sized(preact, "preact", dev, M, N)
        z = preact.data_ptr()
    lddz = max(N, 1) if out is None else _sized(out, "out", dev, M, N)
    ws, ws_bytes = _workspace(workspace, dev)
    lib = sg.load()
    need = 0
    if workspace is None and bias_grad:
        need = lib.sgemm_act_backward_workspace_bytes(M, N)

    def call(s):
        dz = dC.new_empty(M, N) if out is None and act else out
        dbias = dC.new_empty(N) if bias_grad else None
        own, room, size = _own(dC, need, ws, ws_bytes)  # noqa: F841
        st = lib.sgemm_act_backward(M, N, dC.data_ptr(), lddc, z, ldz, act,
                                    None if dz is None else dz.data_ptr(), lddz,
                                    dbias.data_ptr() if bias_grad else None, s, room, size)
        _check(st, "sgemm_act_backward")
        return (dC if dz is None else dz), dbias
    return _on(dev, stream, call)


def linear_backward(dC, A, B, activation="none", preact=None, *, transpose_a=False,
                    transpose_b=False, bias_grad=True, stream=None, workspace=None):
    """``(dA, dB, dbias)`` of ``linear`` for the gradient ``dC`` of its output:
    dA and dB in the shapes A and B are stored in, dbias None without
    ``bias_grad``.  ``preact`` is what ``linear`` stored (not needed for
    activation "none").  The residual's gradient is ``dC``.  Without a
    ``workspace`` one is made for dbias, and the products' sums are not split.
    """
    act = _act(activation)
    dev = _device(dC, "dC")
    M, N, K, lda, ldb = _inner(A, B, dev, transpose_a, transpose_b)
    lddc, ldz = _sized(dC, "dC", dev, M, N), 1
    if act:
        if preact is None:
            raise ValueError(f"activation {activation!r} needs preact")
        ldz = _sized(preact, "preact", dev, M, N)
    room, size = _workspace(workspace, dev)
    ta, tb = bool(transpose_a), bool(transpose_b)
    lib = sg.load()
    need = 0
    if workspace is None and bias_grad:
        need = lib.sgemm_act_backward_workspace_bytes(M, N)

    def call(s):   # dZ, when it is made here, belongs to the stream
        dz, ld, dbias = dC, lddc, dC.new_empty(N) if bias_grad else None
        if act:
            dz, ld = dC.new_empty(M, N), max(N, 1)
        if act or bias_grad:
            own, *sums = _own(dC, need, room, size)  # noqa: F841
            _check(lib.sgemm_act_backward(
                M, N, dC.data_ptr(), lddc, preact.data_ptr() if act else None, ldz, act,
                dz.data_ptr() if act else None, ld, dbias.data_ptr() if bias_grad else None, s,
                *sums), "sgemm_act_backward")
        dA, dB = A.new_empty(A.shape), B.new_empty(B.shape)
        a, b, d = (A.data_ptr(), lda), (B.data_ptr(), ldb), (dz.data_ptr(), ld)

        def product(out, left, trans_left, right, trans_right, m, n, k):
            _check(lib.sgemm_linear(trans_left, trans_right, m, n, k, *left, *right, out.data_ptr(),
                                    max(n, 1), None, s, room, size), "sgemm_linear")
        # d op(A) = dZ op(B)^T and d op(B) = op(A)^T dZ, transposed where A and B are
        if ta:
            product(dA, b, tb, d, True, K, M, N)
        else:
            product(dA, d, False, b, not tb, M, K, N)
        if tb:
            product(dB, d, True, a, ta, N, K, M)
        else:
            product(dB, a, not ta, d, False, K, N, M)
        return dA, dB, dbias
    return _on(dev, stream, call)
