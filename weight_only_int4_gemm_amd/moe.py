"""Python binding of the products in 8-bit floating point (include/w8a8.h) and
of the expert layers (include/w4a16_moe.h).

The functions carry the C interface's names and take torch tensors, whose
shapes and strides give the sizes; as in the package's other functions they
only marshal arguments.  ``stream`` defaults to torch's current stream.  e4m3
codes are ``torch.float8_e4m3fn`` or ``torch.uint8``.

    w8a8_repack(B, Bpacked, stream=None)
    w8a8_quantize(X, Xq, Xs, stream=None)
    w8a8_gemm(A, As, Bpacked, Bs, C, workspace=None, stream=None)
    w8a8_packed_bytes(K, N)
    w8a8_workspace_bytes(M, K, N)
    w8a8_describe(M, K, N, cus=0)
    w8a8_layout_version()
    moe_route(logits, bias, ids, weights, score=MOE_SOFTMAX, groups=1,
              top_groups=1, group_best=1, renorm=True, scale=1.0, stream=None)
    moe_tables(ids, starts, order, where, stream=None)
    w4a16_moe_gemm(A, order, starts, Bpacked, scales, C, k, group,
                   activation=MOE_ACT_NONE, stream=None)
    w8a8_moe_gemm(A, As, order, starts, Bpacked, Bs, C, k,
                  activation=MOE_ACT_NONE, stream=None)
    moe_gemm_describe(form, rows, K, N, E, activation=MOE_ACT_NONE, cus=0)
    moe_combine(Y, where, weights, out, stream=None)
"""

from __future__ import annotations

import ctypes
import functools

from . import kv4 as _base
from .kv4 import _check, _dtype, _flat, _raw_stream, _start, _wrong_device

MOE_MAX_EXPERTS = 1024
MOE_MAX_TOP = 32
MOE_MAX_GROUPS = 64
MOE_SOFTMAX = 0
MOE_SIGMOID = 1
MOE_LOGITS_F16 = 0
MOE_LOGITS_BF16 = 1
MOE_LOGITS_F32 = 2
MOE_ACT_NONE = 0
MOE_ACT_SILU_GATE = 1

W8A8_EXPORTED_SYMBOLS = (
    "w8a8_layout_version", "w8a8_packed_bytes", "w8a8_repack", "w8a8_quantize",
    "w8a8_workspace_bytes", "w8a8_describe", "w8a8_gemm",
)
MOE_EXPORTED_SYMBOLS = (
    "moe_route", "moe_tables", "w4a16_moe_gemm", "w8a8_moe_gemm", "moe_gemm_describe",
    "moe_combine",
)

__all__ = [*W8A8_EXPORTED_SYMBOLS, *MOE_EXPORTED_SYMBOLS, "W8A8_EXPORTED_SYMBOLS",
           "MOE_EXPORTED_SYMBOLS", "MOE_MAX_EXPERTS", "MOE_MAX_TOP", "MOE_MAX_GROUPS",
           "MOE_SOFTMAX", "MOE_SIGMOID", "MOE_LOGITS_F16", "MOE_LOGITS_BF16", "MOE_LOGITS_F32",
           "MOE_ACT_NONE", "MOE_ACT_SILU_GATE", "alloc_w8a8_packed", "alloc_w8a8_workspace",
           "alloc_moe_tables"]


def declare(lib) -> None:
    """Declare the signatures of include/w8a8.h and include/w4a16_moe.h."""
    vp, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    f, text = ctypes.c_float, ctypes.c_char_p
    for name, result, args in (
            ("w8a8_layout_version", i, []),
            ("w8a8_packed_bytes", sz, [i, i]),
            ("w8a8_repack", i, [vp, vp, i, i, vp]),
            ("w8a8_quantize", i, [vp, i64, vp, vp, i, i, i, vp]),
            ("w8a8_workspace_bytes", sz, [i, i, i]),
            ("w8a8_describe", i, [i, i, i, i, text, sz]),
            ("w8a8_gemm", i, [vp, vp, vp, vp, vp, i, i, i, i, vp, vp]),
            ("moe_route", i, [vp, i64, i, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp]),
            ("moe_tables", i, [vp, vp, vp, vp, i, i, i, vp]),
            ("w4a16_moe_gemm", i, [vp, i, vp, i, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]),
            ("w8a8_moe_gemm", i, [vp, vp, i, vp, i, vp, vp, vp, vp, i, i, i, i, i, i, vp]),
            ("moe_gemm_describe", i, [i, i, i, i, i, i, i, text, sz]),
            ("moe_combine", i, [vp, i, vp, vp, vp, i, i, i, i, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = result, args


def _lib():
    return _base._lib


def _codes(t, what, numel, device):
    """The address of a contiguous tensor of e4m3 codes."""
    torch = _base._torch
    if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
        raise TypeError(f"{what}: expected float8_e4m3fn or uint8, got {t.dtype}")
    return _flat(t, t.dtype, what, numel, device)


_INT = 2 ** 31 - 1      # sizes travel as C ints, which would lose their upper bits


def _matrix(t, what):
    try:
        rows, cols = t.shape
    except ValueError:
        raise ValueError(f"{what}: expected a matrix, got {tuple(t.shape)}") from None
    if rows > _INT or cols > _INT:
        raise ValueError(f"{what}: no call takes {rows} x {cols}")
    return rows, cols


def _count(starts):
    """Experts of ``starts`` [E + 1]."""
    E = starts.numel() - 1
    if E > _INT:
        raise ValueError(f"starts: no call takes {E} experts")
    return E


def _strided(t, what, device):
    """(pointer, rows, columns, row stride) of a matrix with contiguous rows."""
    rows, cols = _matrix(t, what)
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    if t.get_device() != device or device < 0:
        _wrong_device(t, what, device)
    return t.data_ptr(), rows, cols, row if rows > 1 else cols


def w8a8_layout_version() -> int:
    _start()
    return _lib().w8a8_layout_version()


def w8a8_packed_bytes(K: int, N: int) -> int:
    _start()
    return _lib().w8a8_packed_bytes(K, N)


def w8a8_repack(B, Bpacked, stream=None) -> None:
    """``B`` [N, K]; ``Bpacked`` K * N codes of any shape."""
    dev = _start()
    N, K = _matrix(B, "B")
    _check("w8a8_repack", _lib().w8a8_repack(
        _codes(B, "B", 0, dev), _codes(Bpacked, "Bpacked", K * N, dev), K, N,
        _raw_stream(stream, dev)))


def w8a8_quantize(X, Xq, Xs, stream=None) -> None:
    """``X`` [T, K], rows may be strided; ``Xq`` [T, K]; ``Xs`` [T, K / 128]."""
    dev = _start()
    _, dtype = _dtype(X, "X")
    x, T, K, row = _strided(X, "X", dev)
    _check("w8a8_quantize", _lib().w8a8_quantize(
        x, row, _codes(Xq, "Xq", T * K, dev),
        _flat(Xs, _base._torch.float32, "Xs", T * (K // 128), dev), T, K, dtype,
        _raw_stream(stream, dev)))


def w8a8_workspace_bytes(M: int, K: int, N: int) -> int:
    _start()
    return _lib().w8a8_workspace_bytes(M, K, N)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(device, M, K, N):
    """w8a8_workspace_bytes of a device: a number that follows from the sizes."""
    return _lib().w8a8_workspace_bytes(M, K, N)


def w8a8_describe(M: int, K: int, N: int, cus: int = 0) -> str:
    _start()
    buf = ctypes.create_string_buffer(256)
    _check("w8a8_describe", _lib().w8a8_describe(M, K, N, cus, buf, 256))
    return buf.value.decode()


def w8a8_gemm(A, As, Bpacked, Bs, C, workspace=None, stream=None) -> None:
    """``A`` [M, K]; ``As`` [M, K / 128]; ``Bs`` [ceil(N / 128), K / 128]; ``C`` [M, N]."""
    dev = _start()
    M, K = _matrix(A, "A")
    rows, N = _matrix(C, "C")
    if rows != M:
        raise ValueError(f"C: {rows} rows, expected {M}")
    out, dtype = _dtype(C, "C")
    f32, KB = _base._torch.float32, K // 128
    ws = None
    if workspace is not None:
        ws = _flat(workspace, workspace.dtype, "workspace",
                   -(-_workspace_bytes(dev, M, K, N) // workspace.element_size()), dev)
    _check("w8a8_gemm", _lib().w8a8_gemm(
        _codes(A, "A", 0, dev), _flat(As, f32, "As", M * KB, dev),
        _codes(Bpacked, "Bpacked", K * N, dev), _flat(Bs, f32, "Bs", -(-N // 128) * KB, dev),
        _flat(C, out, "C", 0, dev), M, K, N, dtype, ws, _raw_stream(stream, dev)))


def moe_route(logits, bias, ids, weights, score: int = MOE_SOFTMAX, groups: int = 1,
              top_groups: int = 1, group_best: int = 1, renorm: bool = True, scale: float = 1.0,
              stream=None) -> None:
    """``logits`` [T, E], rows may be strided; ``bias`` [E] or None; ``ids``
    and ``weights`` [T, k]."""
    dev = _start()
    torch = _base._torch
    x, T, E, row = _strided(logits, "logits", dev)
    if logits.dtype is torch.float32:
        kind = MOE_LOGITS_F32
    elif logits.dtype is torch.float16:
        kind = MOE_LOGITS_F16
    elif logits.dtype is torch.bfloat16:
        kind = MOE_LOGITS_BF16
    else:
        raise TypeError(f"logits: expected float32, float16 or bfloat16, got {logits.dtype}")
    tokens, k = _matrix(ids, "ids")
    if tokens != T:
        raise ValueError(f"ids: {tokens} tokens, expected {T}")
    _check("moe_route", _lib().moe_route(
        x, row, kind, None if bias is None else _flat(bias, torch.float32, "bias", E, dev),
        _flat(ids, torch.int32, "ids", 0, dev),
        _flat(weights, torch.float32, "weights", T * k, dev), T, E, k, score, groups, top_groups,
        group_best, int(renorm), scale, _raw_stream(stream, dev)))


def moe_tables(ids, starts, order, where, stream=None) -> None:
    """``ids`` and ``where`` [T, k]; ``starts`` [E + 1]; ``order`` [T * k]."""
    dev = _start()
    i32 = _base._torch.int32
    T, k = _matrix(ids, "ids")
    E = _count(starts)
    _check("moe_tables", _lib().moe_tables(
        _flat(ids, i32, "ids", 0, dev), _flat(starts, i32, "starts", 2, dev),
        _flat(order, i32, "order", T * k, dev), _flat(where, i32, "where", T * k, dev), T, k, E,
        _raw_stream(stream, dev)))


def _experts(A, order, starts, C, activation, device):
    """Sizes and index tensors that both expert products take."""
    i32 = _base._torch.int32
    a_rows, K = _matrix(A, "A")
    rows, N = _matrix(C, "C")
    E = _count(starts)
    if order is None and a_rows < rows:
        raise ValueError(f"A: {a_rows} rows for {rows} rows of C")
    return (a_rows, K, rows, N, E, N * (2 if activation == MOE_ACT_SILU_GATE else 1),
            None if order is None else _flat(order, i32, "order", rows, device),
            _flat(starts, i32, "starts", 2, device))


def w4a16_moe_gemm(A, order, starts, Bpacked, scales, C, k: int, group: int,
                   activation: int = MOE_ACT_NONE, stream=None) -> None:
    """``A`` [a_rows, K]; ``order`` [rows] or None; ``starts`` [E + 1];
    ``Bpacked`` E packed matrices; ``scales`` [E, K / group, W]; ``C`` [rows, N]."""
    dev = _start()
    dtype, code = _dtype(A, "A")
    a_rows, K, rows, N, E, W, o, s = _experts(A, order, starts, C, activation, dev)
    groups = K // group if group > 0 else 0
    _check("w4a16_moe_gemm", _lib().w4a16_moe_gemm(
        _flat(A, dtype, "A", 0, dev), a_rows, o, k, s,
        _flat(Bpacked, _base._torch.int32, "Bpacked", E * (K * W // 8), dev),
        _flat(scales, dtype, "scales", E * groups * W, dev), _flat(C, dtype, "C", 0, dev), rows,
        K, N, group, E, activation, code, _raw_stream(stream, dev)))


def w8a8_moe_gemm(A, As, order, starts, Bpacked, Bs, C, k: int, activation: int = MOE_ACT_NONE,
                  stream=None) -> None:
    """``A`` [a_rows, K]; ``As`` [a_rows, K / 128]; ``order`` [rows] or None;
    ``starts`` [E + 1]; ``Bpacked`` E packed matrices; ``Bs`` [E, ceil(W / 128),
    K / 128]; ``C`` [rows, N]."""
    dev = _start()
    dtype, code = _dtype(C, "C")
    a_rows, K, rows, N, E, W, o, s = _experts(A, order, starts, C, activation, dev)
    f32, KB = _base._torch.float32, K // 128
    _check("w8a8_moe_gemm", _lib().w8a8_moe_gemm(
        _codes(A, "A", 0, dev), _flat(As, f32, "As", a_rows * KB, dev), a_rows, o, k, s,
        _codes(Bpacked, "Bpacked", E * K * W, dev),
        _flat(Bs, f32, "Bs", E * -(-W // 128) * KB, dev), _flat(C, dtype, "C", 0, dev), rows, K,
        N, E, activation, code, _raw_stream(stream, dev)))


def moe_gemm_describe(form: int, rows: int, K: int, N: int, E: int,
                      activation: int = MOE_ACT_NONE, cus: int = 0) -> str:
    """``form`` 4: w4a16_moe_gemm, 8: w8a8_moe_gemm."""
    _start()
    buf = ctypes.create_string_buffer(256)
    _check("moe_gemm_describe", _lib().moe_gemm_describe(form, rows, K, N, E, activation, cus,
                                                         buf, 256))
    return buf.value.decode()


def moe_combine(Y, where, weights, out, stream=None) -> None:
    """``Y`` [rows, N]; ``where`` and ``weights`` [T, k]; ``out`` [T, N]."""
    dev = _start()
    dtype, code = _dtype(out, "out")
    rows, cols = _matrix(Y, "Y")
    T, N = _matrix(out, "out")
    tokens, k = _matrix(where, "where")
    if cols != N or tokens != T:
        raise ValueError(f"Y {tuple(Y.shape)} and where {tuple(where.shape)} do not fit "
                         f"out {tuple(out.shape)}")
    _check("moe_combine", _lib().moe_combine(
        _flat(Y, dtype, "Y", 0, dev), rows, _flat(where, _base._torch.int32, "where", 0, dev),
        _flat(weights, _base._torch.float32, "weights", T * k, dev),
        _flat(out, dtype, "out", 0, dev), T, k, N, code, _raw_stream(stream, dev)))


# ---------------------------------------------------------------------------
# allocation conveniences (torch owns the memory; the library allocates none)
# ---------------------------------------------------------------------------

def alloc_w8a8_packed(K: int, N: int, experts: int = 1, device=None):
    """Room for the packed weights of ``experts`` matrices, [experts, K * N]."""
    import torch
    if w8a8_packed_bytes(K, N) == 0:
        raise ValueError(f"no packed weights have K={K} N={N}")
    return torch.empty((experts, K * N), dtype=torch.float8_e4m3fn, device=device or "cuda")


def alloc_w8a8_workspace(M: int, K: int, N: int, device=None):
    """A zero-filled workspace of ``w8a8_workspace_bytes`` bytes, or None."""
    import torch
    nbytes = w8a8_workspace_bytes(M, K, N)
    if nbytes == 0:
        return None
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def alloc_moe_tables(T: int, k: int, E: int, device=None):
    """(starts, order, where) for ``moe_tables``, uninitialised."""
    import torch
    dev = device or "cuda"
    return (torch.empty(E + 1, dtype=torch.int32, device=dev),
            torch.empty(T * k, dtype=torch.int32, device=dev),
            torch.empty((T, k), dtype=torch.int32, device=dev))
