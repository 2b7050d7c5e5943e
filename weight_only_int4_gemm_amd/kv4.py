"""Python binding of the paged 4-bit key/value cache (include/w4a16_kv4.h).

The functions carry the C interface's names and take torch tensors, whose
shapes and strides give the sizes; as in the package's other functions they
only marshal arguments.  ``stream`` defaults to torch's current stream.

    kv4_tables(lens, want, table, ring, state, lens_out, state_out, q_start,
               slots, positions, page, stream=None)
    kv4_rope(X, Y, positions, inv_freq, sections, pairs=KV4_ROPE_HALVES,
             stream=None)
    kv4_append(K, V, slots, cache, stream=None)
    kv4_rope_append(Q, K, V, Qout, positions, inv_freq, sections, pairs,
                    slots, cache, stream=None)
    kv4_dequant_debug(slots, cache, K, V, stream=None)
    kv4_attention(Q, cache, table, lens, q_start, O, lse, scale, window,
                  max_q, max_len, workspace, stream=None)
    kv4_attention_workspace_bytes(B, Hq, H, D, max_q, max_len, window=0)
    kv4_attention_describe(B, Hq, H, D, max_q, max_len, window=0, cus=0)
    kv4_cache_bytes(pages, heads, D, page)
    kv4_layout_version()

A cache is a uint8 tensor [pages, heads, page, D + 8] (``alloc_kv4_cache``).
"""

from __future__ import annotations

import ctypes
import functools

KV4_ROPE_HALVES = 0
KV4_ROPE_PAIRS = 1
KV4_MAX_REQUESTS = 4096

KV4_EXPORTED_SYMBOLS = (
    "kv4_layout_version", "kv4_cache_bytes", "kv4_tables", "kv4_rope", "kv4_append",
    "kv4_rope_append", "kv4_dequant_debug", "kv4_attention", "kv4_attention_workspace_bytes",
    "kv4_attention_describe",
)

__all__ = [*KV4_EXPORTED_SYMBOLS, "KV4_EXPORTED_SYMBOLS", "KV4_ROPE_HALVES", "KV4_ROPE_PAIRS",
           "KV4_MAX_REQUESTS", "alloc_kv4_cache", "alloc_kv4_pages", "alloc_kv4_workspace"]


def declare(lib) -> None:
    """Declare the signatures of include/w4a16_kv4.h on the loaded library."""
    vp, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    rows = [vp, i64, i64]
    rope = [vp, i64, vp, vp, i, i]
    lib.kv4_layout_version.argtypes = []
    lib.kv4_layout_version.restype = i
    lib.kv4_cache_bytes.argtypes = [i] * 4
    lib.kv4_cache_bytes.restype = sz
    lib.kv4_tables.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp, vp, vp, i, i, i, vp]
    lib.kv4_tables.restype = i
    lib.kv4_rope.argtypes = [*rows, *rows, *rope, i, i, i, i, vp]
    lib.kv4_rope.restype = i
    lib.kv4_append.argtypes = [*rows, *rows, vp, vp, i, i, i, i, i, i, vp]
    lib.kv4_append.restype = i
    lib.kv4_rope_append.argtypes = [*rows, *rows, *rows, *rows, *rope, vp, vp, i, i, i, i, i, i,
                                    i, vp]
    lib.kv4_rope_append.restype = i
    lib.kv4_dequant_debug.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.kv4_dequant_debug.restype = i
    lib.kv4_attention.argtypes = [*rows, vp, vp, i, vp, vp, *rows, vp, i, i, i, i, i, i, i,
                                  ctypes.c_float, i, i, i, i, vp, vp]
    lib.kv4_attention.restype = i
    lib.kv4_attention_workspace_bytes.argtypes = [i] * 7
    lib.kv4_attention_workspace_bytes.restype = sz
    lib.kv4_attention_describe.argtypes = [i] * 8 + [ctypes.c_char_p, sz]
    lib.kv4_attention_describe.restype = i


# Decode steps call these functions once per layer, so a call's own cost
# counts: the library, torch and the package are looked up once, and a call
# asks for the current device once.
_lib = _torch = _pkg = None


def _bind():
    global _lib, _torch, _pkg
    import torch
    import weight_only_int4_gemm_amd as pkg
    _lib, _torch, _pkg = pkg.load(), torch, pkg


def _start():
    """The current device's index (binds the library on the first call)."""
    if _lib is None:
        _bind()
    return _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else -1


def _raw_stream(stream, device):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return _pkg._stream(stream)


def _check(fn, status):
    if status:
        _pkg._check(fn, status)


def _wrong_device(t, what, device):
    if t.device.type != "cuda":
        raise ValueError(f"{what}: must be a device tensor")
    raise ValueError(f"{what}: on {t.device}, but the current device is cuda:{device}")


def _flat(t, dtype, what, numel, device):
    """The address of a contiguous tensor of at least ``numel`` elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{what}: {t.numel()} elements, the call needs {numel}")
    if t.get_device() != device or device < 0:
        _wrong_device(t, what, device)
    return t.data_ptr()


def _dtype(t, what):
    dtype = t.dtype
    if dtype is _torch.float16:
        return dtype, 0
    if dtype is _torch.bfloat16:
        return dtype, 1
    raise TypeError(f"{what}: expected float16 or bfloat16, got {dtype}")


def _rows(t, what, dtype, device, T=None, heads=None, D=None):
    """(pointer, token stride, head stride) of a [T][heads][D] tensor."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{what}: expected [tokens, heads, channels], got {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    n, h, d = shape
    if T is not None and n != T:
        raise ValueError(f"{what}: {n} tokens, expected {T}")
    if heads is not None and h != heads:
        raise ValueError(f"{what}: {h} heads, expected {heads}")
    if D is not None and d != D:
        raise ValueError(f"{what}: {d} channels, expected {D}")
    token, head, channel = t.stride()
    if channel != 1 and d > 1:
        raise ValueError(f"{what}: channels must be contiguous")
    if t.get_device() != device or device < 0:
        _wrong_device(t, what, device)
    # strides of dimensions of one element mean nothing
    return t.data_ptr(), 0 if n == 1 else token, 0 if h == 1 else head


def _cache(t, device):
    """(pointer, pages, heads, D, page) of a cache."""
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"cache: expected [pages, heads, page, D + 8], got {tuple(shape)}")
    pages, heads, page, d8 = shape
    return _flat(t, _torch.uint8, "cache", 0, device), pages, heads, d8 - 8, page


@functools.lru_cache(maxsize=64)
def _sections(sections):
    return (ctypes.c_int * max(1, len(sections)))(*sections), len(sections), sum(sections)


def _rope(positions, inv_freq, sections, T, device):
    """The rotation's arguments up to the section array."""
    sec, axes, half = _sections(tuple(sections))
    if positions.dtype is not _torch.int32:
        raise TypeError(f"positions: expected torch.int32, got {positions.dtype}")
    shape, stride = positions.shape, positions.stride()
    if len(shape) == 1:
        shape, stride = (1, *shape), (0, *stride)
    if len(shape) != 2 or shape[0] != axes or shape[1] < T:
        raise ValueError(f"positions: expected [{axes}, {T}], got {tuple(positions.shape)}")
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError("positions: tokens must be contiguous")
    if positions.get_device() != device or device < 0:
        _wrong_device(positions, "positions", device)
    return (positions.data_ptr(), stride[0] if axes > 1 else 0,
            _flat(inv_freq, _torch.float64, "inv_freq", half, device), sec, axes)


def kv4_layout_version() -> int:
    _start()
    return _lib.kv4_layout_version()


def kv4_cache_bytes(pages: int, heads: int, D: int, page: int) -> int:
    _start()
    return _lib.kv4_cache_bytes(pages, heads, D, page)


def kv4_tables(lens, want, table, ring, state, lens_out, state_out, q_start, slots, positions,
               page: int, stream=None) -> None:
    dev = _start()
    if table.dim() != 2:
        raise ValueError(f"table: expected [requests, pages], got {tuple(table.shape)}")
    B, max_pages = table.shape
    i32 = _torch.int32
    capacity = slots.numel()
    _check("kv4_tables", _lib.kv4_tables(
        _flat(lens, i32, "lens", B, dev), _flat(want, i32, "want", B, dev),
        _flat(table, i32, "table", 0, dev), max_pages, _flat(ring, i32, "ring", 0, dev),
        ring.numel(), _flat(state, i32, "state", 4, dev),
        _flat(lens_out, i32, "lens_out", B, dev), _flat(state_out, i32, "state_out", 4, dev),
        _flat(q_start, i32, "q_start", B + 1, dev), _flat(slots, i32, "slots", 0, dev),
        _flat(positions, i32, "positions", capacity, dev), capacity, B, page,
        _raw_stream(stream, dev)))


def kv4_rope(X, Y, positions, inv_freq, sections, pairs: int = KV4_ROPE_HALVES,
             stream=None) -> None:
    dev = _start()
    dtype, code = _dtype(X, "X")
    x = _rows(X, "X", dtype, dev)
    T, H, D = X.shape
    _check("kv4_rope", _lib.kv4_rope(
        *x, *_rows(Y, "Y", dtype, dev, T, H, D), *_rope(positions, inv_freq, sections, T, dev),
        pairs, T, H, D, code, _raw_stream(stream, dev)))


def kv4_append(K, V, slots, cache, stream=None) -> None:
    dev = _start()
    dtype, code = _dtype(K, "K")
    c, pages, heads, D, page = _cache(cache, dev)
    k = _rows(K, "K", dtype, dev, None, heads, D)
    T = K.shape[0]
    _check("kv4_append", _lib.kv4_append(
        *k, *_rows(V, "V", dtype, dev, T, heads, D), _flat(slots, _torch.int32, "slots", T, dev),
        c, T, heads, D, pages, page, code, _raw_stream(stream, dev)))


def kv4_rope_append(Q, K, V, Qout, positions, inv_freq, sections, pairs: int, slots, cache,
                    stream=None) -> None:
    """``Q`` and ``Qout`` may be None: only keys are rotated."""
    dev = _start()
    dtype, code = _dtype(K, "K")
    c, pages, heads, D, page = _cache(cache, dev)
    k = _rows(K, "K", dtype, dev, None, heads, D)
    T = K.shape[0]
    v = _rows(V, "V", dtype, dev, T, heads, D)
    q, qo, Hq = (None, 0, 0), (None, 0, 0), 0
    if Q is not None:
        q = _rows(Q, "Q", dtype, dev, T, None, D)
        Hq = Q.shape[1]
        qo = _rows(Qout, "Qout", dtype, dev, T, Hq, D)
    _check("kv4_rope_append", _lib.kv4_rope_append(
        *q, *k, *v, *qo, *_rope(positions, inv_freq, sections, T, dev), pairs,
        _flat(slots, _torch.int32, "slots", T, dev), c, T, Hq, heads, D, pages, page, code,
        _raw_stream(stream, dev)))


def kv4_dequant_debug(slots, cache, K, V, stream=None) -> None:
    dev = _start()
    dtype, code = _dtype(K, "K")
    c, pages, heads, D, page = _cache(cache, dev)
    T = K.shape[0]
    for t, what in ((K, "K"), (V, "V")):
        if t.shape != (T, heads, D):
            raise ValueError(f"{what}: expected {(T, heads, D)}, got {tuple(t.shape)}")
    _check("kv4_dequant_debug", _lib.kv4_dequant_debug(
        _flat(slots, _torch.int32, "slots", T, dev), c, _flat(K, dtype, "K", 0, dev),
        _flat(V, dtype, "V", 0, dev), T, heads, D, pages, page, code,
        _raw_stream(stream, dev)))


def kv4_attention_workspace_bytes(B: int, Hq: int, H: int, D: int, max_q: int, max_len: int,
                                  window: int = 0) -> int:
    _start()
    return _lib.kv4_attention_workspace_bytes(B, Hq, H, D, max_q, max_len, window)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(device, *sizes):
    """kv4_attention_workspace_bytes of a device: a number that follows from
    the sizes alone."""
    return _lib.kv4_attention_workspace_bytes(*sizes)


def kv4_attention_describe(B: int, Hq: int, H: int, D: int, max_q: int, max_len: int,
                           window: int = 0, cus: int = 0) -> str:
    _start()
    buf = ctypes.create_string_buffer(256)
    _check("kv4_attention_describe", _lib.kv4_attention_describe(
        B, Hq, H, D, max_q, max_len, window, cus, buf, 256))
    return buf.value.decode()


def kv4_attention(Q, cache, table, lens, q_start, O, lse, scale: float, window: int, max_q: int,
                  max_len: int, workspace=None, stream=None) -> None:
    """``q_start`` None: one query per request; ``lse`` may be None."""
    dev = _start()
    dtype, code = _dtype(Q, "Q")
    c, pages, heads, D, page = _cache(cache, dev)
    q = _rows(Q, "Q", dtype, dev, None, None, D)
    T, Hq, _ = Q.shape
    o = _rows(O, "O", dtype, dev, T, Hq, D)
    if table.dim() != 2:
        raise ValueError(f"table: expected [requests, pages], got {tuple(table.shape)}")
    B, max_pages = table.shape
    if q_start is None and T < B:
        raise ValueError(f"Q: {T} rows for {B} requests")
    i32 = _torch.int32
    ws = None
    if workspace is not None:
        need = _workspace_bytes(dev, B, Hq, heads, D, max_q, max_len, window)
        ws = _flat(workspace, workspace.dtype, "workspace",
                   -(-need // workspace.element_size()), dev)
    _check("kv4_attention", _lib.kv4_attention(
        *q, c, _flat(table, i32, "table", 0, dev), max_pages, _flat(lens, i32, "lens", B, dev),
        None if q_start is None else _flat(q_start, i32, "q_start", B + 1, dev), *o,
        None if lse is None else _flat(lse, _torch.float32, "lse", T * Hq, dev), T, B, Hq, heads,
        D, pages, page, scale, window, max_q, max_len, code, ws, _raw_stream(stream, dev)))


# ---------------------------------------------------------------------------
# allocation conveniences (torch owns the memory; the library allocates none)
# ---------------------------------------------------------------------------

def alloc_kv4_cache(pages: int, heads: int, D: int, page: int, device=None):
    """An uninitialised cache; no result depends on what it holds."""
    import torch
    if kv4_cache_bytes(pages, heads, D, page) == 0:
        raise ValueError(f"no cache has pages={pages} heads={heads} D={D} page={page}")
    return torch.empty((pages, heads, page, D + 8), dtype=torch.uint8, device=device or "cuda")


def alloc_kv4_pages(pages: int, requests: int, max_pages: int, device=None):
    """(table, ring, state) with every page free and every request empty."""
    import torch
    dev = device or "cuda"
    table = torch.full((requests, max_pages), -1, dtype=torch.int32, device=dev)
    ring = torch.arange(pages, dtype=torch.int32, device=dev)
    state = torch.tensor([0, pages, 0, 0], dtype=torch.int32, device=dev)
    return table, ring, state


def alloc_kv4_workspace(B: int, Hq: int, H: int, D: int, max_q: int, max_len: int,
                        window: int = 0, device=None):
    """A zero-filled workspace of ``kv4_attention_workspace_bytes`` bytes, or None."""
    import torch
    nbytes = kv4_attention_workspace_bytes(B, Hq, H, D, max_q, max_len, window)
    if nbytes == 0:
        return None
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")
