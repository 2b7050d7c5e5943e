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


def _w4():
    import weight_only_int4_gemm_amd as w4
    return w4


def _on_device(t, what):
    import torch
    if t.device.type != "cuda":
        raise ValueError(f"{what}: must be a device tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what}: on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _flat(t, dtype, what, numel):
    """A contiguous tensor of at least ``numel`` elements."""
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{what}: {t.numel()} elements, the call needs {numel}")
    _on_device(t, what)
    return t.data_ptr()


def _dtype(t, what):
    import torch
    if t.dtype == torch.float16:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    raise TypeError(f"{what}: expected float16 or bfloat16, got {t.dtype}")


def _rows(t, what, dtype, T=None, heads=None, D=None):
    """(pointer, token stride, head stride) of a [T][heads][D] tensor."""
    if t.dim() != 3:
        raise ValueError(f"{what}: expected [tokens, heads, channels], got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    for n, m, name in ((t.shape[0], T, "tokens"), (t.shape[1], heads, "heads"),
                       (t.shape[2], D, "channels")):
        if m is not None and n != m:
            raise ValueError(f"{what}: {n} {name}, expected {m}")
    token, head, channel = t.stride()
    if channel != 1 and t.shape[2] > 1:
        raise ValueError(f"{what}: channels must be contiguous")
    _on_device(t, what)
    # strides of dimensions of one element mean nothing
    if t.shape[0] == 1:
        token = 0
    if t.shape[1] == 1:
        head = 0
    return t.data_ptr(), token, head


def _cache(t):
    """(pointer, pages, heads, D, page) of a cache."""
    import torch
    if t.dim() != 4:
        raise ValueError(f"cache: expected [pages, heads, page, D + 8], got {tuple(t.shape)}")
    pages, heads, page, d8 = t.shape
    return _flat(t, torch.uint8, "cache", 0), pages, heads, d8 - 8, page


def _rope(positions, inv_freq, sections, T):
    """The six rotation arguments, and the section array to keep alive."""
    import torch
    axes = len(sections)
    sec = (ctypes.c_int * max(1, axes))(*(int(n) for n in sections))
    if positions.dtype != torch.int32:
        raise TypeError(f"positions: expected torch.int32, got {positions.dtype}")
    if positions.dim() == 1:
        positions = positions[None]
    if positions.dim() != 2 or positions.shape[0] != axes or positions.shape[1] < T:
        raise ValueError(f"positions: expected [{axes}, {T}], got {tuple(positions.shape)}")
    if positions.shape[1] > 1 and positions.stride(1) != 1:
        raise ValueError("positions: tokens must be contiguous")
    _on_device(positions, "positions")
    stride = positions.stride(0) if axes > 1 else 0
    freq = _flat(inv_freq, torch.float64, "inv_freq", sum(int(n) for n in sections))
    return positions.data_ptr(), stride, freq, sec


def kv4_layout_version() -> int:
    return _w4().load().kv4_layout_version()


def kv4_cache_bytes(pages: int, heads: int, D: int, page: int) -> int:
    return _w4().load().kv4_cache_bytes(int(pages), int(heads), int(D), int(page))


def kv4_tables(lens, want, table, ring, state, lens_out, state_out, q_start, slots, positions,
               page: int, stream=None) -> None:
    import torch
    w4 = _w4()
    if table.dim() != 2:
        raise ValueError(f"table: expected [requests, pages], got {tuple(table.shape)}")
    B, max_pages = table.shape
    i32 = torch.int32
    capacity = slots.numel()
    w4._check("kv4_tables", w4.load().kv4_tables(
        _flat(lens, i32, "lens", B), _flat(want, i32, "want", B),
        _flat(table, i32, "table", 0), max_pages, _flat(ring, i32, "ring", 0), ring.numel(),
        _flat(state, i32, "state", 4), _flat(lens_out, i32, "lens_out", B),
        _flat(state_out, i32, "state_out", 4), _flat(q_start, i32, "q_start", B + 1),
        _flat(slots, i32, "slots", 0), _flat(positions, i32, "positions", capacity), capacity,
        B, int(page), w4._stream(stream)))


def kv4_rope(X, Y, positions, inv_freq, sections, pairs: int = KV4_ROPE_HALVES,
             stream=None) -> None:
    w4 = _w4()
    dtype = _dtype(X, "X")
    x = _rows(X, "X", X.dtype)
    T, H, D = X.shape
    y = _rows(Y, "Y", X.dtype, T, H, D)
    pos, stride, freq, sec = _rope(positions, inv_freq, sections, T)
    w4._check("kv4_rope", w4.load().kv4_rope(*x, *y, pos, stride, freq, sec, len(sections),
                                             int(pairs), T, H, D, dtype, w4._stream(stream)))


def kv4_append(K, V, slots, cache, stream=None) -> None:
    import torch
    w4 = _w4()
    dtype = _dtype(K, "K")
    c, pages, heads, D, page = _cache(cache)
    k = _rows(K, "K", K.dtype, None, heads, D)
    T = K.shape[0]
    v = _rows(V, "V", K.dtype, T, heads, D)
    w4._check("kv4_append", w4.load().kv4_append(
        *k, *v, _flat(slots, torch.int32, "slots", T), c, T, heads, D, pages, page, dtype,
        w4._stream(stream)))


def kv4_rope_append(Q, K, V, Qout, positions, inv_freq, sections, pairs: int, slots, cache,
                    stream=None) -> None:
    """``Q`` and ``Qout`` may be None: only keys are rotated."""
    import torch
    w4 = _w4()
    dtype = _dtype(K, "K")
    c, pages, heads, D, page = _cache(cache)
    k = _rows(K, "K", K.dtype, None, heads, D)
    T = K.shape[0]
    v = _rows(V, "V", K.dtype, T, heads, D)
    q, qo, Hq = (None, 0, 0), (None, 0, 0), 0
    if Q is not None:
        q = _rows(Q, "Q", K.dtype, T, None, D)
        Hq = Q.shape[1]
        qo = _rows(Qout, "Qout", K.dtype, T, Hq, D)
    pos, stride, freq, sec = _rope(positions, inv_freq, sections, T)
    w4._check("kv4_rope_append", w4.load().kv4_rope_append(
        *q, *k, *v, *qo, pos, stride, freq, sec, len(sections), int(pairs),
        _flat(slots, torch.int32, "slots", T), c, T, Hq, heads, D, pages, page, dtype,
        w4._stream(stream)))


def kv4_dequant_debug(slots, cache, K, V, stream=None) -> None:
    import torch
    w4 = _w4()
    dtype = _dtype(K, "K")
    c, pages, heads, D, page = _cache(cache)
    T = K.shape[0]
    for t, what in ((K, "K"), (V, "V")):
        if tuple(t.shape) != (T, heads, D):
            raise ValueError(f"{what}: expected {(T, heads, D)}, got {tuple(t.shape)}")
    w4._check("kv4_dequant_debug", w4.load().kv4_dequant_debug(
        _flat(slots, torch.int32, "slots", T), c, _flat(K, K.dtype, "K", 0),
        _flat(V, K.dtype, "V", 0), T, heads, D, pages, page, dtype, w4._stream(stream)))


def kv4_attention_workspace_bytes(B: int, Hq: int, H: int, D: int, max_q: int, max_len: int,
                                  window: int = 0) -> int:
    return _w4().load().kv4_attention_workspace_bytes(int(B), int(Hq), int(H), int(D),
                                                      int(max_q), int(max_len), int(window))


def kv4_attention_describe(B: int, Hq: int, H: int, D: int, max_q: int, max_len: int,
                           window: int = 0, cus: int = 0) -> str:
    w4 = _w4()
    buf = ctypes.create_string_buffer(256)
    w4._check("kv4_attention_describe", w4.load().kv4_attention_describe(
        int(B), int(Hq), int(H), int(D), int(max_q), int(max_len), int(window), int(cus), buf,
        256))
    return buf.value.decode()


def kv4_attention(Q, cache, table, lens, q_start, O, lse, scale: float, window: int, max_q: int,
                  max_len: int, workspace=None, stream=None) -> None:
    """``q_start`` None: one query per request; ``lse`` may be None."""
    import torch
    w4 = _w4()
    dtype = _dtype(Q, "Q")
    c, pages, heads, D, page = _cache(cache)
    q = _rows(Q, "Q", Q.dtype, None, None, D)
    T, Hq, _ = Q.shape
    o = _rows(O, "O", Q.dtype, T, Hq, D)
    if table.dim() != 2:
        raise ValueError(f"table: expected [requests, pages], got {tuple(table.shape)}")
    B, max_pages = table.shape
    if q_start is None and T < B:
        raise ValueError(f"Q: {T} rows for {B} requests")
    i32 = torch.int32
    ws = None
    if workspace is not None:
        need = kv4_attention_workspace_bytes(B, Hq, heads, D, max_q, max_len, window)
        ws = _flat(workspace, workspace.dtype, "workspace",
                   -(-need // workspace.element_size()))
    w4._check("kv4_attention", w4.load().kv4_attention(
        *q, c, _flat(table, i32, "table", 0), max_pages, _flat(lens, i32, "lens", B),
        None if q_start is None else _flat(q_start, i32, "q_start", B + 1), *o,
        None if lse is None else _flat(lse, torch.float32, "lse", T * Hq), T, B, Hq, heads, D,
        pages, page, float(scale), int(window), int(max_q), int(max_len), dtype, ws,
        w4._stream(stream)))


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
