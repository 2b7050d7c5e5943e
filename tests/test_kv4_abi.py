"""The C interface of the 4-bit key/value cache on the CPU: exports, sizes,
plans, and every refusal before anything touches a device."""

from __future__ import annotations

import ctypes
import os
import re

import pytest

import weight_only_int4_gemm_amd as w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w4a16_kv4.h")

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, DTYPE = 0, -1, -2, -4, -5, -7, -9

# Fake, 16-byte aligned addresses far apart: the checks return before any of
# them is dereferenced or handed to the runtime.
A = [0x100000000000 + i * 0x10000000000 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    return w4.load()


def _sections(*n):
    return (ctypes.c_int * max(1, len(n)))(*n)


def test_header_binding_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kv4_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(w4.KV4_EXPORTED_SYMBOLS)
    for name in names:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr) and callable(getattr(w4, name))
    for name in ("KV4_ROPE_HALVES", "KV4_ROPE_PAIRS"):
        assert int(re.search(name + r"\s*=\s*(\d+)", text).group(1)) == getattr(w4, name)
    assert int(re.search(r"KV4_MAX_REQUESTS\s+(\d+)", text).group(1)) == w4.KV4_MAX_REQUESTS
    assert w4.kv4_layout_version() == 1


def test_cache_bytes():
    assert w4.kv4_cache_bytes(10, 8, 128, 64) == 10 * 8 * 64 * 136
    assert w4.kv4_cache_bytes(100000, 32, 256, 64) == 100000 * 32 * 64 * 264
    for bad in ((0, 8, 128, 64), (1, 0, 128, 64), (1, 8, 96, 64), (1, 8, 128, 48),
                (1, 8, 128, 8), (1, 8, 128, 2048), (1 << 26, 1, 64, 32), (-1, 1, 64, 32)):
        assert w4.kv4_cache_bytes(*bad) == 0, bad


TABLES = dict(lens=A[0], want=A[1], table=A[2], max_pages=8, ring=A[3], pages=100, state=A[4],
              lens_out=A[5], state_out=A[6], q_start=A[7], slots=A[8], positions=A[9],
              capacity=64, B=4, page=16, stream=None)


def _refused(call, base, expect, **change):
    args = {**base, **change}
    assert call(*args.values()) == expect, change


def test_tables_refusals(lib):
    def no(expect, **change):
        _refused(lib.kv4_tables, TABLES, expect, **change)
    for k in ("lens", "want", "table", "ring", "state", "lens_out", "state_out", "q_start",
              "slots", "positions"):
        no(NULL, **{k: None})
        no(ALIGN, **{k: TABLES[k] + 2})
    for bad in (dict(B=-1), dict(B=4097), dict(capacity=-1), dict(pages=0), dict(max_pages=0),
                dict(page=0), dict(page=24), dict(page=2048), dict(pages=1 << 28),
                dict(max_pages=1 << 27)):
        no(SHAPE, **bad)
    no(SHAPE, slots=A[9] + 4)                 # overlaps positions
    no(SHAPE, q_start=A[2] + 64)              # overlaps the table
    no(SHAPE, lens_out=A[1])                  # want may not be overwritten
    no(SHAPE, lens_out=A[0] + 4)              # lens itself only whole
    no(SHAPE, state_out=A[4] + 4)


ROPE = dict(X=A[0], x_token=512, x_head=128, Y=A[1], y_token=512, y_head=128, positions=A[2],
            pos_stride=10, inv_freq=A[3], sections=_sections(16, 24, 24), axes=3, pairs=0, T=10,
            H=4, D=128, dtype=0, stream=None)


def test_rope_refusals(lib):
    def no(expect, **change):
        _refused(lib.kv4_rope, ROPE, expect, **change)
    for k in ("X", "Y", "positions", "inv_freq", "sections"):
        no(NULL, **{k: None})
    for k, by in (("X", 8), ("Y", 2), ("positions", 2), ("inv_freq", 4)):
        no(ALIGN, **{k: ROPE[k] + by})
    for k in ("x_token", "x_head", "y_token", "y_head"):
        no(ALIGN, **{k: ROPE[k] + 4})
        no(SHAPE, **{k: -128})
        no(SHAPE, **{k: 1 << 40})
    no(DTYPE, dtype=2)
    no(DTYPE, dtype=-1)
    for bad in (dict(D=96), dict(T=-1), dict(H=-1), dict(axes=0), dict(axes=4), dict(pairs=2),
                dict(pairs=-1), dict(sections=_sections(64, 64, 64)),
                dict(sections=_sections(0, 0, 0)), dict(sections=_sections(-8, 40, 32)),
                dict(sections=_sections(16, 20, 24)), dict(y_head=64), dict(y_token=256),
                dict(pos_stride=-1),
                dict(Y=A[0] + 256),            # shifted onto X
                dict(Y=A[0], y_token=1024)):   # the same memory, other strides
        no(SHAPE, **bad)
    assert lib.kv4_rope(*{**ROPE, "T": 0, "X": None}.values()) == OK
    assert lib.kv4_rope(*{**ROPE, "H": 0, "X": None}.values()) == OK


APPEND = dict(K=A[0], k_token=512, k_head=128, V=A[1], v_token=512, v_head=128, slots=A[2],
              cache=A[3], T=10, H=4, D=128, pages=100, page=16, dtype=0, stream=None)


def test_append_refusals(lib):
    def no(expect, **change):
        _refused(lib.kv4_append, APPEND, expect, **change)
    for k in ("K", "V", "slots", "cache"):
        no(NULL, **{k: None})
    for k, by in (("K", 8), ("V", 2), ("slots", 2), ("cache", 8)):
        no(ALIGN, **{k: APPEND[k] + by})
    for bad in (dict(D=32), dict(D=512), dict(T=-1), dict(H=0), dict(pages=0), dict(page=20),
                dict(page=8), dict(pages=1 << 30), dict(k_token=-512),
                dict(K=A[3] + 1024), dict(V=A[3] + 1024), dict(slots=A[3])):
        no(SHAPE, **bad)
    no(ALIGN, v_token=516)
    no(DTYPE, dtype=3)
    assert lib.kv4_append(*{**APPEND, "T": 0, "K": None}.values()) == OK


# q, k and v as parts of one fused buffer [T][8 + 2 + 2 heads][128]
FUSED = dict(Q=A[0], q_token=1536, q_head=128, K=A[0] + 2048, k_token=1536, k_head=128,
             V=A[0] + 2560, v_token=1536, v_head=128, Qout=A[1], qo_token=1024, qo_head=128,
             positions=A[2], pos_stride=0, inv_freq=A[3], sections=_sections(64), axes=1,
             pairs=0, slots=A[4], cache=A[5], T=10, Hq=8, H=2, D=128, pages=100, page=16,
             dtype=1, stream=None)


def test_rope_append_refusals(lib):
    def no(expect, **change):
        _refused(lib.kv4_rope_append, FUSED, expect, **change)
    for k in ("Q", "K", "V", "Qout", "positions", "inv_freq", "sections", "slots", "cache"):
        no(NULL, **{k: None})
    no(DTYPE, dtype=2)
    for bad in (dict(Hq=-1), dict(Hq=65536), dict(T=-1), dict(axes=0), dict(pairs=5),
                dict(Qout=A[0] + 2048, qo_token=1536),  # over the keys
                dict(Qout=A[0] + 16, qo_token=1536),    # shifted onto the queries
                dict(Qout=A[5]), dict(Q=A[5] + 16, q_token=1024)):
        no(SHAPE, **bad)
    # in place, and a fourth part of the same rows: past the overlap checks,
    # to the first look at the device
    import torch
    if not torch.cuda.is_available():
        no(DEVICE, Qout=A[0], qo_token=1536)
        no(DEVICE, q_token=2560, k_token=2560, v_token=2560, qo_token=2560, Qout=A[0] + 3072)
        no(DEVICE, Q=None, Qout=None, Hq=0)


def test_dequant_refusals(lib):
    base = dict(slots=A[0], cache=A[1], K=A[2], V=A[3], T=4, H=2, D=64, pages=10, page=16,
                dtype=0, stream=None)

    def no(expect, **change):
        _refused(lib.kv4_dequant_debug, base, expect, **change)
    for k in ("slots", "cache", "K", "V"):
        no(NULL, **{k: None})
        no(ALIGN, **{k: base[k] + 2})
    for bad in (dict(T=-1), dict(D=80), dict(H=0), dict(K=A[3]), dict(K=A[1] + 64)):
        no(SHAPE, **bad)
    no(DTYPE, dtype=9)
    assert lib.kv4_dequant_debug(*{**base, "T": 0, "K": None}.values()) == OK


ATTEND = dict(Q=A[0], q_token=1024, q_head=128, cache=A[1], table=A[2], max_pages=8, lens=A[3],
              q_start=A[4], O=A[5], o_token=1024, o_head=128, lse=A[6], T=6, B=3, Hq=8, H=2,
              D=128, pages=100, page=16, scale=0.1, window=0, max_q=4, max_len=128, dtype=0,
              workspace=A[7], stream=None)


def test_attention_refusals(lib):
    def no(expect, **change):
        _refused(lib.kv4_attention, ATTEND, expect, **change)
    for k in ("Q", "cache", "table", "lens", "O"):
        no(NULL, **{k: None})
    for k, by in (("Q", 8), ("O", 8), ("cache", 8), ("table", 2), ("lens", 1), ("q_start", 2),
                  ("lse", 2)):
        no(ALIGN, **{k: ATTEND[k] + by})
    no(ALIGN, q_head=132)
    no(DTYPE, dtype=2)
    for bad in (dict(B=-1), dict(Hq=0), dict(Hq=9), dict(H=0), dict(H=3), dict(D=32),
                dict(T=-1), dict(pages=0), dict(page=40), dict(max_pages=0), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(window=-1), dict(max_q=-1), dict(max_len=-1), dict(max_q=1 << 30),
                dict(max_pages=1 << 28), dict(o_head=64), dict(o_token=512),
                dict(O=A[0]), dict(O=A[1] + 4096), dict(lse=A[5] + 64), dict(lse=A[4])):
        no(SHAPE, **bad)
    for empty in (dict(T=0), dict(B=0), dict(max_q=0)):
        assert lib.kv4_attention(*{**ATTEND, **empty, "Q": None}.values()) == OK
    assert w4.kv4_attention_workspace_bytes(0, 8, 2, 128, 4, 128) == 0
    assert w4.kv4_attention_workspace_bytes(1, 9, 2, 128, 4, 128) == 0


def test_attention_plans():
    def plan(*a, window=0, cus=256):
        d = w4.kv4_attention_describe(*a, window, cus)
        return d, {k: int(v) for k, v in re.findall(r"(\w+)=(\d+)", d)}
    # a lone short request and a lone long one are split, a full batch is not
    d, p = plan(1, 32, 32, 128, 1, 1000)
    assert "tokens" in d and p["splits"] > 1 and p["workspace"] > 0
    d, p = plan(1, 64, 8, 128, 1, 131072)
    assert p["splits"] * 8 >= 256
    d, p = plan(64, 32, 32, 128, 1, 4096)
    assert p["splits"] == 1 and p["workspace"] == 0
    # prefill: waves take rows
    d, p = plan(2, 64, 8, 128, 2048, 8192)
    assert "rows" in d and p["splits"] == 1
    # chunks cover the planned length, and the workspace stays bounded
    for B in (1, 2, 7, 64, 4096):
        for Hq, H in ((1, 1), (8, 1), (28, 4), (32, 32), (128, 1)):
            for D in (64, 128, 256):
                for q in (1, 3, 17, 400):
                    for n in (0, 1, 31, 1000, 100000):
                        for w in (0, 512):
                            _, p = plan(B, Hq, H, D, q, n, window=w)
                            keys = min(n, w + q) if w else n
                            assert p["splits"] * p["chunk"] >= keys
                            assert p["chunk"] % 32 == 0
                            assert p["workspace"] <= 192 << 20
    with pytest.raises(w4.W4A16Error):
        w4.kv4_attention_describe(1, 9, 2, 128, 1, 10, 0, 256)
    with pytest.raises(w4.W4A16Error):
        w4.kv4_attention_describe(0, 8, 2, 128, 1, 10, 0, 256)


def test_binding_refuses_wrong_tensors():
    """Types, shapes and devices, before any pointer reaches the library."""
    import torch
    h = torch.zeros((4, 2, 64), dtype=torch.float16)
    cache = torch.zeros((3, 2, 16, 72), dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        w4.kv4_append(h, h, slots, cache)
    with pytest.raises(TypeError):
        w4.kv4_append(h.float(), h, slots, cache)
    with pytest.raises(ValueError, match="expected"):
        w4.kv4_append(h, h, slots, cache[0])
    with pytest.raises(ValueError, match="no cache"):
        w4.alloc_kv4_cache(3, 2, 65, 16, device="cpu")
    with pytest.raises(ValueError, match="table"):
        z = torch.zeros(4, dtype=torch.int32)
        w4.kv4_tables(z, z, z, z, z, z, z, z, z, z, 16)
