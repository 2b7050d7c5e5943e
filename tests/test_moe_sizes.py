"""Tensors with more rows or columns than a C int: the binding refuses them, so
that no call sees a size without its upper bits.  No memory is behind them."""

from __future__ import annotations

import pytest

import weight_only_int4_gemm_amd as w4

MANY = (1 << 32) + 4          # 4 in 32 bits


def _meta(shape, dtype):
    import torch
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", ["repack", "quantize", "gemm", "route", "tables", "tables experts",
                                  "w4a16 rows", "w4a16 experts", "w8a8 rows", "combine"])
def test_sizes_beyond_an_int_are_refused(call):
    import torch
    f16, u8, f32, i32 = torch.float16, torch.uint8, torch.float32, torch.int32
    few = {t: _meta((4, 128), t) for t in (f16, u8, f32, i32)}
    many = {t: _meta((MANY, 128), t) for t in (f16, u8, f32, i32)}
    starts, experts = _meta((3,), i32), _meta((MANY + 1,), i32)
    calls = {
        "repack": lambda: w4.w8a8_repack(many[u8], few[u8]),
        "quantize": lambda: w4.w8a8_quantize(many[f16], many[u8], few[f32]),
        "gemm": lambda: w4.w8a8_gemm(many[u8], few[f32], few[u8], few[f32], many[f16]),
        "route": lambda: w4.moe_route(many[f32], None, many[i32], many[f32]),
        "tables": lambda: w4.moe_tables(many[i32], starts, many[i32], many[i32]),
        "tables experts": lambda: w4.moe_tables(few[i32], experts, few[i32], few[i32]),
        "w4a16 rows": lambda: w4.w4a16_moe_gemm(many[f16], None, starts, few[i32], few[f16],
                                                many[f16], 1, 128),
        "w4a16 experts": lambda: w4.w4a16_moe_gemm(few[f16], None, experts, few[i32], few[f16],
                                                   few[f16], 1, 128),
        "w8a8 rows": lambda: w4.w8a8_moe_gemm(many[u8], few[f32], None, starts, few[u8], few[f32],
                                              many[f16], 1),
        "combine": lambda: w4.moe_combine(many[f16], few[i32], few[f32], few[f16]),
    }
    with pytest.raises(ValueError, match="no call takes"):
        calls[call]()
