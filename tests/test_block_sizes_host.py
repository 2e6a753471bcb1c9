"""Sizes that a 32-bit argument cannot hold (no GPU needed: meta tensors have
shapes and no memory).  Wrapped around, they would pass for small ones."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import _binding as B

WRAP = 1 << 32


def meta(*shape, dt=torch.bfloat16):
    return torch.empty(shape, dtype=dt, device="meta")


def f32(*shape):
    return meta(*shape, dt=torch.float32)


def i32(*shape):
    return meta(*shape, dt=torch.int32)


BIG = WRAP + 16
CALLS = {
    "x of grouped_mm": lambda: moe.moe_grouped_mm(meta(BIG, 16), meta(2, 16, 16), i32(3),
                                                  meta(16, 16), i32(16)),
    "y of grouped_mm": lambda: moe.moe_grouped_mm(meta(16, 16), meta(2, 16, 16), i32(3),
                                                  meta(BIG, 16), i32(BIG)),
    "experts": lambda: moe.moe_grouped_mm(meta(16, 16), meta(WRAP + 2, 16, 16), i32(WRAP + 3),
                                          meta(16, 16)),
    "rows_div": lambda: moe.moe_grouped_mm(meta(16, 16), meta(2, 16, 16), i32(3), meta(16, 16),
                                           i32(16), WRAP + 1),
    "grouped_mm_dx": lambda: moe.moe_grouped_mm_dx(meta(BIG, 16), meta(2, 16, 16), i32(3),
                                                   meta(BIG, 16)),
    "grouped_mm_dw": lambda: moe.moe_grouped_mm_dw(meta(BIG, 16), meta(BIG, 16), i32(3),
                                                   f32(2, 16, 16)),
    "rows_div of dw": lambda: moe.moe_grouped_mm_dw(meta(16, 16), meta(16, 16), i32(3),
                                                    f32(2, 16, 16), None, i32(16), 1 - WRAP),
    "quantize": lambda: moe.moe_blockscale_quantize(
        meta(BIG, 16), 1, meta(BIG, 16, dt=torch.uint8), f32(BIG, 1)),
    "quantize matrices": lambda: moe.moe_blockscale_quantize(
        meta(WRAP + 1, 8, 16), 128, meta(WRAP + 1, 8, 16, dt=torch.uint8), f32(WRAP + 1, 1, 1)),
    "block_rows": lambda: moe.moe_blockscale_quantize(
        meta(256, 16), WRAP + 1, meta(256, 16, dt=torch.uint8), f32(2, 1)),
    "blockscale_mm": lambda: moe.moe_blockscale_mm(
        meta(BIG, 16, dt=torch.uint8), f32(BIG, 1), meta(2, 16, 16, dt=torch.uint8), f32(2, 1, 1),
        i32(3), meta(BIG, 16)),
    "swiglu": lambda: moe.moe_swiglu(meta(BIG, 32), meta(BIG, 16)),
    "swiglu_quantize": lambda: moe.moe_swiglu_quantize(
        meta(BIG, 32), meta(BIG, 16, dt=torch.uint8), f32(BIG, 1)),
    "swiglu_grad": lambda: moe.moe_swiglu_grad(meta(BIG, 32), meta(BIG, 16), meta(BIG, 32)),
    "combine_grad": lambda: moe.moe_combine_grad(
        (64, 64, 8, 1, 64, 0), meta(BIG, 64), meta(BIG, 64), i32(BIG), f32(BIG, 1), meta(BIG, 64),
        f32(BIG, 1)),
    "block_norm": lambda: moe.moe_block_norm(meta(BIG, 16), None, meta(BIG, 16), None),
    "block_norm gate": lambda: moe.moe_block_norm(meta(1, 16), None, meta(1, 16), None,
                                                  gate=meta(WRAP + 1, 16)),
    "block_norm_grad": lambda: moe.moe_block_norm_grad(
        meta(BIG, 16), None, meta(BIG, 16), None, meta(BIG, 16), None, None, None, None),
}


@pytest.mark.parametrize("what", list(CALLS))
def test_sizes_past_32_bits_are_refused(what):
    with pytest.raises(moe.MoeError, match="MOE_ERR_UNSUPPORTED"):
        CALLS[what]()


def test_workspaces_of_sizes_past_32_bits_are_empty():
    assert moe.moe_grouped_mm_dw_workspace_bytes(1, 1 << 20, 64, 64) > 0
    assert moe.moe_grouped_mm_dw_workspace_bytes(1, WRAP + (1 << 20), 64, 64) == 0
    assert moe.moe_block_norm_grad_workspace_bytes(WRAP + 8, 64) == 0
    assert moe.moe_block_norm_grad_workspace_bytes(8, WRAP + 64) == 0


def test_the_largest_sizes_pass():
    """2^31 - 1 is the library's to judge; here it finds the tensors off the GPU."""
    n = (1 << 31) - 1
    with pytest.raises(ValueError, match="not on the GPU"):
        moe.moe_swiglu(meta(n, 32), meta(n, 16))
    assert B.MOE_OK == 0
