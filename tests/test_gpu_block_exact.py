"""The grouped products of include/moe_int4_block.h on values whose sums float32
holds exactly, so that every order of adding them gives the same bits and a
result is compared with equality.

Small integers: products up to 64 and sums of a few thousand of them stay under
2^24.  A float32 result is then the exact one, a bf16 result its one rounding.
"""
import pytest
import torch

import block_ref as ref
import int4_routed_expert_logits_amd as moe
from test_gpu_block import BF16, COUNTS, F32, gen, offsets_of, poison, say

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
KERNELS = ("few", "small", "tiles")


def kernel_of(E, P, cols, dx=False, bm=256):
    """Which kernel a product of these sizes takes (launch_grouped_mm's rule)."""
    if not dx and P <= 64 + 3 * E:
        return "few"
    return "tiles" if (P // bm + min(E, P)) * -(-cols // 256) >= 160 else "small"


def ints(g, *shape, top=8):
    return torch.randint(-top, top + 1, shape, generator=g).float()


def rounded(want, dtype):
    """float64 integers below 2^24: exact in float32, then one rounding."""
    return want.float().to(dtype)


def same(got, want, what):
    off = got.cpu() != rounded(want, got.dtype)
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} differ"


# ----------------------------------------------------------------------------
# 8-bit products: blocks whose large products cancel
# ----------------------------------------------------------------------------

def cancelling_codes(g, E, P, N, K):
    """Of four neighbouring columns two have products of +-448 * 448, which cancel,
    and two products of integers up to 15; a block's partial sums stay under
    32 * 448^2 + 64 * 15^2 < 2^23, in units of 1."""
    x, w = ints(g, P, K, top=15), ints(g, E, N, K, top=15)
    x[:, 0::4] = x[:, 1::4] = 448.0
    w[:, :, 0::4], w[:, :, 1::4] = 448.0, -448.0
    return x.to(E4M3), w.to(E4M3)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("kernel,counts,N,K", [
    ("few", [5, 0, 20], 72, 400), ("small", [300, 1, 70], 136, 656), ("tiles", COUNTS["heights"], 1544, 272)])
def test_blockscale_mm_keeps_what_cancelling_products_leave(gpu_lib, kernel, counts, N, K, out):
    say(f"blockscale_mm cancelling {kernel} {out}")
    E, P = len(counts), sum(counts)
    assert kernel_of(E, P, N) == kernel
    g = gen(K)
    xq, wq = cancelling_codes(g, E, P, N, K)
    xs, ws = torch.ones((P, -(-K // 128))), torch.ones((E, -(-N // 128), -(-K // 128)))
    y = poison((P, N), out)
    moe.moe_blockscale_mm(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), offsets_of(counts), y)
    want, _ = ref.grouped_mm(xq.float(), wq.float(), offsets_of(counts), P)
    same(y, want, "y")
