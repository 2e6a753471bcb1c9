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


# ----------------------------------------------------------------------------
# large tiles with their ring of stages going round
# ----------------------------------------------------------------------------

# contractions of over three turns of the longest ring (4 stages of 32 or 3 of 64
# elements, 3 of 128 codes) and a ragged end
RING, RING_CODES = 1096, 1936


def int_case(counts, N, K, seed, gather=False):
    """dy [P, N], x, w [E, N, K] of integers; rows and div for a gathered x."""
    g = gen(seed)
    E, P = len(counts), sum(counts)
    rows, div, X = None, 1, P
    if gather:
        div, X = 3, P // 2
        rows = torch.randint(0, X * div, (P,), generator=g, dtype=torch.int32)
        rows[1], rows[P // 2] = -1, X * div  # no row of x
    return dict(E=E, P=P, N=N, K=K, x=ints(g, X, K), w=ints(g, E, N, K), dy=ints(g, P, N),
                offsets=offsets_of(counts), rows=rows, div=div)


def on_gpu(t, dt=BF16):
    return None if t is None else t.cuda() if t.dtype == torch.int32 else t.to(dt).cuda()


TALL = ["heights", "heights_of_200"]  # the tallest tiles first, and in order


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", TALL)
def test_grouped_mm_ring(gpu_lib, counts, gather, out):
    say(f"grouped_mm ring {counts} gather={gather} {out}")
    c = int_case(COUNTS[counts], 776, RING, 1, gather)
    assert kernel_of(c["E"], c["P"], c["N"]) == "tiles"
    y = poison((c["P"], c["N"]), out)
    moe.moe_grouped_mm(on_gpu(c["x"]), on_gpu(c["w"]), c["offsets"], y, on_gpu(c["rows"]), c["div"])
    want, _ = ref.grouped_mm(c["x"], c["w"], c["offsets"], c["P"], c["rows"], c["div"])
    same(y, want, "y")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("counts", TALL)
def test_grouped_mm_dx_ring(gpu_lib, counts, out):
    say(f"grouped_mm_dx ring {counts} {out}")
    c = int_case(COUNTS[counts], RING, 776, 2)
    assert kernel_of(c["E"], c["P"], c["K"], dx=True) == "tiles"
    dx = poison((c["P"], c["K"]), out)
    moe.moe_grouped_mm_dx(on_gpu(c["dy"]), on_gpu(c["w"]), c["offsets"], dx)
    want, _ = ref.grouped_mm_dx(c["dy"], c["w"], c["offsets"])
    same(dx, want, "dx")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", TALL)
def test_blockscale_mm_ring(gpu_lib, counts, gather, out):
    """Every block with scales of its own, powers of two: a wrong stage's row or
    weight scale shows.  Products up to 64 in units of 2^-4, times K, under 2^24."""
    say(f"blockscale_mm ring {counts} gather={gather} {out}")
    c = int_case(COUNTS[counts], 776, RING_CODES, 3, gather)
    assert kernel_of(c["E"], c["P"], c["N"], bm=128) == "tiles"
    g, kb = gen(4), -(-RING_CODES // 128)
    two = lambda *s: 2.0 ** -torch.randint(0, 3, s, generator=g).float()  # noqa: E731
    xs, ws = two(c["x"].shape[0], kb), two(c["E"], -(-c["N"] // 128), kb)
    y = poison((c["P"], c["N"]), out)
    moe.moe_blockscale_mm(on_gpu(c["x"], E4M3), xs.cuda(), on_gpu(c["w"], E4M3), ws.cuda(),
                          c["offsets"], y, on_gpu(c["rows"]), c["div"])
    x = ref.dequantize(c["x"].to(E4M3), xs, 1)
    w = ref.dequantize(c["w"].to(E4M3), ws, 128)
    want, _ = ref.grouped_mm(x, w, c["offsets"], c["P"], c["rows"], c["div"])
    same(y, want, "y")


# 256 x 256 and 128 x 128 tiles; whole, in parts of the rows, ragged everywhere
DW = [("heights", 1416, 1552), ("heights", 136, 72), ("parts", 2320, 2456), ("parts", 264, 136),
      ("eight", 1352, 1552), ("heights_of_200", 72, 200)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K", DW + [("long rows", 64, 320), ("long rows", 8, 16)])
def test_grouped_mm_dw_exactly(gpu_lib, counts, N, K, gather):
    """A row lost or taken twice where the rows are cut into parts shows."""
    say(f"grouped_mm_dw exactly {counts} {N}x{K} gather={gather}")
    c = int_case([20000] if counts == "long rows" else COUNTS[counts], N, K, 5, gather)
    n = moe.moe_grouped_mm_dw_workspace_bytes(c["E"], c["P"], N, K)
    want, _ = ref.grouped_mm_dw(c["dy"], c["x"], c["offsets"], c["E"], c["rows"], c["div"])
    for out in (BF16, F32):
        dw = poison((c["E"], N, K), out)
        ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
        moe.moe_grouped_mm_dw(on_gpu(c["dy"]), on_gpu(c["x"]), c["offsets"], dw, ws,
                              on_gpu(c["rows"]), c["div"])
        same(dw, want, f"dw {out}")


# ----------------------------------------------------------------------------
# infinities and NaN, by kernel
# ----------------------------------------------------------------------------

BY_KERNEL = [("few", [7, 0, 30, 1], 72), ("small", [40, 0, 300, 1], 72),
             ("tiles", COUNTS["heights"], 1544)]
INF, NAN = float("inf"), float("nan")


def bad_rows(P):
    return ((0, INF), (P // 2, NAN), (P - 1, -INF))


def only(row, got, clean):
    """Every row but `row` as in the clean result, and nothing finite in that one."""
    keep = torch.ones(got.shape[0], dtype=torch.bool, device=got.device)
    keep[row] = False
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[row]).any()


@pytest.mark.parametrize("kernel,counts,N", BY_KERNEL, ids=KERNELS)
def test_nonfinite_rows_stay_alone(gpu_lib, kernel, counts, N):
    """In the last, ragged chunk of K; every weight of its expert is nonzero."""
    K = 136
    c = int_case(counts, N, K, 6)
    assert kernel_of(c["E"], c["P"], N) == kernel
    w = on_gpu(torch.where(c["w"] == 0, 1.0, c["w"]))
    clean, got = (torch.empty((c["P"], N), device="cuda") for _ in range(2))
    moe.moe_grouped_mm(on_gpu(c["x"]), w, c["offsets"], clean)
    for row, v in bad_rows(c["P"]):
        x = on_gpu(c["x"])
        x[row, -1] = v
        moe.moe_grouped_mm(x, w, c["offsets"], got)
        only(row, got, clean)


@pytest.mark.parametrize("kernel,counts,K", BY_KERNEL[1:], ids=KERNELS[1:])
def test_nonfinite_rows_stay_alone_in_dx(gpu_lib, kernel, counts, K):
    N = 136
    c = int_case(counts, N, K, 7)
    assert kernel_of(c["E"], c["P"], K, dx=True) == kernel
    w = on_gpu(torch.where(c["w"] == 0, 1.0, c["w"]))
    clean, got = (torch.empty((c["P"], K), device="cuda") for _ in range(2))
    moe.moe_grouped_mm_dx(on_gpu(c["dy"]), w, c["offsets"], clean)
    for row, v in bad_rows(c["P"]):
        dy = on_gpu(c["dy"])
        dy[row, -1] = v
        moe.moe_grouped_mm_dx(dy, w, c["offsets"], got)
        only(row, got, clean)


@pytest.mark.parametrize("N,K", [(1416, 1552), (136, 72)])
def test_nonfinite_values_stay_in_their_expert_of_dw(gpu_lib, N, K):
    """In x they reach a column of their expert's dw, in dy a row of it."""
    counts = COUNTS["heights"]
    c = int_case(counts, N, K, 8)
    n = moe.moe_grouped_mm_dw_workspace_bytes(c["E"], c["P"], N, K)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    def run(dy, x):
        dw = torch.empty((c["E"], N, K), device="cuda")
        moe.moe_grouped_mm_dw(dy, x, c["offsets"], dw, ws)
        return dw

    dy = on_gpu(torch.where(c["dy"] == 0, 1.0, c["dy"]))
    x = on_gpu(torch.where(c["x"] == 0, 1.0, c["x"]))
    clean = run(dy, x)
    for row, v in bad_rows(c["P"]):
        e = next(e for e, a, b in ref.groups(c["offsets"]) if a <= row < b)
        for of_x in (True, False):
            bad = (x if of_x else dy).clone()
            bad[row, -1] = v
            got = run(dy, bad) if of_x else run(bad, x)
            hit = got[e, :, -1] if of_x else got[e, -1]
            assert not torch.isfinite(hit).any()
            hit.copy_(clean[e, :, -1] if of_x else clean[e, -1])
            assert torch.equal(got, clean)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("kernel,counts,N", BY_KERNEL, ids=KERNELS)
def test_nan_codes_stay_alone(gpu_lib, kernel, counts, N, out):
    """A NaN code of x is a NaN row, one of the weights a NaN column of its expert."""
    K = 144
    c = int_case(counts, N, K, 9)
    E, P = c["E"], c["P"]
    assert kernel_of(E, P, N, bm=128) == kernel
    xs, ws = torch.ones((P, 2), device="cuda"), torch.ones((E, -(-N // 128), 2), device="cuda")
    x, w = on_gpu(c["x"], E4M3), on_gpu(c["w"], E4M3)

    def run(x, w):
        y = torch.empty((P, N), dtype=out, device="cuda")
        moe.moe_blockscale_mm(x, xs, w, ws, c["offsets"], y)
        return y

    clean = run(x, w)
    for row, code in ((0, 0x7F), (P // 2, 0xFF), (P - 1, 0x7F)):
        bad = x.clone()
        bad.view(torch.uint8)[row, -1] = code
        only(row, run(bad, w), clean)
    for e, n in ((2, 0), (2, N - 1)):
        bad = w.clone()
        bad.view(torch.uint8)[e, n, 0] = 0x7F
        got = run(x, bad)
        a, b = int(c["offsets"][e]), int(c["offsets"][e + 1])
        assert torch.isnan(got[a:b, n]).all() and b > a
        got[a:b, n] = clean[a:b, n]
        assert torch.equal(got, clean)


# ----------------------------------------------------------------------------
# a row and the rows beside it
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kernel,counts,N", BY_KERNEL, ids=KERNELS)
def test_a_row_has_the_bits_it_has_beside_other_rows(gpu_lib, kernel, counts, N):
    """Of values whose sums round: every third row beside rows of other values, and
    the group without its first row (so that all rows change places in their
    tiles), by the same kernel."""
    K = 520
    g, E, P = gen(11), len(counts), sum(counts)
    assert kernel_of(E, P, N) == kernel
    x, w = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((P, K), (E, N, K)))

    def run(x, offsets):
        y = torch.empty((x.shape[0], N), device="cuda")
        moe.moe_grouped_mm(x, w, offsets, y)
        return y

    y = run(x, offsets_of(counts))
    kept = torch.arange(P, device="cuda") % 3 == 0
    other = torch.where(kept[:, None], x, torch.randn((P, K), generator=g).to(BF16).cuda())
    assert torch.equal(run(other, offsets_of(counts))[kept], y[kept])
    big = max(range(E), key=lambda e: counts[e])
    a, less = sum(counts[:big]), list(counts)
    less[big] -= 1
    assert kernel_of(E, P - 1, N) == kernel
    keep = torch.arange(P, device="cuda") != a
    assert torch.equal(run(x[keep].contiguous(), offsets_of(less)), y[keep])
