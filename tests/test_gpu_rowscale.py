"""GPU parity of the calls on 8-bit integers with a scale per row.

Codes and scales are decided exactly and products of integers are exact, so the
quantiser and the product are compared bit for bit with the documented
roundings (tests/more_ref.py); SwiGLU's codes are held to its float32 result's
own error and half a code."""
import pytest
import torch

import block_ref
import int4_routed_expert_logits_amd as moe
import more_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
    return o.cuda()


def quantize(x):
    codes = torch.full(x.shape, 77, dtype=torch.int8, device="cuda")
    scales = torch.full(x.shape[:-1], -1.0, device="cuda")
    moe.moe_rowscale_quantize(x, codes, scales)
    return codes, scales


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 16), (3, 48), (5, 512), (4, 2048), (7, 2064), (2, 6144),
                                   (3, 8192), (2, 8208), (1, 65536), (1030, 64), (3, 5, 1040),
                                   (0, 64)])
def test_quantize(gpu_lib, shape, dt):
    say(f"rowscale_quantize {shape} {dt}")
    x = (torch.randn(shape, generator=gen(len(shape) * 7 + shape[-1])) * 3).to(dt)
    if x.numel():
        rows = x.view(-1, shape[-1])
        rows[0, -1] = 300.0   # the largest in the last column
        if len(rows) > 2:
            rows[1] = 0
            rows[2] *= 1e-30
    want, ws = ref.row_quantize(x)
    codes, scales = quantize(x.cuda())
    assert torch.equal(codes.cpu().long(), want)
    assert torch.equal(scales.cpu(), ws)


def test_quantize_halfway_and_extreme_values(gpu_lib):
    """Quotients at and around half-way points, the smallest and largest scales."""
    base = torch.arange(-127, 128, dtype=F32)
    rows = []
    for top in (127.0, 1.0, 0.37, 2.0 ** 120, 3e38, 1e-36, 2.0 ** -126, 1e-44):
        half = (torch.arange(64, dtype=F32) - 31.5) * (top / 127)
        near = torch.cat([half, torch.nextafter(half, torch.full_like(half, torch.inf)),
                          torch.nextafter(half, torch.full_like(half, -torch.inf))])
        row = torch.cat([base * (top / 127), near, torch.tensor([top, -top])])
        rows.append(torch.nn.functional.pad(row, (0, -len(row) % 16)))
    x = torch.stack(rows)
    want, ws = ref.row_quantize(x)
    codes, scales = quantize(x.cuda())
    assert torch.equal(scales.cpu(), ws)
    assert torch.equal(codes.cpu().long(), want)
    assert int(want.abs().max()) == 127


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("K", [32, 2048, 4096, 16384])
def test_quantize_marks_rows_that_are_not_finite(gpu_lib, K, dt):
    x = torch.randn((6, K), generator=gen(K)).to(dt)
    x[1, 3], x[2, -1], x[4, K // 2] = float("inf"), float("nan"), float("-inf")
    codes, scales = quantize(x.cuda())
    bad = torch.tensor([False, True, True, False, True, False])
    assert torch.equal(torch.isnan(scales.cpu()), bad) and (codes.cpu()[bad] == 0).all()
    want, ws = ref.row_quantize(x[~bad])
    assert torch.equal(codes.cpu()[~bad].long(), want) and torch.equal(scales.cpu()[~bad], ws)


# rows per expert
COUNTS = {
    "one": [1], "empty_ends": [0, 3, 0, 1, 0], "edges": [15, 16, 17, 127, 128, 129, 0, 1],
    "long": [300, 0, 555], "many": [i % 5 for i in range(300)], "last_of_1024": [0] * 1023 + [7],
    "none": [0, 0, 0],
    "heights": [257, 288, 289, 320, 321, 512, 513, 576, 640, 641, 768, 900, 960, 961, 1, 33, 65,
                129, 255, 256],
    "row_of_2000": [2000],
}
SIZES = [(8, 16), (64, 64), (72, 208), (264, 144), (512, 320), (1544, 80), (72, 1552),
         (1416, 1552)]  # N, K
MM = [("one", 0), ("one", 4), ("empty_ends", 2), ("edges", 1), ("edges", 3), ("edges", 4),
      ("long", 2), ("long", 4), ("many", 0), ("many", 2), ("last_of_1024", 2), ("none", 1),
      ("heights", 5), ("heights", 7), ("row_of_2000", 6), ("edges", 6)]


def mm_case(counts, N, K, gather, tail, seed):
    P = sum(counts) + tail
    g = gen(seed)
    rows, div, X = None, 1, P
    if gather:
        div, X = 3, max(P // 2, 1)
        rows = torch.randint(0, X * div, (P,), generator=g, dtype=torch.int32)
        if P > 2:
            rows[1], rows[P // 2] = -1, X * div  # no row of x
        rows = rows.cuda()
    ints = lambda *s: torch.randint(-128, 128, s, generator=g).to(torch.int8).cuda()  # noqa: E731
    return dict(xq=ints(X, K), xs=torch.rand(X, generator=g).cuda(), wq=ints(len(counts), N, K),
                ws=(torch.rand((len(counts), N), generator=g) - 0.5).cuda(),
                offsets=offsets_of(counts), rows=rows, div=div, P=P)


def run_mm(c, out):
    y = torch.full((c["P"], c["wq"].shape[1]), 768.0, dtype=out, device="cuda")
    moe.moe_rowscale_mm(c["xq"], c["xs"], c["wq"], c["ws"], c["offsets"], y, c["rows"], c["div"])
    return y


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather,tail", [(False, 0), (True, 5)])
@pytest.mark.parametrize("counts,size", MM)
def test_rowscale_mm_is_exact(gpu_lib, counts, size, gather, tail, out):
    say(f"rowscale_mm {counts} {SIZES[size]} gather={gather} tail={tail} {out}")
    c = mm_case(COUNTS[counts], *SIZES[size], gather, tail, 11 * size + gather)
    y = run_mm(c, out)
    want = ref.rowscale_mm(c["xq"], c["xs"], c["wq"], c["ws"], c["offsets"], c["P"], out,
                           c["rows"], c["div"])
    n = sum(COUNTS[counts])
    assert torch.equal(y[:n].cpu(), want[:n])
    assert (y[n:] == 768).all()


def test_longest_sums_do_not_overflow(gpu_lib):
    """65536 products of -128 and -128 (2^30), on few rows and on many."""
    for P in (3, 400):
        c = dict(xq=torch.full((P, 65536), -128, dtype=torch.int8, device="cuda"),
                 xs=torch.ones(P, device="cuda"),
                 wq=torch.full((1, 16, 65536), -128, dtype=torch.int8, device="cuda"),
                 ws=torch.ones((1, 16), device="cuda"), offsets=offsets_of([P]), rows=None, div=1,
                 P=P)
        assert (run_mm(c, F32) == 2.0 ** 30).all()


def test_scales_that_are_not_finite_stay_in_their_row_and_column(gpu_lib):
    c = mm_case(COUNTS["edges"], 264, 144, False, 0, 5)
    clean = run_mm(c, F32)
    xs, ws = c["xs"].clone(), c["ws"].clone()
    xs[20], ws[:, 7] = float("nan"), float("inf")
    y = run_mm(dict(c, xs=xs, ws=ws), F32)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[20], keep[:, 7] = False, False
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[20]).all() and not torch.isfinite(y[:, 7]).any()


def test_offsets_are_clamped(gpu_lib):
    c = mm_case([4, 5, 6], 72, 208, False, 0, 9)
    c["offsets"] = torch.tensor([-5, 4, 3, 1000], dtype=torch.int32, device="cuda")
    y = run_mm(c, F32)
    want = ref.rowscale_mm(c["xq"], c["xs"], c["wq"][[0, 2]], c["ws"][[0, 2]],
                           torch.tensor([0, 4, 15]), c["P"], F32)
    # group 1 is empty (its end lies before its start); group 2 begins at 3: row 3 is
    # written by both 0 and 2, so only the others are looked at
    assert torch.equal(y[:3].cpu(), want[:3]) and torch.equal(y[4:].cpu(), want[4:])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("P,f,used", [(1, 16, 1), (5, 64, 3), (9, 2048, 9), (7, 2064, 5),
                                      (3, 8192, 2), (2, 8208, 2), (1, 32768, 1), (300, 192, 0)])
def test_swiglu_rowscale(gpu_lib, P, f, used, dt):
    say(f"swiglu_rowscale {P}x{f} used={used} {dt}")
    gu = (torch.randn((P, 2 * f), generator=gen(f + P)) * 2).to(dt).cuda()
    codes = torch.full((P, f), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((P,), -1.0, device="cuda")
    n = torch.tensor([used], dtype=torch.int32, device="cuda")
    moe.moe_swiglu_rowscale(gu, codes, scales, n)
    assert (codes[used:] == 77).all() and (scales[used:] == -1).all()
    h = block_ref.swiglu(gu)[:used]
    top = h.abs().amax(1) if used else torch.zeros(0)
    s = block_ref.d64(scales[:used])
    # exp (its argument's and its own rounding: 2 + |g| units at |g| <= 12), sum,
    # quotient and product: 16 units of 2^-24; the scale two more
    assert ((s - top / 127).abs() <= 20 * ref.U * top / 127).all()
    err = (codes[:used].cpu().double() * s[:, None] - h).abs()
    assert (err <= s[:, None] * (0.5 + 127 * 20 * ref.U) + 16 * ref.U * h.abs()).all()
    assert (codes[:used].abs().amax(1) == 127).all() if used else True


def test_swiglu_rowscale_of_all_rows_and_not_finite(gpu_lib):
    gu = torch.randn((4, 256), generator=gen(3)).cuda()
    gu[2, 5] = float("nan")
    codes, scales = torch.empty((4, 128), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    moe.moe_swiglu_rowscale(gu, codes, scales)
    assert torch.isnan(scales[2]) and (codes[2] == 0).all()
    h = torch.empty((4, 128), device="cuda")
    moe.moe_swiglu(gu, h)
    rest = [0, 1, 3]
    want, ws = ref.row_quantize(h[rest])  # the same float32 values, quantised
    assert torch.equal(codes[rest].cpu().long(), want) and torch.equal(scales[rest].cpu(), ws)


def test_captured_on_a_side_stream(gpu_lib):
    """Quantise, product, SwiGLU to codes, product, captured once and replayed with
    new inputs between eager calls."""
    g = gen(17)
    T, d, f, E = 40, 320, 192, 8
    x = torch.randn((T, d), generator=g).to(BF16).cuda()
    wq = [torch.randint(-127, 128, s, generator=g).to(torch.int8).cuda()
          for s in ((E, 2 * f, d), (E, d, f))]
    ws = [torch.rand(w.shape[:2], generator=g).cuda() * 1e-3 for w in wq]
    offsets = offsets_of([T // E] * E)
    xq, xs = torch.empty((T, d), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    gu = torch.empty((T, 2 * f), dtype=BF16, device="cuda")
    hq, hs = torch.empty((T, f), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y = torch.empty((T, d), dtype=BF16, device="cuda")

    def run():
        moe.moe_rowscale_quantize(x, xq, xs)
        moe.moe_rowscale_mm(xq, xs, wq[0], ws[0], offsets, gu)
        moe.moe_swiglu_rowscale(gu, hq, hs)
        moe.moe_rowscale_mm(hq, hs, wq[1], ws[1], offsets, y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        run()
    for i in range(4):
        x.copy_(torch.randn((T, d), generator=g).to(BF16))
        run()
        torch.cuda.synchronize()
        want = y.clone()
        y.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
