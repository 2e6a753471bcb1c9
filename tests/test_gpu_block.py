"""GPU parity of the calls in include/moe_int4_block.h with plain float64 forms
on the CPU (tests/block_ref.py).

Allowances.  A product of two bf16 (or e4m3) values is exact in float32, and a
float32 sum of n terms is off by at most n * 2^-23 of the terms' magnitudes
(2^-24 per addition, twice that where an adder truncates); the result is
rounded once to its type, half_step(type) of its magnitude.  Elementwise
results take a few float32 roundings (2^-24 each, with exp and division within
a few of those) and the last one.  Each test states its own count.
"""
import pytest
import torch

import block_ref as ref
import int4_routed_expert_logits_amd as moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U32 = 2.0 ** -23  # a float32 operation, truncating or not


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def rand(g, *shape, dt=BF16, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dt).cuda()


def check(got, want, allow, what):
    """|got - want| <= allow elementwise."""
    got = ref.d64(got)
    assert torch.isfinite(got).all(), what
    worst = ((got - want).abs() - allow).max() if got.numel() else torch.tensor(-1.0)
    ratio = ((got - want).abs() / allow.clamp(min=1e-300)).max() if got.numel() else 0.0
    say(f"  {what}: worst error / allowance {float(ratio):.3f}")
    assert float(worst) <= 0.0, f"{what}: error over its allowance (ratio {float(ratio):.3f})"


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
    return o.cuda()


def poison(shape, dt):
    """An output whose untouched elements show."""
    return torch.full(shape, 768.0, dtype=dt, device="cuda")


# ----------------------------------------------------------------------------
# grouped products
# ----------------------------------------------------------------------------

# rows per expert: none at all, one, tile edges, long, ragged
COUNTS = {
    "one": [1],
    "empty_ends": [0, 3, 0, 1, 0],
    "edges": [15, 16, 17, 127, 128, 129, 0, 1],
    "long": [300, 0, 555],
    "many": [i % 5 for i in range(300)],
    "last_of_1024": [0] * 1023 + [7],
    "none": [0, 0, 0],
    # around every height of the large tiles (tall ones first, and in order)
    "heights": [257, 288, 289, 320, 321, 512, 513, 576, 640, 641, 768, 900, 960, 961, 1, 33, 65,
                129, 255, 256],
}
COUNTS["eight"] = [0, 1, 63, 64, 65, 200, 300, 107]
COUNTS["parts"] = [4100]
COUNTS["heights_of_200"] = [n for h in COUNTS["heights"] for n in (h, *[0] * 9)]
SIZES = [(8, 8), (64, 64), (72, 200), (264, 136), (512, 320), (1544, 72), (72, 1544),
         (1416, 1552), (1352, 1552), (2320, 2456)]  # N, K
# enough tiles for the large ones: forward, input gradient
HEIGHTS = [("heights", 5), ("heights_of_200", 3)]
HEIGHTS_DX = [("heights", 6), ("heights_of_200", 2)]
# large tiles of a weight gradient: whole, short, in two parts of the rows
LARGE_DW = [("heights", 3), ("eight", 7), ("eight", 8), ("parts", 9)]
MM = [("one", 0), ("one", 4), ("empty_ends", 2), ("edges", 1), ("edges", 3), ("edges", 4),
      ("long", 2), ("long", 4), ("many", 0), ("many", 2), ("last_of_1024", 2), ("none", 1)]


def mm_case(counts, size, gather, tail, seed):
    """x, w, dy, offsets, rows, div, P with `tail` positions of no group."""
    N, K = SIZES[size]
    counts = COUNTS[counts]
    P = sum(counts) + tail
    g = gen(seed)
    rows, div, X = None, 1, P
    if gather:
        div, X = 3, max(P // 2, 1)
        rows = torch.randint(0, X * div, (P,), generator=g, dtype=torch.int32)
        if P > 2:
            rows[1], rows[P // 2] = -1, X * div  # no row of x
        rows = rows.cuda()
    return dict(x=rand(g, X, K), w=rand(g, len(counts), N, K, scale=0.1), dy=rand(g, P, N),
                offsets=offsets_of(counts), rows=rows, div=div, P=P, N=N, K=K, E=len(counts),
                used=sum(counts))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather,tail", [(False, 0), (True, 5)])
@pytest.mark.parametrize("counts,size", MM + HEIGHTS)
def test_grouped_mm(gpu_lib, counts, size, gather, tail, out):
    say(f"grouped_mm {counts} {SIZES[size]} gather={gather} tail={tail} {out}")
    c = mm_case(counts, size, gather, tail, 11 * size + gather)
    y = poison((c["P"], c["N"]), out)
    moe.moe_grouped_mm(c["x"], c["w"], c["offsets"], y, c["rows"], c["div"])
    want, mag = ref.grouped_mm(c["x"], c["w"], c["offsets"], c["P"], c["rows"], c["div"])
    n = c["used"]
    check(y[:n], want[:n], c["K"] * U32 * mag[:n] + ref.half_step(out) * want[:n].abs(), "y")
    assert (y[n:] == 768).all()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("counts,size", MM + HEIGHTS_DX)
def test_grouped_mm_dx(gpu_lib, counts, size, out):
    say(f"grouped_mm_dx {counts} {SIZES[size]} {out}")
    c = mm_case(counts, size, False, 3, 100 + size)
    dx = poison((c["P"], c["K"]), out)
    moe.moe_grouped_mm_dx(c["dy"], c["w"], c["offsets"], dx)
    want, mag = ref.grouped_mm_dx(c["dy"], c["w"], c["offsets"])
    n = c["used"]
    check(dx[:n], want[:n], c["N"] * U32 * mag[:n] + ref.half_step(out) * want[:n].abs(), "dx")
    assert (dx[n:] == 768).all()


def run_dw(c, out, dw=None):
    dw = poison((c["E"], c["N"], c["K"]), out) if dw is None else dw
    ws = torch.full((max(256, moe.moe_grouped_mm_dw_workspace_bytes(c["E"], c["P"], c["N"], c["K"])),),
                    255, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_mm_dw(c["dy"], c["x"], c["offsets"], dw, ws, c["rows"], c["div"])
    return dw


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather,tail", [(False, 0), (True, 5)])
@pytest.mark.parametrize("counts,size",
                         [m for m in MM + LARGE_DW if m[0] != "last_of_1024"])
def test_grouped_mm_dw(gpu_lib, counts, size, gather, tail, out):
    say(f"grouped_mm_dw {counts} {SIZES[size]} gather={gather} tail={tail} {out}")
    c = mm_case(counts, size, gather, tail, 200 + 11 * size + gather)
    dw = run_dw(c, out)
    want, mag = ref.grouped_mm_dw(c["dy"], c["x"], c["offsets"], c["E"], c["rows"], c["div"])
    check(dw, want, max(c["P"], 1) * U32 * mag + ref.half_step(out) * want.abs(), "dw")


@pytest.mark.parametrize("E,P,N,K", [(1, 5000, 8, 16), (1, 20000, 64, 320), (2, 9000, 264, 40),
                                     (3, 4100, 8, 8)])
def test_grouped_mm_dw_few_weights_over_many_rows(gpu_lib, E, P, N, K):
    """Few output tiles and long sums (a router's or a small expert's weights)."""
    say(f"grouped_mm_dw long E={E} P={P} {N}x{K}")
    g = gen(P)
    cut = sorted(int(v) for v in torch.randint(0, P, (E - 1,), generator=g))
    ends = [0, *cut, P]
    c = dict(x=rand(g, P, K), dy=rand(g, P, N), rows=None, div=1, E=E, P=P, N=N, K=K,
             offsets=offsets_of([b - a for a, b in zip(ends, ends[1:])]))
    want, mag = ref.grouped_mm_dw(c["dy"], c["x"], c["offsets"], E)
    got = run_dw(c, F32)
    # partial sums are added in float32 too: fewer terms each, one more level
    check(got, want, (P + 64) * U32 * mag + ref.half_step(F32) * want.abs(), "dw")
    assert torch.equal(got, run_dw(c, F32))


def test_grouped_mm_dw_of_no_rows_is_zero(gpu_lib):
    for out in (BF16, F32):
        dw = poison((3, 16, 24), out)
        moe.moe_grouped_mm_dw(torch.empty((0, 16), dtype=BF16, device="cuda"),
                              torch.empty((0, 24), dtype=BF16, device="cuda"),
                              torch.zeros(4, dtype=torch.int32, device="cuda"), dw,
                              torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        assert (dw == 0).all()


def test_grouped_mm_nonfinite_stay_in_their_rows(gpu_lib):
    """An infinity or NaN in one row of x (or dy) reaches that row's outputs
    alone; in dw, its expert's alone -- the zero-filled edges of a tile never
    multiply it."""
    c = mm_case("edges", 2, False, 0, 5)
    clean = torch.empty((c["P"], c["N"]), dtype=F32, device="cuda")
    moe.moe_grouped_mm(c["x"], c["w"], c["offsets"], clean)
    for row, v in ((0, float("inf")), (20, float("nan")), (c["used"] - 1, float("-inf"))):
        x = c["x"].clone()
        x[row, -1] = v
        y = torch.empty_like(clean)
        moe.moe_grouped_mm(x, c["w"], c["offsets"], y)
        same = torch.ones(c["P"], dtype=torch.bool, device="cuda")
        same[row] = False
        assert torch.equal(y[same], clean[same]) and not torch.isfinite(y[row]).any()
        cx = dict(c, x=x)
        dw, base = run_dw(cx, F32), run_dw(c, F32)
        e = next(e for e, a, b in ref.groups(c["offsets"]) if a <= row < b)
        keep = [i for i in range(c["E"]) if i != e]
        assert torch.equal(dw[keep], base[keep])
        assert torch.equal(dw[e][:, :-1], base[e][:, :-1])


def test_grouped_mm_offsets_are_clamped(gpu_lib):
    """Offsets outside [0, P], or falling, address nothing outside the arrays."""
    c = mm_case("empty_ends", 2, False, 0, 6)
    P = c["P"]
    bad = torch.tensor([-5, 2, 1, P + 100, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    y = poison((P, c["N"]), F32)
    moe.moe_grouped_mm(c["x"], c["w"], bad, y)
    dx = poison((P, c["K"]), F32)
    moe.moe_grouped_mm_dx(c["dy"], c["w"], bad, dx)
    dw = run_dw(dict(c, offsets=bad), F32)
    torch.cuda.synchronize()
    want, mag = ref.grouped_mm(c["x"], c["w"], [0, 2], 2)
    check(y[:1], want[:1], c["K"] * U32 * mag[:1] + 1e-30, "expert 0's first row")
    assert torch.isfinite(dw).all()


def test_grouped_mm_rows_are_independent_of_their_batch(gpu_lib):
    """A row alone gives the same bits as the row in a batch served by the same
    kernel, and a repeated call the same bits."""
    c = mm_case("long", 4, False, 0, 7)
    y = [poison((c["P"], c["N"]), F32) for _ in range(2)]
    for o in y:
        moe.moe_grouped_mm(c["x"], c["w"], c["offsets"], o)
    assert torch.equal(*y)


# ----------------------------------------------------------------------------
# 8-bit codes
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (3, 128), (5, 144), (130, 272), (2, 129, 48),
                                   (3, 256, 128), (2, 1, 400)])
def test_blockscale_quantize(gpu_lib, shape, block_rows, dt):
    say(f"quantize {shape} {block_rows} {dt}")
    x = rand(gen(1), *shape, dt=F32)
    flat = x.view(-1, shape[-1])
    flat[0] *= 1e-3
    flat[-1] *= 1e30
    if flat.shape[0] > 2:
        flat[1] = 0.0
        flat[2] = torch.randn(shape[-1], generator=gen(2)).cuda() * 3e-40  # subnormal
    # values at the half steps of e4m3 and at the border of a scale
    flat[0, :8] = torch.tensor([448.0, 1.0625, 1.1875, 448 * 2.0 ** -12, 2.0 ** -10, -17.0, 0.0,
                                -0.0]).cuda()
    x = x.to(dt)
    sr = shape[-2] if block_rows == 1 else -(-shape[-2] // 128)
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = poison((*shape[:-2], sr, -(-shape[-1] // 128)), F32)
    moe.moe_blockscale_quantize(x, block_rows, codes, scales)
    values, want = ref.quantize(x, block_rows)
    assert torch.equal(ref.d64(scales), want)
    assert torch.equal(codes.cpu().float().to(torch.float64), values)


def test_blockscale_quantize_borders(gpu_lib):
    """absmax at, just below and just above 448 * 2^n; every e4m3 half step;
    non-finite values get a NaN code and do not move the scale."""
    rows = []
    for top in (448.0, 447.9, 448.1, 1.75, 1.7500001, 1.7499999, 3.4e38, 1e-45, 2.0 ** -126):
        r = torch.zeros(128)
        r[5] = top
        r[6] = -top / 3
        rows.append(r)
    t = ref.e4m3_values()
    half = ((t[1:] + t[:-1]) / 2).float()  # exact in float32
    for eps in (0.0, 2.0 ** -23, -(2.0 ** -23)):
        r = torch.zeros(128)
        r[0] = 448.0
        r[1:127] = half[:126] * (1 + eps)
        rows.append(r)
    bad = torch.randn(128, generator=gen(3))
    bad[3], bad[4], bad[5] = float("inf"), float("-inf"), float("nan")
    rows.append(bad)
    x = torch.stack(rows).cuda()
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = poison((x.shape[0], 1), F32)
    moe.moe_blockscale_quantize(x, 1, codes, scales)
    values, want = ref.quantize(x, 1)
    assert torch.equal(ref.d64(scales), want)
    got = codes.cpu().view(torch.float8_e4m3fn).float().to(torch.float64)
    assert torch.equal(torch.isnan(got), torch.isnan(values))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(values))


def code_case(counts, size, gather, tail, seed):
    c = mm_case(counts, size, gather, tail, seed)
    g = gen(seed + 1)
    N, K, E = c["N"], c["K"], c["E"]
    K = -(-K // 16) * 16
    X, kb = c["x"].shape[0], -(-K // 128)
    code = lambda *s: (torch.randn(s, generator=g) * 100).clamp(-448, 448).to(  # noqa: E731
        torch.float8_e4m3fn).cuda()
    c.update(K=K, xq=code(X, K), wq=code(E, N, K),
             xs=(torch.rand((X, kb), generator=g) * 0.1 + 0.01).cuda(),
             ws=(torch.rand((E, -(-N // 128), kb), generator=g) * 0.1 - 0.05).cuda())
    return c


def blockscale_ref(c):
    x = ref.dequantize(c["xq"], c["xs"], 1)
    w = ref.dequantize(c["wq"], c["ws"], 128)
    return ref.grouped_mm(x, w, c["offsets"], c["P"], c["rows"], c["div"])


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather,tail", [(False, 0), (True, 5)])
@pytest.mark.parametrize("counts,size", MM + HEIGHTS)
def test_blockscale_mm(gpu_lib, counts, size, gather, tail, out):
    """float32: exact products, a float32 sum, and per block one product of the
    scales and one fused multiply-add: K + 2 operations' roundings.  bf16: a
    block's products are summed by the 8-bit matrix instructions, whose sums of
    128 were 2.5e-5 of the terms' magnitudes off at most where measured; four
    times that is allowed (1e-4) before the rounding to bf16."""
    say(f"blockscale_mm {counts} {SIZES[size]} gather={gather} tail={tail} {out}")
    c = code_case(counts, size, gather, tail, 300 + 11 * size + gather)
    y = poison((c["P"], c["N"]), out)
    moe.moe_blockscale_mm(c["xq"], c["xs"], c["wq"], c["ws"], c["offsets"], y, c["rows"], c["div"])
    want, mag = blockscale_ref(c)
    n = c["used"]
    sums = (c["K"] + 2) * U32 + (1e-4 if out == BF16 else 0.0)
    check(y[:n], want[:n], sums * mag[:n] + ref.half_step(out) * want[:n].abs(), "y")
    assert (y[n:] == 768).all()


# ----------------------------------------------------------------------------
# SwiGLU
# ----------------------------------------------------------------------------

SWIGLU = [(1, 8), (1, 64), (3, 200), (77, 128), (5, 2048), (300, 24), (2, 4104)]


def silu_allow(want, gu, dt):
    """exp, 1 +, division, two products: under 16 float32 roundings, and the
    result's; results below float32's smallest normal have its spacing."""
    return 16 * U32 * want.abs() + ref.half_step(dt) * want.abs() + 1e-37


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("P,f", SWIGLU)
def test_swiglu(gpu_lib, P, f, dt):
    say(f"swiglu {P} {f} {dt}")
    gu = rand(gen(P + f), P, 2 * f, dt=dt, scale=3.0)
    gu[0, 0], gu[0, 1], gu[-1, 2] = 60.0, -80.0, 0.0
    h = poison((P, f), dt)
    moe.moe_swiglu(gu, h)
    want = ref.swiglu(gu)
    check(h, want, silu_allow(want, gu, dt), "h")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("P,f", SWIGLU)
def test_swiglu_grad(gpu_lib, P, f, dt):
    """1 + g (1 - s) cancels near its root (g = -1.28), where the error is that
    of its terms: the allowance goes by |1| + |g (1 - s)|."""
    say(f"swiglu_grad {P} {f} {dt}")
    g = gen(P + f)
    gu, dh = rand(g, P, 2 * f, dt=dt, scale=3.0), rand(g, P, f, dt=dt)
    gu[0, 0], gu[0, 1], gu[-1, 2] = 60.0, -80.0, 0.0
    want = ref.swiglu_grad(gu, dh)
    a, u = ref.d64(gu).chunk(2, 1)
    s = 1 / (1 + torch.exp(-a))
    # (1 - s) is a rounded s away from 1: 2^-23 absolute, times |g|
    mag = torch.cat([(ref.d64(dh) * u * s).abs() * (1 + (a * (1 - s)).abs() + a.abs()),
                     want[:, f:].abs()], 1)
    dgu = poison((P, 2 * f), dt)
    moe.moe_swiglu_grad(gu, dh, dgu)
    check(dgu, want, 16 * U32 * mag + ref.half_step(dt) * want.abs() + 1e-37, "dgu")
    again = gu.clone()
    moe.moe_swiglu_grad(again, dh, again)  # in place
    assert torch.equal(again, dgu)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("P,f", [(1, 16), (3, 208), (77, 128), (5, 2048), (9, 4112)])
def test_swiglu_quantize(gpu_lib, P, f, dt):
    """Exactly the quantiser on moe_swiglu's float32 result."""
    say(f"swiglu_quantize {P} {f} {dt}")
    gu = rand(gen(P + f), P, 2 * f, dt=dt, scale=2.0)
    h = torch.empty((P, f), dtype=F32, device="cuda")
    moe.moe_swiglu(gu.float(), h)
    kb = -(-f // 128)
    codes = [torch.empty((P, f), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [poison((P, kb), F32) for _ in range(2)]
    moe.moe_swiglu_quantize(gu, codes[0], scales[0])
    moe.moe_blockscale_quantize(h, 1, codes[1], scales[1])
    assert torch.equal(*codes) and torch.equal(*scales)
    values, want = ref.quantize(h, 1)
    assert torch.equal(ref.d64(scales[0]), want)


def test_swiglu_leaves_rows_behind_the_last(gpu_lib):
    P, f = 37, 64
    g = gen(4)
    gu, dh = rand(g, P, 2 * f), rand(g, P, f)
    full = torch.empty((P, f), dtype=BF16, device="cuda")
    moe.moe_swiglu(gu, full)
    for n in (0, 1, 20, P, P + 9, -3):
        nr, m = torch.tensor([n], dtype=torch.int32).cuda(), min(max(n, 0), P)
        h, dgu = poison((P, f), BF16), poison((P, 2 * f), BF16)
        codes = torch.full((P, f), 77, dtype=torch.uint8, device="cuda")
        scales = poison((P, 1), F32)
        moe.moe_swiglu(gu, h, nr)
        moe.moe_swiglu_grad(gu, dh, dgu, nr)
        moe.moe_swiglu_quantize(gu, codes, scales, nr)
        assert torch.equal(h[:m], full[:m])
        assert (h[m:] == 768).all() and (dgu[m:] == 768).all()
        assert (codes[m:] == 77).all() and (scales[m:] == 768).all()


# ----------------------------------------------------------------------------
# the combine's gradient
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("ydt,odt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T,k,d", [(1, 1, 64), (5, 8, 512), (33, 3, 1088), (2, 32, 8192)])
def test_combine_grad(gpu_lib, T, k, d, ydt, odt):
    say(f"combine_grad {T} {k} {d} {ydt} {odt}")
    g = gen(T + d)
    inv = torch.randperm(T * k, generator=g).int()
    if T > 1:
        inv[3], inv[T * k - 1] = -1, T * k  # slots without a row
    inv = inv.cuda()
    dout, y = rand(g, T, d, dt=odt), rand(g, T * k, d, dt=ydt)
    w = torch.rand((T, k), generator=g).cuda()
    dy, dw = poison((T * k, d), ydt), poison((T, k), F32)
    sh = (d, 64, 64, k, 64, 0)
    moe.moe_combine_grad(sh, dout, y, inv, w, dy, dw)
    rdy, rdw, mag = ref.combine_grad(dout, y, inv, w)
    unused = torch.isnan(rdy[:, 0])
    got = ref.d64(dy)
    assert (got[unused] == 768).all()
    # one float32 product and the rounding to y's type
    check(got[~unused], rdy[~unused], (U32 + ref.half_step(ydt)) * rdy[~unused].abs(), "dy")
    # y * dout is exact for bf16, else rounded inside a fused sum of d terms
    check(dw, rdw, d * U32 * mag + 1e-30, "dtopk_w")
    inplace = y.clone()
    moe.moe_combine_grad(sh, dout, inplace, inv, w, inplace, dw)
    assert torch.equal(inplace[~unused.cuda()], dy[~unused.cuda()])
    assert torch.equal(inplace[unused.cuda()], y[unused.cuda()])


# ----------------------------------------------------------------------------
# block norm
# ----------------------------------------------------------------------------

NORM_SHAPES = [(1, 8), (1, 6144), (3, 520), (7, 8192), (600, 64), (130, 1000)]
# y, res, post, pre, gate
NORM_FORMS = [(1, 1, 1, 1, "none"), (1, 1, 1, 1, "row"), (1, 1, 1, 1, "token"), (0, 1, 0, 1, "none"),
              (1, 0, 1, 0, "token"), (1, 1, 0, 1, "row"), (1, 1, 0, 0, "none"), (1, 0, 0, 1, "none")]


def norm_case(T, d, form, ydt, rdt, ndt, seed):
    hy, hr, post, pre, gate = form
    g = gen(seed)
    t = dict(y=rand(g, T, d, dt=ydt) if hy else None, res=rand(g, T, d, dt=rdt) if hr else None,
             w_post=(1 + rand(g, d, dt=F32, scale=0.2)) if post else None,
             w_pre=(1 + rand(g, d, dt=F32, scale=0.2)) if pre else None,
             gate=None if gate == "none" else rand(g, 1 if gate == "row" else T, d, dt=ydt),
             dr=rand(g, T, d, dt=rdt), dn=rand(g, T, d, dt=ndt) if pre else None)
    return t, 0.75, 1e-5


def up(t):
    return None if t is None else ref.d64(t)


@pytest.mark.parametrize("dts", [(BF16, BF16, BF16), (F32, BF16, BF16), (F32, F32, F32),
                                 (BF16, F32, BF16)])
@pytest.mark.parametrize("form", NORM_FORMS)
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_block_norm(gpu_lib, T, d, form, dts):
    """r: two norms' statistics are sums of d squares (relative error d * 2^-24 of
    positive terms, halved by the root), then under 8 roundings of p and res;
    n: the same again, the error of r carried through."""
    say(f"block_norm {T} {d} {form} {dts}")
    ydt, rdt, ndt = dts
    c, scale, eps = norm_case(T, d, form, ydt, rdt, ndt, T + d)
    if not form[1]:
        rdt = dts[1]
    r = poison((T, d), rdt)
    n = poison((T, d), ndt) if form[3] else None
    moe.moe_block_norm(c["y"], c["res"], r, n, c["w_post"], c["w_pre"], c["gate"], scale, eps)
    wr, wn = ref.block_norm(up(c["y"]), up(c["res"]), up(c["w_post"]), up(c["w_pre"]),
                            up(c["gate"]), scale, eps)
    stat = (d / 2 + 8) * U32
    res = torch.zeros_like(wr) if c["res"] is None else up(c["res"])
    err_r = stat * ((wr - res).abs() + wr.abs())
    check(r, wr, err_r + ref.half_step(rdt) * wr.abs() + 1e-30, "r")
    if n is not None:
        b = 1 / torch.sqrt((wr * wr).mean(1, keepdim=True) + eps)
        # errors of r move n directly and through the mean of r^2
        rel = (err_r * wr.abs()).sum(1, keepdim=True) / ((wr * wr).sum(1, keepdim=True) + eps * d)
        err_n = up(c["w_pre"]).abs() * b * err_r + wn.abs() * (rel + stat)
        check(n, wn, err_n + ref.half_step(ndt) * wn.abs() + 1e-30, "n")
    if c["res"] is not None:  # in place
        again = c["res"].clone()
        moe.moe_block_norm(c["y"], again, again, n, c["w_post"], c["w_pre"], c["gate"], scale, eps)
        assert torch.equal(again, r)


def grad_outputs(c, T, d, ydt, rdt):
    new = lambda like, dt: None if like is None else poison(like.shape, dt)  # noqa: E731
    return dict(dy=new(c["y"], ydt), dres=poison((T, d), rdt), dw_post=new(c["w_post"], F32),
                dw_pre=new(c["w_pre"], F32), dgate=new(c["gate"], ydt))


def run_norm_grad(c, o, T, d, scale, eps):
    ws = torch.full((max(256, moe.moe_block_norm_grad_workspace_bytes(T, d)),), 255,
                    dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_grad(c["y"], c["res"], c["dr"], c["dn"], o["dy"], o["dres"], o["dw_post"],
                            o["dw_pre"], o["dgate"], c["w_post"], c["w_pre"], c["gate"], scale,
                            eps, ws)


@pytest.mark.parametrize("dts", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16)])
@pytest.mark.parametrize("form", NORM_FORMS)
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_block_norm_grad(gpu_lib, T, d, form, dts):
    """Errors are relative to the magnitudes that enter each formula: per row
    (d + 16) roundings of the terms' magnitudes with their means, per column T
    more."""
    say(f"block_norm_grad {T} {d} {form} {dts}")
    ydt, rdt, ndt = dts
    c, scale, eps = norm_case(T, d, form, ydt, rdt, ndt, 2 * T + d)
    o = grad_outputs(c, T, d, ydt, rdt)
    run_norm_grad(c, o, T, d, scale, eps)
    u = {k: up(v) for k, v in c.items()}
    want = ref.block_norm_grad(u["y"], u["res"], u["w_post"], u["w_pre"], u["gate"], scale, eps,
                               u["dr"], u["dn"])
    # magnitudes: the same formula on absolute values, every minus a plus
    a = {k: None if v is None else v.abs() for k, v in u.items()}
    r, _ = ref.block_norm(u["y"], u["res"], u["w_post"], u["w_pre"], u["gate"], scale, eps)
    p = 0.0
    if u["y"] is not None:
        p = (r - (u["res"] if u["res"] is not None else 0.0)).abs()
    rm = p + (a["res"] if a["res"] is not None else 0.0)  # magnitude in r
    t = a["dr"].clone()
    if u["w_pre"] is not None:
        b = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
        v = a["w_pre"] * a["dn"]
        t = t + b * v + rm * b ** 3 * (v * rm).sum(1, keepdim=True) / d
    one = torch.ones((1, d), dtype=torch.float64)
    e = 4 * (d + 16) * U32
    check(o["dres"], want["dres"], e * t + ref.half_step(rdt) * want["dres"].abs() + 1e-30, "dres")
    col = e + 2 * T * U32
    if o["dw_pre"] is not None:
        check(o["dw_pre"], want["dw_pre"], col * (a["dn"] * rm * b).sum(0) + 1e-30, "dw_pre")
    if u["y"] is not None:
        g, w = (one if a["gate"] is None else a["gate"]), (one if a["w_post"] is None else a["w_post"])
        ay = one[:, :1]
        if u["w_post"] is not None:
            ay = 1 / torch.sqrt((u["y"] ** 2).mean(1, keepdim=True) + eps)
        dp, yh = scale * g * t, a["y"] * ay
        if o["dw_post"] is not None:
            check(o["dw_post"], want["dw_post"], col * (dp * yh).sum(0) + 1e-30, "dw_post")
        if o["dgate"] is not None:
            m = scale * t * w * yh
            m = m if g.shape[0] == T and form[4] == "token" else m.sum(0, keepdim=True)
            check(o["dgate"], want["dgate"],
                  col * m + ref.half_step(ydt) * want["dgate"].abs() + 1e-30, "dgate")
        m = w * dp
        if u["w_post"] is not None:
            m = ay * (m + yh * (m * yh).sum(1, keepdim=True) / d)
        check(o["dy"], want["dy"], e * m + ref.half_step(ydt) * want["dy"].abs() + 1e-30, "dy")
    again = grad_outputs(c, T, d, ydt, rdt)
    run_norm_grad(c, again, T, d, scale, eps)
    for k, v in o.items():
        assert v is None or torch.equal(v, again[k]), k


@pytest.mark.parametrize("form", [NORM_FORMS[1], NORM_FORMS[2]])
@pytest.mark.parametrize("dts", [(BF16, BF16, BF16), (F32, F32, F32)])
def test_block_norm_grad_in_place(gpu_lib, form, dts):
    """dy over y, and dres over dr or over res: the rows fetched ahead are read
    before any row of theirs is written (more rows than workgroups)."""
    T, d = 700, 2056
    ydt, rdt, ndt = dts
    c, scale, eps = norm_case(T, d, form, ydt, rdt, ndt, 17)
    want = grad_outputs(c, T, d, ydt, rdt)
    run_norm_grad(c, want, T, d, scale, eps)
    for over in ("dr", "res"):
        m = dict(c, y=c["y"].clone(), dr=c["dr"].clone(), res=c["res"].clone())
        o = grad_outputs(m, T, d, ydt, rdt)
        o["dy"], o["dres"] = m["y"], m[over]
        run_norm_grad(m, o, T, d, scale, eps)
        for k, v in want.items():
            assert v is None or torch.equal(v, o[k]), (over, k)


def test_block_norm_grad_outputs_may_be_left_out(gpu_lib):
    """Each output alone equals the same output among all; without sums over the
    rows no workspace is needed."""
    T, d = 40, 320
    c, scale, eps = norm_case(T, d, NORM_FORMS[1], BF16, BF16, BF16, 18)
    want = grad_outputs(c, T, d, BF16, BF16)
    run_norm_grad(c, want, T, d, scale, eps)
    for k, v in want.items():
        o = dict.fromkeys(want)
        o[k] = torch.empty_like(v)
        if k in ("dy", "dres"):
            moe.moe_block_norm_grad(c["y"], c["res"], c["dr"], c["dn"], o["dy"], o["dres"], None,
                                    None, None, c["w_post"], c["w_pre"], c["gate"], scale, eps)
        else:
            run_norm_grad(c, o, T, d, scale, eps)
        assert torch.equal(o[k], v), k


def test_block_norm_grad_of_no_rows_is_zero(gpu_lib):
    d = 72
    e = torch.empty((0, d), dtype=BF16, device="cuda")
    w = torch.ones(d, device="cuda")
    dw = [poison((d,), F32) for _ in range(2)]
    dg = poison((1, d), BF16)
    moe.moe_block_norm_grad(e, e, e, e, e.clone(), e.clone(), dw[0], dw[1], dg, w, w,
                            torch.ones((1, d), dtype=BF16, device="cuda"))
    assert (dw[0] == 0).all() and (dw[1] == 0).all() and (dg == 0).all()


def test_block_norm_rows_of_zeros(gpu_lib):
    """A row of zeros has a finite norm (eps) and a finite gradient."""
    d = 256
    z = torch.zeros((2, d), device="cuda")
    w = torch.ones(d, device="cuda")
    r, n = poison((2, d), F32), poison((2, d), F32)
    moe.moe_block_norm(z, z, r, n, w, w)
    assert (r == 0).all() and (n == 0).all()
    c = dict(y=z, res=z, w_post=w, w_pre=w, gate=None, dr=z + 1, dn=z + 1)
    o = grad_outputs(c, 2, d, F32, F32)
    run_norm_grad(c, o, 2, d, 1.0, 1e-6)
    u = {k: up(v) for k, v in c.items()}
    want = ref.block_norm_grad(u["y"], u["res"], u["w_post"], u["w_pre"], None, 1.0, 1e-6, u["dr"],
                               u["dn"])
    for k in ("dres", "dy"):
        check(o[k], want[k], 64 * U32 * want[k].abs(), k)


def test_more_rows_than_one_turn_of_a_grid(gpu_lib):
    """Row-wise calls on more rows than their largest grid takes at once: the
    first and last rows equal the same rows alone."""
    g = gen(90)

    def ends(big, small):
        return torch.equal(torch.cat([big[:3], big[-3:]]), small)

    T, d = (1 << 21) + 5, 8
    x = torch.zeros((T, d), dtype=BF16, device="cuda")
    some = rand(g, 6, d)
    x[:3], x[-3:] = some[:3], some[3:]
    w = torch.ones(d, device="cuda")
    big, small = torch.empty_like(x), torch.empty_like(some)
    moe.moe_block_norm(None, x, None, big, w_pre=w)
    moe.moe_block_norm(None, some, None, small, w_pre=w)
    assert ends(big, small)
    for block_rows, shape in ((1, ((1 << 26) + 7, 16)), (128, ((1 << 22) + 7, 1, 16))):
        x = torch.zeros(shape, dtype=BF16, device="cuda")
        some = rand(g, 6, *shape[1:])
        x[:3], x[-3:] = some[:3], some[3:]
        out = []
        for t in (x, some):
            c = torch.full(t.shape, 9, dtype=torch.uint8, device="cuda")
            s = torch.zeros((*t.shape[:-1], 1), device="cuda")
            moe.moe_blockscale_quantize(t, block_rows, c, s)
            out.append((c, s))
        assert ends(out[0][0], out[1][0]) and ends(out[0][1], out[1][1])
        assert int((out[0][1] == 0).sum()) == 0  # a scale for every block
    del x, out
    P, f = (1 << 21) + 5, 2056
    gu = torch.zeros((P, 2 * f), dtype=BF16, device="cuda")
    some = rand(g, 6, 2 * f)
    gu[:3], gu[-3:] = some[:3], some[3:]
    big, small = (torch.empty((n, f), dtype=BF16, device="cuda") for n in (P, 6))
    moe.moe_swiglu(gu, big)
    moe.moe_swiglu(some, small)
    assert ends(big, small)
    dgu = torch.empty((6, 2 * f), dtype=BF16, device="cuda")
    moe.moe_swiglu_grad(some, small, dgu)
    moe.moe_swiglu_grad(gu, big, gu)
    assert ends(gu, dgu)
