"""Arrays past 4 GB: what lies at their end is computed as it is alone."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe

pytestmark = pytest.mark.gpu

BF16, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(shape, seed):
    return torch.randint(-128, 128, shape, generator=gen(seed), device="cuda", dtype=I8)


def test_rows_to_codes(gpu_lib):
    K = 4096
    rows = 2 ** 32 // K + 5  # 2^32 codes and some: 8.6 GB of bf16, 4.3 GB of codes
    x = torch.empty((rows, K), dtype=BF16, device="cuda").fill_(1.0)
    x[-7:] = torch.randn((7, K), generator=gen(1), device="cuda").to(BF16)
    q, s = torch.empty((rows, K), dtype=I8, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_rowscale_quantize(x, q, s)
    alone, scales = torch.empty((7, K), dtype=I8, device="cuda"), torch.empty(7, device="cuda")
    moe.moe_rowscale_quantize(x[-7:], alone, scales)
    assert torch.equal(q[-7:], alone) and torch.equal(s[-7:], scales)
    assert (q[:3] == 127).all() and (q[-12:-7] == 127).all()


def test_swiglu_to_codes(gpu_lib):
    f = 4096
    P = 2 ** 31 // f + 3  # gate and up: 8.6 GB of bf16
    gu = torch.zeros((P, 2 * f), dtype=BF16, device="cuda")
    gu[-5:] = torch.randn((5, 2 * f), generator=gen(2), device="cuda").to(BF16)
    q, s = torch.empty((P, f), dtype=I8, device="cuda"), torch.empty(P, device="cuda")
    moe.moe_swiglu_rowscale(gu, q, s)
    alone, scales = torch.empty((5, f), dtype=I8, device="cuda"), torch.empty(5, device="cuda")
    moe.moe_swiglu_rowscale(gu[-5:].clone(), alone, scales)
    assert torch.equal(q[-5:], alone) and torch.equal(s[-5:], scales)
    assert (q[:5] == 0).all() and (s[:5] == 1).all()


@pytest.mark.parametrize("P", [5, 300])
def test_integer_products(gpu_lib, P):
    """The last of 261 experts (4.4 GB); few rows and tiles."""
    E, N, K = 261, 4096, 4112
    w = codes((E, N, K), 3)
    ws = torch.rand((E, N), generator=gen(4), device="cuda")
    x, xs = codes((P, K), 5), torch.rand(P, generator=gen(6), device="cuda")
    offsets = torch.zeros(E + 1, dtype=I32, device="cuda")
    offsets[E] = P
    y, alone = torch.empty((P, N), device="cuda"), torch.empty((P, N), device="cuda")
    moe.moe_rowscale_mm(x, xs, w, ws, offsets, y)
    moe.moe_rowscale_mm(x, xs, w[E - 1:], ws[E - 1:], torch.tensor([0, P], dtype=I32, device="cuda"),
                        alone)
    assert torch.equal(y, alone)  # exact sums: the same bits whichever kernel


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_layer_for_a_few_tokens(gpu_lib, kind):
    """The last expert of 96 (bf16) or 176 (codes) of 4096 x 4096: its down weights begin
    3.2 or 2.9 GB in, gate and up 6.4 or 5.9 GB."""
    d = f = 4096
    E, T, k = (96 if kind == "bf16" else 176), 3, 2
    n = E * 2 * f * d
    if kind == "bf16":
        gu = torch.empty((E, 2 * f, d), dtype=BF16, device="cuda").normal_(0, d ** -0.5, generator=gen(7))
        dn = torch.empty((E, d, f), dtype=BF16, device="cuda").normal_(0, f ** -0.5, generator=gen(8))
        sc = ()
    else:
        gu, dn = codes((E, 2 * f, d), 7), codes((E, d, f), 8)
        if kind == "e4m3":
            for w in (gu, dn):
                w.bitwise_and_(-17)  # without that bit no code is NaN
            gu, dn = gu.view(torch.uint8).view(torch.float8_e4m3fn), dn.view(torch.uint8).view(torch.float8_e4m3fn)
            sc = tuple(torch.rand(s, generator=gen(9), device="cuda").add_(0.5).mul_(1e-3)
                       for s in ((E, 2 * f // 128, d // 128), (E, d // 128, f // 128)))
        else:
            sc = tuple(torch.rand(s, generator=gen(9), device="cuda").add_(0.5).mul_(1e-3)
                       for s in ((E, 2 * f), (E, d)))
    assert n * gu.element_size() > 2 ** 32
    x = torch.randn((T, d), generator=gen(10), device="cuda").to(BF16)
    idx = E - 1 - torch.tensor([[0, 4], [2, 0], [0, 5]], dtype=I32, device="cuda")
    w = torch.rand((T, k), generator=gen(11), device="cuda")

    def run(experts, E, idx):
        shape = (d, f, E, k, 64, 0)
        ws = torch.empty(moe.moe_layer_few_workspace_bytes(shape, T), dtype=torch.uint8, device="cuda")
        out = torch.empty((T, d), device="cuda")
        moe.moe_layer_few(shape, x, None, None, experts, None, idx, w, out, ws)
        return out

    got = run((gu, dn, *sc), E, idx)
    last = tuple(t[E - 6:].clone() for t in (gu, dn, *sc))
    want = run(last, 6, idx - (E - 6))
    assert torch.isfinite(got).all()
    # no fewer experts than pairs either way, so the same layout and the same sums
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [32, 8])
def test_optimiser_step(gpu_lib, bits):
    """A tensor past 2^32 bytes of each array: its last blocks as on their own."""
    n = 2 ** 30 + 600 if bits == 32 else 2 ** 32 + 600
    tail = 600 + 512  # whole blocks
    new = lambda dt: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    p, g = new(BF16 if bits == 8 else F32), new(BF16 if bits == 8 else F32)
    g[-tail:] = torch.randn(tail, generator=gen(12), device="cuda").to(g.dtype)
    p[-tail:] = torch.randn(tail, generator=gen(13), device="cuda").to(p.dtype)
    if bits == 8:
        m, v = new(torch.float8_e4m3fn), new(torch.uint8)
        ms, vs = ([torch.ones(-(-n // 256), device="cuda")] for _ in range(2))
    else:
        m, v, ms, vs = new(F32), new(F32), None, None
    small = [t[-tail:].clone() for t in (p, g, m, v)]
    scales = [None if q is None else [torch.ones(-(-tail // 256), device="cuda")] for q in (ms, vs)]
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    for q in (moe.AdamWTensors([p], [g], [m], [v], None, ms, vs),
              moe.AdamWTensors(*([t] for t in small), None, *scales)):
        moe.moe_adamw(q, step, 1e-2, 0.9, 0.95, 1e-8, 0.1)
    for whole, alone in zip((p, m, v), (small[0], small[2], small[3])):
        assert torch.equal(whole[-tail:].view(torch.uint8), alone.view(torch.uint8))
    assert (p[:n - tail] == 0).all()
