"""moe_layer_few's h between its kernels: all 24 bits where out is float32, 17 of
each value where it is bfloat16.

Exact cases: x = (256, k, 0, ..) and gate and up rows of (16, a) and (16, -b), small
integers, so that gate = 4096 + k a is past 17, where silu(z) is z in float32, and h =
gate * up is an integer below 2^24 that only three bf16 values hold together."""
import pytest
import torch

import int4_routed_expert_logits_amd as moe

pytestmark = pytest.mark.gpu

BF16, F32, F64, F8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
KINDS = ("bf16", "e4m3", "int8")


def say(msg):
    print(msg, flush=True)


def held(w, kind):
    """A matrix [n, R, K] of integers up to 16, as the kind holds it with scales of 1."""
    n, r, k = w.shape
    if kind == "bf16":
        return w.to(BF16).cuda(), None
    if kind == "int8":
        return w.to(torch.int8).cuda(), torch.ones((n, r), device="cuda")
    return w.float().to(F8).cuda(), torch.ones((n, -(-r // 128), -(-k // 128)), device="cuda")


def run(shape, x, experts, idx, w, out):
    T = x.shape[0]
    ws = torch.empty(max(moe.moe_layer_few_workspace_bytes(shape, T), 256), dtype=torch.uint8, device="cuda")
    got = torch.empty((T, shape[0]), dtype=out, device="cuda")
    moe.moe_layer_few(shape, x, None, None, experts, None, idx, w, got, ws)
    return got


def parts(h, n):
    """h as a sum of n bf16 values."""
    total = torch.zeros_like(h)
    for _ in range(n):
        total = total + (h - total).to(BF16).to(h.dtype)
    return total


def case(kind, d, f, T, E, cancel):
    """(x, experts, idx, expected [T, d]) in integers.  Row n of down takes column n % f
    of h, less the next one where `cancel`."""
    g = torch.Generator().manual_seed(d + f + T)
    a = 1 + 2 * torch.randint(0, 4, (E, f), generator=g)
    b = a + 2 * torch.randint(0, 4, (E, f), generator=g)
    gu, dn = torch.zeros((E, 2 * f, d)), torch.zeros((E, d, f))
    gu[:, :, 0] = 16
    gu[:, :f, 1], gu[:, f:, 1] = a.float(), -b.float()
    n = torch.arange(d)
    dn[:, n, n % f] = 1
    if cancel:
        dn[:, n, (n + 1) % f] = -1
    k = 1 + torch.arange(T) % 5
    x = torch.zeros((T, d))
    x[:, 0], x[:, 1] = 256, k.float()
    idx = torch.randint(0, E, (T, 1), generator=g)
    h = ((4096 + k[:, None] * a[idx[:, 0]]) * (4096 - k[:, None] * b[idx[:, 0]])).to(F64)
    assert h.max() < 2 ** 24 and h.min() > 2 ** 23
    want = h[:, n % f] - h[:, (n + 1) % f] if cancel else h[:, n % f]
    (gq, gs), (dq, ds) = held(gu, kind), held(dn, kind)
    return (x.to(BF16).cuda(), (gq, dq) if gs is None else (gq, dq, gs, ds), idx.int().cuda(), h, want)


SIZES = [(64, 64, 1, 1), (192, 320, 3, 2), (512, 128, 9, 4), (320, 1024, 32, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,f,T,E", SIZES)
def test_a_float32_out_holds_all_of_h(gpu_lib, d, f, T, E, kind):
    say(f"parts f32 {kind} {d} {f} {T} {E}")
    for cancel in (False, True):
        x, experts, idx, h, want = case(kind, d, f, T, E, cancel)
        assert (parts(h, 2) != h).any() and (parts(h, 3) == h).all()
        got = run((d, f, E, 1, 64, 0), x, experts, idx, torch.ones((T, 1), device="cuda"), F32)
        assert torch.equal(got.cpu().to(F64), want)  # every product and sum is below 2^24


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,f,T,E", SIZES)
def test_a_bfloat16_out_holds_17_bits_of_each_value_of_h(gpu_lib, d, f, T, E, kind):
    """Also where two of them, 2^24 each, cancel to a few thousand: 2^-17 of each, and
    half a place of the result."""
    say(f"parts bf16 {kind} {d} {f} {T} {E}")
    n = torch.arange(d)
    for cancel in (False, True):
        x, experts, idx, h, want = case(kind, d, f, T, E, cancel)
        got = run((d, f, E, 1, 64, 0), x, experts, idx, torch.ones((T, 1), device="cuda"), BF16)
        off = 2.0 ** -17 * (h[:, n % f] + (h[:, (n + 1) % f] if cancel else 0))
        assert ((got.cpu().to(F64) - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,f,E,k,T", [(6144, 2048, 8, 8, 1), (2048, 512, 24, 8, 3), (2048, 1024, 16, 8, 32),
                                       (320, 192, 5, 2, 7)])
def test_error_of_a_float32_out_as_a_whole(gpu_lib, d, f, E, k, T, kind):
    """Float32 sums of d and f products leave some 4e-7 of the result's norm (each sum
    is some 2^6 partial sums whose roundings, 2^-24 each, are independent); h in two
    parts would leave 2.5e-6, in one 6e-4."""
    say(f"norm {kind} {d} {f} {E} {k} {T}")
    g = torch.Generator(device="cuda").manual_seed(d + T)

    def matrix(n, r, c):
        if kind == "bf16":
            w = torch.randn((n, r, c), generator=g, device="cuda").mul_(0.02).to(BF16)
            return w, None, w.to(F64)
        if kind == "int8":
            w = torch.randint(-127, 128, (n, r, c), generator=g, device="cuda", dtype=torch.int8)
            s = 2e-4 * (1 + torch.rand((n, r), generator=g, device="cuda"))
            return w, s, w.to(F64) * s.to(F64)[:, :, None]
        w = torch.randn((n, r, c), generator=g, device="cuda").mul_(100).clamp_(-448, 448).to(F8)
        s = 2e-4 * (1 + torch.rand((n, -(-r // 128), -(-c // 128)), generator=g, device="cuda"))
        at = lambda m: torch.arange(m, device="cuda") // 128  # noqa: E731
        return w, s, w.float().to(F64) * s.to(F64)[:, at(r)][:, :, at(c)]

    gu, gus, gu64 = matrix(E, 2 * f, d)
    dn, dns, dn64 = matrix(E, d, f)
    x = torch.randn((T, d), generator=g, device="cuda").to(BF16)
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    got = run((d, f, E, k, 64, 0), x, (gu, dn) if gus is None else (gu, dn, gus, dns), idx, w, F32)
    want = torch.zeros((T, d), dtype=F64, device="cuda")
    for t in range(T):
        for j, e in enumerate(idx[t].tolist()):
            gate, up = (gu64[e] @ x[t].to(F64)).chunk(2)
            want[t] += w[t, j].to(F64) * (dn64[e] @ (gate / (1 + torch.exp(-gate)) * up))
    rel = float((got.to(F64) - want).norm() / want.norm())
    say(f"{rel:.2e}")
    assert rel < 1e-6
