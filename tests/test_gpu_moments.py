"""8-bit moments over many AdamW steps: bit for bit with their plain form
(tests/moments_ref.py), and beside float32 moments at the betas that callers use."""
import numpy as np
import pytest
import torch

import int4_routed_expert_logits_amd as moe
import moments_ref as mom
import more_ref as ref
from int4_routed_expert_logits_amd import layer as L

pytestmark = pytest.mark.gpu

BF16, F32, F8, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
F = np.float32


def say(msg):
    print(msg, flush=True)


def state(n, store, shift=0):
    """(p, master, m, v, m_scales, v_scales) of zeros on the GPU, `shift` elements
    into their storage."""
    new = lambda dt: torch.zeros(n + shift, dtype=dt, device="cuda")[shift:]  # noqa: E731
    ones = lambda: torch.ones(-(-n // 256), device="cuda")  # noqa: E731
    return (new(F32 if store == "f32" else BF16), new(F32) if store == "master" else None, new(F8),
            new(U8), ones(), ones())


@pytest.mark.parametrize("b1,b2", [(0.9, 0.999), (0.9, 0.99), (0.95, 0.95), (0.0, 0.9999), (0.9, 0.9),
                                   (0.9, 0.951), (0.5, 0.95), (0.9, 0.95), (0.8, 0.9), (0.5, 0.9)])
@pytest.mark.parametrize("store,gdt,shift", [("f32", F32, 0), ("master", BF16, 0), ("bf16", F32, 1),
                                            ("f32", BF16, 3)])
def test_steps_are_the_forms(gpu_lib, store, gdt, shift, b1, b2):
    sizes = [1, 255, 256, 257, 3000]
    say(f"moments {store} {gdt} {shift} {b1} {b2}")
    drawn = (b1, b2) not in ((0.9, 0.95), (0.8, 0.9), (0.5, 0.9))
    rng = np.random.default_rng(3)
    states = [state(n, store, shift) for n in sizes]
    grads = [torch.zeros(n + shift, dtype=gdt, device="cuda")[shift:] for n in sizes]
    cat = lambda k: [s[k] for s in states]  # noqa: E731
    q = moe.AdamWTensors(cat(0), grads, cat(2), cat(3), cat(1) if store == "master" else None, cat(4),
                         cat(5))
    want = [(np.zeros(n, F),) * 3 for n in sizes]
    spread = [np.exp(rng.uniform(-9, 0, n)).astype(F) for n in sizes]
    for t in range(1, 41):
        for i, n in enumerate(sizes):
            grads[i].copy_(torch.from_numpy(rng.standard_normal(n).astype(F) * spread[i]))
        step = torch.tensor([t], dtype=torch.int64, device="cuda")
        moe.moe_adamw(q, step, 1e-2, b1, b2, 1e-8, 0.1)
        for i, (p, m, v) in enumerate(want):
            p, m, v, r = ref.adamw32(p, grads[i].float().cpu().numpy(), m, v, t, 1e-2, b1, b2, 1e-8, 0.1)
            (mc, ms), (vc, vs) = (codes(a, t if drawn else None) for codes, a in
                                  ((mom.m_codes, m), (mom.v_codes, r)))
            got = states[i]
            new = torch.from_numpy(p)
            if store == "master":
                assert torch.equal(got[1].cpu(), new), (t, i)
            assert torch.equal(got[0].cpu(), new.to(got[0].dtype)), (t, i)
            assert np.array_equal(got[2].float().cpu().numpy(), mc), (t, i)
            assert np.array_equal(got[3].cpu().numpy(), vc), (t, i)
            assert np.array_equal(got[4].cpu().numpy(), ms) and np.array_equal(got[5].cpu().numpy(), vs)
            m, v = mom.m_of(mc, ms), mom.v_of(vc, vs)
            want[i] = (got[0].float().cpu().numpy() if store == "bf16" else p, m, v)


@pytest.mark.parametrize("kind", mom.KINDS)
@pytest.mark.parametrize("b2", [None, 0.99, 0.9999])
def test_runs_follow_float32_moments(gpu_lib, b2, kind):
    """3000 steps of the class, its default beta2 among them: the update's norm within
    a tenth of the one with float32 moments."""
    n, steps = 2048, 3000
    kw = {} if b2 is None else dict(beta2=b2)
    sizes = torch.exp(torch.rand(n, generator=torch.Generator().manual_seed(1)) * 3 - 8).cuda()
    p, g = [torch.zeros(n, device="cuda") for _ in range(2)], torch.zeros(n, device="cuda")
    opt = [L.AdamW([p[0]], [g], bits=32), L.AdamW([p[1]], [g], bits=8)]
    norms = torch.zeros(2, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    signs = torch.randn(n, generator=gen, device="cuda").sign()
    for t in range(steps):
        if kind == "constant":
            g.copy_(signs * sizes)
        else:
            g.normal_(generator=gen).mul_(sizes)
            if kind == "shrinking" and t >= steps // 3:
                g.mul_(0.05)
        for i in (0, 1):
            p[i].zero_()
            opt[i].step(1.0, **kw)
            if 3 * t >= 2 * steps:
                norms[i] += p[i].square().sum()
        if t % 1000 == 0:
            say(f"step {t}")
    ratio = float(norms[1] / norms[0]) ** 0.5
    say(f"{kind} {b2}: {ratio:.4f}")
    assert abs(ratio - 1) < 0.1


def test_captured_steps_draw_by_their_number(gpu_lib):
    n = 3000
    g = torch.zeros(n, device="cuda")
    p = [torch.zeros(n, device="cuda") for _ in range(2)]
    one, eager = L.AdamW([p[0]], [g], bits=8), L.AdamW([p[1]], [g], bits=8)
    moe.load()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.step(1e-2)
    for i in range(6):
        g.normal_(generator=torch.Generator(device="cuda").manual_seed(i))
        eager.step(1e-2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((one.m, eager.m), (one.v, eager.v), (one.params, eager.params),
                     (one.m_scales, eager.m_scales), (one.v_scales, eager.v_scales)):
            assert torch.equal(a[0].view(U8), b[0].view(U8)), i


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("store", ["f32", "master"])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf"), 1e25])
def test_elements_that_are_not_finite_spoil_no_other(gpu_lib, bad, store, beta2):
    """One step with such gradients (the square of 1e25 is none of float32) and four
    without: the moments by the form, the other parameters as in a clean run."""
    n, at = 1000, [300, 999]
    say(f"not finite {bad} {store} {beta2}")
    same = torch.ones(n, dtype=torch.bool)
    same[at] = False
    runs = []
    for spoilt in (True, False):
        p, w, m, v, ms, vs = state(n, store)
        g = torch.zeros(n, device="cuda")
        q = moe.AdamWTensors([p], [g], [m], [v], [w] if store == "master" else None, [ms], [vs])
        p32, m32, v32 = (np.zeros(n, F),) * 3
        for t in range(1, 6):
            g.normal_(generator=torch.Generator(device="cuda").manual_seed(t)).mul_(1e-2)
            g[::256] = 1.0  # each block's largest
            if spoilt and t == 1:
                g[at] = bad
            step = torch.tensor([t], dtype=torch.int64, device="cuda")
            moe.moe_adamw(q, step, 1e-2, 0.9, beta2, 1e-8, 0.1)
            with np.errstate(all="ignore"):
                p32, m32, v32, r = ref.adamw32(p32, g.cpu().numpy(), m32, v32, t, 1e-2, 0.9, beta2, 1e-8, 0.1)
                draw = None if beta2 == 0.95 else t
                (mc, sm), (vc, sv) = mom.m_codes(m32, draw, 0, r), mom.v_codes(r, draw)
                m32, v32 = mom.m_of(mc, sm), mom.v_of(vc, sv)
            got = (w if store == "master" else p).cpu().numpy()
            assert np.array_equal(got, p32, equal_nan=True), t
            assert np.array_equal(m.float().cpu().numpy(), mc, equal_nan=True), t
            assert np.array_equal(v.cpu().numpy(), vc), t
            assert np.array_equal(vs.cpu().numpy().view(np.uint32), sv.view(np.uint32)), t
        runs.append((p.cpu(), v.cpu(), vs.cpu()))
    (p, v, vs), (p0, v0, _) = runs
    assert torch.isnan(vs).tolist() == [False, True, False, True]
    assert torch.equal(p[same], p0[same]) and torch.equal(v[same], v0[same])
    assert torch.isfinite(p[~same]).all() == (bad == 1e25)


def test_places_past_four_billion(gpu_lib):
    """The last blocks of 2^32 + 600 elements, by the form at their places."""
    n, tail = 2 ** 32 + 600, 600 + 512
    p, _, m, v, ms, vs = state(n, "bf16")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-tail:] = torch.randn(tail, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF16)
    q = moe.AdamWTensors([p], [g], [m], [v], None, [ms], [vs])
    z, first = np.zeros(tail, F), n - tail
    assert first % 256 == 0
    want = (z, z)
    for t in (1, 2):
        moe.moe_adamw(q, torch.tensor([t], dtype=torch.int64, device="cuda"), 1e-2)
        _, wm, wv, r = ref.adamw32(z, g[-tail:].float().cpu().numpy(), *want, t, 1e-2, 0.9, 0.999, 1e-8, 0.0)
        assert np.array_equal(m[-tail:].float().cpu().numpy(), mom.m_codes(wm, t, first)[0])
        assert np.array_equal(v[-tail:].cpu().numpy(), mom.v_codes(r, t, first)[0])
        want = mom.moments(wm, r, t, first)
    assert (m[:first].view(U8) == 0).all() and (v[:first] == 0).all()
