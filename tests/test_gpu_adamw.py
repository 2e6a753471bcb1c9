"""GPU parity of the AdamW step: bit for bit with its documented float32
operations and codes (tests/more_ref.py), and near its float64 form."""
import math

import numpy as np
import pytest
import torch

import int4_routed_expert_logits_amd as moe
import more_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


class State:
    """Tensors of the given sizes on the GPU, offset by `shift` elements in their
    storage."""

    def __init__(self, sizes, store, gdt, bits, seed, shift=0):
        g = gen(seed)
        blocks = [-(-n // 256) for n in sizes]

        def new(n, dt, scale):
            t = torch.randn(n, generator=g) * scale
            if n > 3:
                t[n // 2] = 0
            return t.to(dt)

        def place(t):
            whole = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
            whole[shift:] = t.cuda()
            return whole[shift:]

        full = [new(n, F32, 0.1) for n in sizes]
        self.master = [place(t) for t in full] if store == "master" else None
        self.p = [place(t if store == "f32" else t.to(BF16)) for t in full]
        self.g = [place(new(n, gdt, 1e-2)) for n in sizes]
        m, v = [new(n, F32, 1e-2) for n in sizes], [new(n, F32, 1e-2).square() for n in sizes]
        self.ms = self.vs = None
        if bits == 8:
            mc = [ref.m_codes(t.numpy()) for t in m]
            vc = [ref.v_codes(np.sqrt(t.numpy())) for t in v]
            m = [torch.from_numpy(a).float().to(torch.float8_e4m3fn) for a, _ in mc]
            v = [torch.from_numpy(a) for a, _ in vc]
            self.ms = [torch.from_numpy(s).cuda() for _, s in mc]
            self.vs = [torch.from_numpy(s).cuda() for _, s in vc]
            assert all(len(s) == b for s, b in zip(self.ms, blocks))
        self.m, self.v = [place(t) for t in m], [place(t) for t in v]

    def tensors(self):
        return moe.AdamWTensors(self.p, self.g, self.m, self.v, self.master, self.ms, self.vs)

    def snapshot(self):
        """Host copies: (store, g, m, v) of each tensor as float32 arrays."""
        got = []
        for i, p in enumerate(self.p):
            m, v = self.m[i].float().cpu().numpy(), self.v[i].float().cpu().numpy()
            if self.ms is not None:
                spread = lambda s, n: np.repeat(s.cpu().numpy(), 256)[:n]  # noqa: E731
                m = m * spread(self.ms[i], len(m))
                r = ref.root_values()[self.v[i].cpu().numpy()].astype(np.float32)
                r = r * spread(self.vs[i], len(v))
                v = r * r
            s = p if self.master is None else self.master[i]
            got.append((s.float().cpu().numpy(), self.g[i].float().cpu().numpy(), m, v))
        return got


def step_tensor(n):
    return torch.tensor([n], dtype=torch.int64, device="cuda")


def check(s, before, step, gs=None, h=HYPER):
    args = (step, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"])
    for i, (p, g, m, v) in enumerate(before):
        wp, wm, wv, wr = ref.adamw32(p, g, m, v, *args, gs)
        new = torch.from_numpy(wp)
        if s.master is not None:
            assert torch.equal(s.master[i].cpu(), new)
        assert torch.equal(s.p[i].cpu(), new.to(s.p[i].dtype))
        if s.ms is None:
            assert np.array_equal(s.m[i].cpu().numpy(), wm)
            assert np.array_equal(s.v[i].cpu().numpy(), wv)
        else:
            q, scale = ref.m_codes(wm)
            assert np.array_equal(s.ms[i].cpu().numpy(), scale)
            assert np.array_equal(s.m[i].float().cpu().numpy(), q.astype(np.float32))
            q, scale = ref.v_codes(wr)
            assert np.array_equal(s.vs[i].cpu().numpy(), scale)
            assert np.array_equal(s.v[i].cpu().numpy(), q)
        # the float64 form: each moment three roundings; the quotient ten more of
        # the update (root of v, bias corrections, eps, division, size), p's two
        t = [torch.from_numpy(a.astype(np.float64)) for a in (p, g, m, v)]
        xp, xm, xv = ref.adamw64(*t, *args, 1.0 if gs is None else gs)
        em = 4 * ref.U * (h["beta1"] * t[2].abs() + (1 - h["beta1"]) * t[1].abs() * (gs or 1))
        size = h["lr"] / (1 - h["beta1"] ** step)
        den = torch.sqrt(xv) / math.sqrt(1 - h["beta2"] ** step) + h["eps"]
        allow = size / den * (em + 12 * ref.U * xm.abs()) + 4 * ref.U * (t[0].abs() + size * xm.abs() / den)
        assert ((torch.from_numpy(wp.astype(np.float64)) - xp).abs() <= allow).all()


SIZES = {"one": [1], "blocks": [255, 256, 257, 511, 512, 513, 1, 3, 1025],
         "many": [(7 * i * i) % 301 for i in range(100)], "large": [5000, 70001],
         "empty": [0, 5, 0], "long": [4096 * 600 + 17]}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("store", ["f32", "bf16", "master"])
@pytest.mark.parametrize("gdt", [F32, BF16])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_step(gpu_lib, sizes, gdt, store, bits):
    if sizes == "long" and (gdt == BF16) != (store == "bf16"):
        sizes = "large"
    say(f"adamw {sizes} {store} {gdt} {bits} bits")
    s = State(SIZES[sizes], store, gdt, bits, 5)
    q, gs = s.tensors(), torch.tensor([0.37], device="cuda")
    for step, scale in ((1, None), (2, gs)):
        before = s.snapshot()
        moe.moe_adamw(q, step_tensor(step), grad_scale=scale, **HYPER)
        check(s, before, step, None if scale is None else float(scale))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_addresses_that_are_not_aligned_for_wide_accesses(gpu_lib, shift, bits):
    for store, gdt in (("f32", BF16), ("bf16", F32), ("master", BF16)):
        s = State([300, 1023, 6], store, gdt, bits, shift, shift=shift)
        before = s.snapshot()
        moe.moe_adamw(s.tensors(), step_tensor(7), **HYPER)
        check(s, before, 7)


def test_nothing_beside_the_tensors_is_written(gpu_lib):
    whole = torch.full((5, 1000), 7.0, device="cuda")
    rows = [whole[i][100:613] for i in range(5)]
    rows[1].fill_(0.1)
    q = moe.AdamWTensors([rows[0]], [rows[1]], [rows[2]], [rows[3]])
    moe.moe_adamw(q, step_tensor(1), **HYPER)
    edges = torch.ones((5, 1000), dtype=torch.bool)
    edges[:, 100:613] = False
    assert (whole.cpu()[edges] == 7).all() and (whole[4] == 7).all()
    assert not (whole[0, 100:613] == 7).any()


def test_kinds_mixed_in_one_call_and_their_order(gpu_lib):
    kinds = [("f32", F32, 32), ("master", BF16, 8), ("bf16", BF16, 32), ("bf16", F32, 8),
             ("master", F32, 32)]
    states = [State([700, 33, 256], st, g, b, i) for i, (st, g, b) in enumerate(kinds)]
    n = 3
    none = [None] * n

    def listed(order):
        cat = lambda name: [t for i in order for t in (getattr(states[i], name) or none)]  # noqa: E731
        return moe.AdamWTensors(*(cat(k) for k in ("p", "g", "m", "v", "master", "ms", "vs")))

    before = [s.snapshot() for s in states]
    moe.moe_adamw(listed([3, 0, 4, 2, 1]), step_tensor(3), **HYPER)
    for s, b in zip(states, before):
        check(s, b, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_zeros_and_the_smallest_values(gpu_lib, bits):
    """Blocks of zeros keep scales of 1; tiny roots get code 1, not 0."""
    s = State([768], "f32", F32, bits, 3)
    for t in (s.g[0], s.m[0], s.v[0]):
        t.zero_()
    if bits == 8:
        s.ms[0].fill_(1)
        s.vs[0].fill_(1)
    s.g[0][256] = 1.0
    s.g[0][257:300] = 1e-5
    s.g[0][512:] = 1e-30
    before = s.snapshot()
    moe.moe_adamw(s.tensors(), step_tensor(1), **HYPER)
    check(s, before, 1)
    if bits == 8:
        assert s.vs[0][0] == 1 and s.ms[0][0] == 1 and (s.v[0][:256] == 0).all()
        assert (s.v[0][257:300] == 1).all() and (s.v[0][300:512] == 0).all()


def test_gradients_that_are_not_finite_stay_in_their_place(gpu_lib):
    for bits in (32, 8):
        s, clean = State([1000], "f32", F32, bits, 9), State([1000], "f32", F32, bits, 9)
        s.g[0][300], s.g[0][999] = float("nan"), float("inf")
        moe.moe_adamw(s.tensors(), step_tensor(1), **HYPER)
        moe.moe_adamw(clean.tensors(), step_tensor(1), **HYPER)
        same = torch.ones(1000, dtype=torch.bool, device="cuda")
        same[300], same[999] = False, False
        assert torch.equal(s.p[0][same], clean.p[0][same])
        assert not torch.isfinite(s.p[0][~same]).any()
        if bits == 8:
            assert torch.isnan(s.m[0].float()[~same]).all()
            assert torch.isnan(s.vs[0]).tolist() == [False, True, False, True]
            assert torch.equal(s.ms[0][[0, 2]], clean.ms[0][[0, 2]])


def test_step_numbers(gpu_lib):
    """The powers at far steps, and numbers below 1 as 1."""
    for step, as_ in ((10 ** 9, 10 ** 9), (0, 1), (-5, 1), (2 ** 62, 2 ** 62)):
        s = State([300], "f32", F32, 32, 2)
        before = s.snapshot()
        moe.moe_adamw(s.tensors(), step_tensor(step), **HYPER)
        check(s, before, as_)


def test_betas_of_zero(gpu_lib):
    s = State([300], "f32", F32, 32, 2)
    before = s.snapshot()
    h = dict(HYPER, beta1=0.0, beta2=0.0, weight_decay=0.0)
    moe.moe_adamw(s.tensors(), step_tensor(4), **h)
    check(s, before, 4, h=h)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_with_the_step_advanced_in_the_graph(gpu_lib, bits):
    sizes = [5000, 3, 257]
    s, eager = State(sizes, "master", BF16, bits, 8), State(sizes, "master", BF16, bits, 8)
    q, e = s.tensors(), eager.tensors()
    step, count = step_tensor(0), step_tensor(0)
    moe.load()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        moe.moe_adamw(q, step, **HYPER)
    for i in range(5):
        for a, b in zip(s.g, eager.g):
            a.copy_(torch.randn(a.shape, generator=gen(i)).to(BF16))
            b.copy_(a)
        count += 1
        moe.moe_adamw(e, count, **HYPER)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("p", "master", "m", "v", "ms", "vs"):
            for a, b in zip(getattr(s, name) or (), getattr(eager, name) or ()):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (name, i)


def test_on_another_stream(gpu_lib):
    s, other = State([70000], "f32", F32, 32, 8), State([70000], "f32", F32, 32, 8)
    moe.moe_adamw(s.tensors(), step_tensor(1), **HYPER)
    side = torch.cuda.Stream()
    q, one = other.tensors(), step_tensor(1)
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_adamw(q, one, stream=side, **HYPER)
    side.synchronize()
    assert torch.equal(s.p[0], other.p[0])
