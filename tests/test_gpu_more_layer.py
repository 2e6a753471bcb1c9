"""The calls on 8-bit integers, the layer for a few tokens and the AdamW step
together, as layer.py issues them: a layer on bf16 experts is trained, its
weights are quantised, a prompt and then single tokens are served from them;
captured and replayed, on other streams, around norms.

Allowances: each link's rounding of its value, carried on by the magnitudes of
the coefficients behind it (tests/more_ref.py for the few tokens')."""
import pytest
import torch

import block_ref
import int4_routed_expert_logits_amd as moe
import more_ref as ref
from int4_routed_expert_logits_amd import layer as L
from test_gpu_block import BF16, F32, check, gen, rand, say

pytestmark = pytest.mark.gpu

HALF = block_ref.half_step(BF16)
SHAPES = {"shared": moe.Shape(320, 192, 8, 2, 64, 192), "plain": moe.Shape(512, 256, 32, 8, 64, 0)}


def make(sh, T, seed):
    g = gen(seed)
    d, f, E = sh.d, sh.f, sh.n_experts
    ex = L.FloatExperts(rand(g, E, 2 * f, d, scale=d ** -0.5), rand(g, E, d, f, scale=f ** -0.5))
    if sh.f_shared:
        ex.shared_gate_up = rand(g, 1, 2 * f, d, scale=d ** -0.5)
        ex.shared_down = rand(g, 1, d, f, scale=f ** -0.5)
    return rand(g, T, d), rand(g, E, d, dt=F32, scale=0.05), rand(g, E, dt=F32, scale=0.3), ex


def four(ex):
    """(experts, shared) as the plain forms take them."""
    sc, ssc = ex.scales or (None, None), ex.shared_scales or (None, None)
    return (ex.gate_up, ex.down, *sc), None if ex.shared_gate_up is None else (
        ex.shared_gate_up, ex.shared_down, *ssc)


def ints_reference(x, idx, w, ex):
    """The layer on int8 experts for x as its codes stand for it, with what bf16
    gate, up, y and out and h's codes may take the call from it."""
    def ffn(weights, e, v):
        gu = ref.matrix(weights[0][e:e + 1], weights[2][e:e + 1])[0]
        dn = ref.matrix(weights[1][e:e + 1], weights[3][e:e + 1])[0]
        g, u = (v @ gu.T).chunk(2, 1)
        s = 1 / (1 + torch.exp(-g))
        h = g * s * u
        # gate and up off by half a bf16 step each (and their scales' roundings)
        eh = 1.01 * HALF * (h.abs() + (g * s * (1 + g * (1 - s)) * u).abs())
        # the code by half a step of the row's scale, itself off as h's largest is
        top = (h.abs() + eh).amax(1, keepdim=True)
        eh = eh + top / 254 * 1.01
        y = h @ dn.T
        return y, eh @ dn.abs().T + HALF * y.abs()
    experts, shared = four(ex)
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            y, a = ffn(experts, int(idx[t, j]), x[t:t + 1])
            out[t] += w[t, j] * y[0]
            err[t] += w[t, j] * a[0]
    if shared is not None:
        y, a = ffn(shared, 0, x)
        out, err = out + y, err + a
    return out, 1.02 * err + HALF * out.abs() + 1e-6


@pytest.mark.parametrize("T", [1, 7, 40, 300])
@pytest.mark.parametrize("name", list(SHAPES))
def test_layer_on_integer_experts(gpu_lib, name, T):
    say(f"layer int8 {name} T={T}")
    sh = SHAPES[name]
    x, wr, bias, ex = make(sh, T, T)
    q = L.FloatExperts.quantize(ex, ints=True)
    buf = L.FloatLayerBuffers.allocate(sh, T, ints=True)
    L.run_layer_float(x, wr, bias, q, buf)
    xq, xs = buf.codes["x"]
    xv = block_ref.d64(xq) * block_ref.d64(xs)[:, None]
    assert ((xv - block_ref.d64(x)).abs() <= 0.5001 * block_ref.d64(xs)[:, None]).all()
    want, err = ints_reference(xv, buf.topk_idx.cpu(), block_ref.d64(buf.topk_w), q)
    check(buf.out, want, err, "out")


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_few_tokens_through_layer(gpu_lib, name, kind):
    sh = SHAPES[name]
    for T in (1, 6, 32):
        x, wr, bias, ex = make(sh, T, 20 + T)
        if kind != "bf16":
            ex = L.FloatExperts.quantize(ex, ints=kind == "int8")
        buf = L.FewLayerBuffers.allocate(sh, T, out_dtype=F32)
        L.run_layer_few(x, wr, bias, ex, buf)
        want, allow = ref.layer_few(x, buf.topk_idx, buf.topk_w, *four(ex), F32)
        check(buf.out, want, allow, f"{kind} T={T}")
        # routed beforehand: the same bits
        given = L.FewLayerBuffers.allocate(sh, T, out_dtype=F32)
        given.topk_idx.copy_(buf.topk_idx)
        given.topk_w.copy_(buf.topk_w)
        L.run_layer_few(x, None, None, ex, given)
        assert torch.equal(given.out, buf.out)


@pytest.mark.parametrize("name,bits", [("shared", 32), ("shared", 8), ("plain", 32)])
def test_trained_quantised_and_served(gpu_lib, name, bits):
    """Two training steps, then a prompt and single tokens on the new weights, each
    link against the form of its own inputs."""
    sh, T = SHAPES[name], 24
    x, wr, bias, ex = make(sh, T, 7)
    buf = L.FloatLayerBuffers.allocate(sh, T)
    grads = L.FloatLayerGrads.allocate(buf, ex)
    opt = L.AdamW.of_experts(ex, grads, bits)
    dout = rand(gen(3), T, sh.d)
    hyper = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    m = [torch.zeros(p.numel(), dtype=F32).numpy() for p in opt.params]
    v = [a.copy() for a in m]
    p = [w.cpu().view(-1).numpy() for w in opt.masters]
    for step in (1, 2):
        L.run_layer_float(x, wr, bias, ex, buf)
        L.run_layer_float_grad(dout, x, ex, buf, grads)
        opt.step(**hyper)
        for i, g in enumerate(opt.grads):
            p[i], m[i], v[i], r = ref.adamw32(p[i], g.cpu().view(-1).numpy(), m[i], v[i], step, 1e-2,
                                              0.9, 0.95, 1e-8, 0.1)
            new = torch.from_numpy(p[i]).view(opt.params[i].shape)
            assert torch.equal(opt.masters[i].cpu(), new)
            assert torch.equal(opt.params[i].cpu(), new.to(BF16))
            if bits == 8:
                q, s = ref.m_codes(m[i])
                m[i] = q.astype("float32") * s.repeat(256)[:len(q)]
                c, s = ref.v_codes(r)
                v[i] = (ref.root_values()[c].astype("float32") * s.repeat(256)[:len(c)]) ** 2
    assert int(opt.count) == 2
    q = L.FloatExperts.quantize(ex, ints=True)
    assert torch.equal(q.gate_up.cpu().long(), ref.row_quantize(ex.gate_up)[0])
    prompt = L.FloatLayerBuffers.allocate(sh, T, ints=True)
    L.run_layer_float(x, wr, bias, q, prompt)
    xq, xs = prompt.codes["x"]
    want, err = ints_reference(block_ref.d64(xq) * block_ref.d64(xs)[:, None],
                               prompt.topk_idx.cpu(), block_ref.d64(prompt.topk_w), q)
    check(prompt.out, want, err, "prompt")
    few = L.FewLayerBuffers.allocate(sh, 3)
    L.run_layer_few(x[5:8], wr, bias, q, few)
    assert torch.equal(few.topk_idx, prompt.topk_idx[5:8])
    want, allow = ref.layer_few(x[5:8], few.topk_idx, few.topk_w, *four(q), BF16)
    check(few.out, want, allow, "few")


def test_captured_and_replayed(gpu_lib):
    """A token's layer on integers and the optimiser's step in one graph, replayed
    among eager calls."""
    sh = SHAPES["shared"]
    x, wr, bias, ex = make(sh, 2, 9)
    q = L.FloatExperts.quantize(ex, ints=True)
    few, prompt = L.FewLayerBuffers.allocate(sh, 2), L.FloatLayerBuffers.allocate(sh, 2, ints=True)
    g = [rand(gen(4), *ex.down.shape, scale=1e-2)]
    opt = L.AdamW([ex.down], g, bits=8)
    L.run_layer_few(x, wr, bias, q, few)
    L.run_layer_float(x, wr, bias, q, prompt)
    opt.step(0.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run_layer_few(x, wr, bias, q, few)
        L.run_layer_float(x, wr, bias, q, prompt)
        opt.step(1e-3)
    eager = L.AdamW([ex.down.clone()], g, bits=8)
    eager.masters[0].copy_(opt.masters[0])
    for a, b in ((eager.m, opt.m), (eager.v, opt.v), (eager.m_scales, opt.m_scales),
                 (eager.v_scales, opt.v_scales)):
        a[0].copy_(b[0])
    eager.count.copy_(opt.count)
    for i in range(4):
        x.copy_(rand(gen(i), 2, sh.d))
        g[0].copy_(rand(gen(50 + i), *ex.down.shape, scale=1e-2))
        other, wide = L.FewLayerBuffers.allocate(sh, 2), L.FloatLayerBuffers.allocate(sh, 2, ints=True)
        L.run_layer_few(x, wr, bias, q, other)
        L.run_layer_float(x, wr, bias, q, wide)
        eager.step(1e-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(few.out, other.out) and torch.equal(prompt.out, wide.out)
        assert torch.equal(opt.masters[0], eager.masters[0]) and int(opt.count) == int(eager.count)
        assert torch.equal(opt.v[0], eager.v[0])


def test_streams(gpu_lib):
    """Everything issued on a side stream by its argument, and as the current one."""
    sh = SHAPES["plain"]
    x, wr, bias, ex = make(sh, 5, 13)
    want = L.FewLayerBuffers.allocate(sh, 5)
    qi = L.FloatExperts.quantize(ex, ints=True)
    L.run_layer_few(x, wr, bias, qi, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for how in ("argument", "current", "handle"):
        buf = L.FewLayerBuffers.allocate(sh, 5)
        opt = L.AdamW([ex.down.clone()], [rand(gen(1), *ex.down.shape)])
        torch.cuda.synchronize()
        stream = dict(argument=side, current=None, handle=side.cuda_stream)[how]
        with torch.cuda.stream(side if how == "current" else torch.cuda.current_stream()):
            q = L.FloatExperts.quantize(ex, stream, ints=True)
            L.run_layer_few(x, wr, bias, q, buf, stream)
            opt.step(1e-3, stream=stream)
            opt.step(1e-3, stream=stream)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want.out), how
        assert int(opt.count) == 2 and not torch.equal(opt.params[0], ex.down)


def test_block_around_few_tokens(gpu_lib):
    """A block whose layer is run_layer_few, pre and post norm around it."""
    sh = SHAPES["shared"]
    res, wr, bias, ex = make(sh, 4, 15)
    g = gen(2)
    norms = L.BlockNorms(1 + rand(g, sh.d, dt=F32, scale=0.1), 1 + rand(g, sh.d, dt=F32, scale=0.1))
    few = L.FewLayerBuffers.allocate(sh, 4, out_dtype=BF16)
    normed, out = torch.empty_like(res), torch.empty_like(res)
    L.run_block(res, norms, lambda v: L.run_layer_few(v, wr, bias, ex, few), normed, out)
    y, allow = ref.layer_few(normed, few.topk_idx, few.topk_w, *four(ex), BF16)
    check(few.out, y, allow, "layer")
    want, _ = block_ref.block_norm(block_ref.d64(few.out), block_ref.d64(res),
                                   block_ref.d64(norms.w_post), None, None, 1.0, norms.eps)
    check(out, want, 2 * HALF * want.abs() + 1e-5, "block")


def test_layer_of_no_tokens(gpu_lib):
    sh = SHAPES["plain"]
    x, wr, bias, ex = make(sh, 0, 1)
    q = L.FloatExperts.quantize(ex, ints=True)
    assert L.run_layer_few(x, wr, bias, q, L.FewLayerBuffers.allocate(sh, 0)).shape == (0, sh.d)
    buf = L.FloatLayerBuffers.allocate(sh, 0, ints=True)
    assert L.run_layer_float(x, wr, bias, q, buf).shape == (0, sh.d)
