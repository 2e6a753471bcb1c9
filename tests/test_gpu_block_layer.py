"""The calls of include/moe_int4_block.h together, as layer.py issues them:
the layer on bf16 and on 8-bit experts, its gradient, a block with its norms
around either kind of layer; captured and replayed, on other streams.

The references are float64 on the CPU.  A layer's intermediates are stored in
bf16: each link's allowance is its rounding (half_step) of the value, carried
on through the links behind it by the magnitudes of their coefficients.
"""
import functools

import pytest
import torch

import block_ref as ref
import synth
import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import layer as L
from test_gpu_block import BF16, F32, U32, check, gen, rand, say, up
from test_gpu_parity import dev_layer, tokens

pytestmark = pytest.mark.gpu

HALF = ref.half_step(BF16)
SHAPES = {  # d, f, E, k, shared
    "shared": moe.Shape(320, 192, 8, 2, 64, 192),
    "plain": moe.Shape(512, 256, 32, 8, 64, 0),
}


def make(shape, T, seed):
    g = gen(seed)
    d, f, E = shape.d, shape.f, shape.n_experts
    ex = L.FloatExperts(rand(g, E, 2 * f, d, scale=d ** -0.5), rand(g, E, d, f, scale=f ** -0.5))
    if shape.f_shared:
        ex.shared_gate_up = rand(g, 1, 2 * f, d, scale=d ** -0.5)
        ex.shared_down = rand(g, 1, d, f, scale=f ** -0.5)
    return rand(g, T, d), rand(g, E, d, dt=F32, scale=0.05), rand(g, E, dt=F32, scale=0.3), ex


def ffn(x, gu_w, dn_w, gu_err=0.0, h_err=0.0):
    """SwiGLU expert on rows x, and an allowance for gu and h stored with the
    given relative errors and y in bf16."""
    gu = x @ gu_w.T
    g, u = gu.chunk(2, 1)
    s = 1 / (1 + torch.exp(-g))
    h = g * s * u
    dh = gu_err * ((g * s * u).abs() + (g * s * (1 + g * (1 - s)) * u).abs()) + h_err * h.abs()
    y = h @ dn_w.T
    return y, dh @ dn_w.abs().T + HALF * y.abs()


def reference(x, idx, w, ex, k, gu_err, h_err):
    """The layer for the routing (idx, w), with its allowance."""
    x, w = ref.d64(x), ref.d64(w)
    gu, dn = ref.d64(ex.gate_up), ref.d64(ex.down)
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(k):
            e = int(idx[t, j])
            y, a = ffn(x[t:t + 1], gu[e], dn[e], gu_err, h_err)
            out[t] += w[t, j] * y[0]
            err[t] += w[t, j] * a[0]
    if ex.shared_gate_up is not None:
        y, a = ffn(x, ref.d64(ex.shared_gate_up[0]), ref.d64(ex.shared_down[0]), gu_err, h_err)
        out, err = out + y, err + a
    return out, err + HALF * out.abs()


@pytest.mark.parametrize("T", [1, 7, 40, 300])
@pytest.mark.parametrize("name", list(SHAPES))
def test_layer_on_bf16_experts(gpu_lib, name, T):
    say(f"layer bf16 {name} T={T}")
    sh = SHAPES[name]
    x, wr, bias, ex = make(sh, T, T)
    buf = L.FloatLayerBuffers.allocate(sh, T)
    L.run_layer_float(x, wr, bias, ex, buf)
    # the routing is moe_route_union's own, checked elsewhere
    want, err = reference(x, buf.topk_idx.cpu(), buf.topk_w, ex, sh.top_k, HALF, HALF)
    # float32 sums over d and f terms: a hundredth of the roundings counted
    check(buf.out, want, 1.1 * err + 1e-6, "out")


@pytest.mark.parametrize("T", [1, 7, 40, 300])
@pytest.mark.parametrize("name", list(SHAPES))
def test_layer_on_8bit_experts(gpu_lib, name, T):
    """Against the float64 layer on the values that the codes stand for (weights
    and x), h's codes off by a rounding of e4m3 (2^-4 of the value, 2^-10 of the
    scale where subnormal) and the 8-bit sums' 1e-4 of the terms."""
    say(f"layer 8-bit {name} T={T}")
    sh = SHAPES[name]
    x, wr, bias, ex = make(sh, T, 50 + T)
    q = L.FloatExperts.quantize(ex)
    buf = L.FloatLayerBuffers.allocate(sh, T, codes=True)
    L.run_layer_float(x, wr, bias, q, buf)
    val = lambda c, s: None if c is None else ref.dequantize(c, s, 128).cuda()  # noqa: E731
    sgu, sdn = q.shared_scales or (None, None)
    deq = L.FloatExperts(val(q.gate_up, q.scales[0]), val(q.down, q.scales[1]),
                         val(q.shared_gate_up, sgu), val(q.shared_down, sdn))
    xv = ref.dequantize(*buf.codes["x"], 1).cuda()
    want, err = reference(xv, buf.topk_idx.cpu(), buf.topk_w, deq, sh.top_k, 2 * HALF, 2.0 ** -4)
    rms = float(want.square().mean().sqrt())
    check(buf.out, want, 1.2 * err + 2e-2 * rms, "out")


def torch_layer(x, ex, idx, w, k):
    """The layer as float64 torch operations, for autograd."""
    def ffn1(v, gu, dn):
        g, u = (v @ gu.T).chunk(2, -1)
        return (g * torch.sigmoid(g) * u) @ dn.T
    out = []
    for t in range(x.shape[0]):
        o = sum(w[t, j] * ffn1(x[t], ex[0][idx[t, j]], ex[1][idx[t, j]]) for j in range(k))
        if ex[2] is not None:
            o = o + ffn1(x[t], ex[2][0], ex[3][0])
        out.append(o)
    return torch.stack(out)


@pytest.mark.parametrize("name,T", [("shared", 1), ("shared", 33), ("plain", 20), ("shared", 150)])
def test_layer_gradient(gpu_lib, name, T):
    """Every gradient of the chain against autograd of the float64 layer, by
    norms: the chain stores gu, h, y, dy, dh and dgu in bf16 (2^-8 each, at
    random signs) and dx twice more, under 8 * 2^-8 = 3 % together; a wrong link
    is off by the order of the gradient itself.  Each link's own test is
    elementwise."""
    say(f"layer grad {name} T={T}")
    sh = SHAPES[name]
    x, wr, bias, ex = make(sh, T, 100 + T)
    buf = L.FloatLayerBuffers.allocate(sh, T)
    L.run_layer_float(x, wr, bias, ex, buf)
    g = L.FloatLayerGrads.allocate(buf, ex)
    dout = rand(gen(7), T, sh.d)
    L.run_layer_float_grad(dout, x, ex, buf, g)
    leaves = [None if t is None else ref.d64(t).requires_grad_() for t in (
        x, ex.gate_up, ex.down, ex.shared_gate_up, ex.shared_down, buf.topk_w)]
    y = torch_layer(leaves[0], leaves[1:5], buf.topk_idx.cpu().long(), leaves[5], sh.top_k)
    (y * ref.d64(dout)).sum().backward()
    for what, got, leaf in zip(("dx", "dgate_up", "ddown", "dshared_gate_up", "dshared_down",
                                "dtopk_w"),
                               (g.dx, g.dgate_up, g.ddown, g.dshared_gate_up, g.dshared_down,
                                g.dtopk_w), leaves):
        if leaf is None:
            assert got is None
            continue
        off = float((ref.d64(got) - leaf.grad).norm() / leaf.grad.norm())
        say(f"  {what}: {off:.4f} of its norm off")
        assert off <= 8 * HALF, what


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_block_around_a_layer(gpu_lib, kind):
    """Pre norm, layer, post norm with gate, scale and residual, and the next
    block's pre norm: against the same done on the layer's own output."""
    T = 5
    if kind == "int4":
        Lr, dev = dev_layer(6)
        sh = moe.shape_of(Lr.shape)
        buf = L.LayerBuffers.allocate(sh, T, moe.MOE_PATH_DECODE_F32)
        layer = functools.partial(L.run_layer, w_router=dev["w_router"], bias=dev["bias"],
                                  experts=dev["experts"], shared=dev["shared"], buf=buf)
    else:
        sh = SHAPES["shared"]
        x, wr, bias, ex = make(sh, T, 3)
        buf = L.FloatLayerBuffers.allocate(sh, T)
        layer = functools.partial(L.run_layer_float, w_router=wr, bias=bias, experts=ex, buf=buf)
    g, d = gen(8), sh.d
    odt = buf.out.dtype
    w = [1 + rand(g, d, dt=F32, scale=0.1) for _ in range(3)]
    gate = rand(g, 1, d, dt=odt)
    norms = L.BlockNorms(w[0], w[1], gate, 0.5, 1e-5)
    res = rand(g, T, d)
    normed, res_out, nxt = (torch.empty((T, d), dtype=BF16, device="cuda") for _ in range(3))
    L.run_block(res, norms, layer, normed, res_out, L.BlockNorms(w[2], eps=1e-5), nxt)
    _, wn = ref.block_norm(None, up(res), None, up(w[0]), None, 1.0, 1e-5)
    check(normed, wn, (HALF + (d + 16) * U32) * wn.abs(), "normed")
    alone = layer(normed).clone()
    assert torch.equal(alone, buf.out)
    wr, wn = ref.block_norm(up(buf.out), up(res), up(w[1]), up(w[2]), up(gate), 0.5, 1e-5)
    small = (d + 32) * U32
    check(res_out, wr, HALF * wr.abs() + small * ((wr - up(res)).abs() + wr.abs()) + 1e-6, "res")
    check(nxt, wn, HALF * wn.abs() + 4 * small * wn.abs() + 1e-5, "next")


def test_block_without_a_post_norm_takes_the_next_eps(gpu_lib):
    """eps decides these norms: the rows' squares are far below it."""
    T, d = 3, 64
    g = gen(21)
    res, out = rand(g, T, d, scale=1e-3), rand(g, T, d, scale=1e-3)
    w = [1 + rand(g, d, dt=F32, scale=0.1) for _ in range(2)]
    normed, res_out, nxt = (torch.empty((T, d), dtype=BF16, device="cuda") for _ in range(3))
    L.run_block(res, L.BlockNorms(w[0], eps=1e-2), lambda n: out, normed, res_out,
                L.BlockNorms(w[1], eps=1e-4), nxt)
    wr, wn = ref.block_norm(up(out), up(res), None, up(w[1]), None, 1.0, 1e-4)
    # three float32 roundings of r and the d squares of its sum
    check(res_out, wr, (HALF + 3 * U32) * wr.abs(), "res")
    check(nxt, wn, (HALF + 3 * U32) * wn.abs() + (d + 16) * U32 * wn.abs() + 1e-9, "next")


def test_layer_of_no_tokens(gpu_lib):
    """T = 0: nothing to route, empty outputs, zero gradients of every weight."""
    sh = SHAPES["shared"]
    x, wr, bias, ex = make(sh, 0, 70)
    b = L.FloatLayerBuffers.allocate(sh, 0)
    assert L.run_layer_float(x, wr, bias, ex, b).shape == (0, sh.d)
    g = L.FloatLayerGrads.allocate(b, ex)
    for t in (g.dgate_up, g.ddown, g.dshared_gate_up, g.dshared_down):
        t.fill_(7.0)
    L.run_layer_float_grad(rand(gen(71), 0, sh.d), x, ex, b, g)
    for t in (g.dgate_up, g.ddown, g.dshared_gate_up, g.dshared_down):
        assert (t == 0).all()
    q = L.FloatLayerBuffers.allocate(sh, 0, codes=True)
    assert L.run_layer_float(x, wr, bias, L.FloatExperts.quantize(ex), q).shape == (0, sh.d)


def test_captured_and_replayed(gpu_lib):
    """Forward (bf16 and 8-bit), gradient and norms in one graph, replayed over
    new inputs between eager runs of the same calls: every replay equals them."""
    sh, T = SHAPES["shared"], 24
    x, wr, bias, ex = make(sh, T, 9)
    q = L.FloatExperts.quantize(ex)
    dout = rand(gen(10), T, sh.d)
    w = torch.ones(sh.d, device="cuda")

    def program():
        o = dict(f=L.FloatLayerBuffers.allocate(sh, T), c=L.FloatLayerBuffers.allocate(sh, T, True))
        o["g"] = L.FloatLayerGrads.allocate(o["f"], ex)
        ws = torch.empty(moe.moe_block_norm_grad_workspace_bytes(T, sh.d), dtype=torch.uint8,
                         device="cuda")
        n = [torch.empty_like(x) for _ in range(4)]
        dw = [torch.empty(sh.d, device="cuda") for _ in range(2)]

        def run():
            L.run_layer_float(x, wr, bias, ex, o["f"])
            L.run_layer_float(x, wr, bias, q, o["c"])
            L.run_layer_float_grad(dout, x, ex, o["f"], o["g"])
            moe.moe_block_norm(o["f"].out, x, n[0], n[1], w, w)
            moe.moe_block_norm_grad(o["f"].out, x, dout, n[1], n[2], n[3], *dw, None, w, w,
                                    workspace=ws)

        outs = [o["f"].out, o["c"].out, o["g"].dx, o["g"].dgate_up, o["g"].ddown,
                o["g"].dshared_gate_up, o["g"].dtopk_w, *n, *dw]
        return run, outs

    run, outs = program()
    run()  # loads every kernel before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    eager, want = program()
    for rep in range(4):
        x.copy_(rand(gen(20 + rep), T, sh.d))
        for t in outs:
            t.fill_(3.0)
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (rep, i)


def test_streams(gpu_lib):
    """Two layers on two streams at once, each with its own buffers and
    workspace, give what each gives alone; `stream` overrides the current one."""
    sh, T = SHAPES["plain"], 64
    jobs = []
    for i in range(2):
        x, wr, bias, ex = make(sh, T, 30 + i)
        dout = rand(gen(40 + i), T, sh.d)
        b = [L.FloatLayerBuffers.allocate(sh, T) for _ in range(2)]
        g = [L.FloatLayerGrads.allocate(b[0], ex) for _ in range(2)]
        jobs.append((x, wr, bias, ex, dout, b, g))
    for x, wr, bias, ex, dout, b, g in jobs:
        L.run_layer_float(x, wr, bias, ex, b[0])
        L.run_layer_float_grad(dout, x, ex, b[0], g[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for rep in range(5):
        for s, (x, wr, bias, ex, dout, b, g) in zip(streams, jobs):
            L.run_layer_float(x, wr, bias, ex, b[1], stream=s)
            with torch.cuda.stream(s):
                L.run_layer_float_grad(dout, x, ex, b[1], g[1])
        torch.cuda.synchronize()
        for x, wr, bias, ex, dout, b, g in jobs:
            assert torch.equal(b[0].out, b[1].out)
            for name in ("dx", "dgate_up", "ddown", "dtopk_w"):
                assert torch.equal(getattr(g[0], name), getattr(g[1], name)), name


def test_padded_batch(gpu_lib):
    """Tokens routed nowhere (every expert id out of range) leave their rows of
    every buffer as they were, get zero from the combine, and pass zero back."""
    sh, T = moe.Shape(320, 192, 8, 2, 64, 0), 12
    x, wr, bias, ex = make(sh, T, 60)
    b = L.FloatLayerBuffers.allocate(sh, T)
    L.run_layer_float(x, wr, bias, ex, b)
    full = b.out.clone()
    pad = torch.arange(T, device="cuda") % 3 == 1
    b.topk_idx[pad] = -1
    moe.moe_union(sh, T, b.topk_idx, b.counts, b.offsets, b.perm, b.inv_perm, b.active, b.n_active)
    used = int((~pad).sum()) * 2
    assert int(b.n_rows) == used
    for t in (b.gu, b.h, b.y):
        t.fill_(7.0)
    moe.moe_grouped_mm(x, ex.gate_up, b.offsets, b.gu, b.perm, 2)
    moe.moe_swiglu(b.gu, b.h, b.n_rows)
    moe.moe_grouped_mm(b.h, ex.down, b.offsets, b.y)
    moe.moe_combine(sh, b.y, None, b.inv_perm, b.topk_w, b.out)
    assert torch.equal(b.out[~pad], full[~pad]) and (b.out[pad] == 0).all()
    for t in (b.gu, b.h, b.y):
        assert (t[used:] == 7).all()
    g = L.FloatLayerGrads.allocate(b, ex)
    for t in (g.dy, g.dh, g.dgu, g.dx_slots):
        t.fill_(7.0)
    L.run_layer_float_grad(rand(gen(61), T, sh.d), x, ex, b, g)
    for t in (g.dy, g.dh, g.dgu, g.dx_slots):
        assert (t[used:] == 7).all()
    assert (g.dx[pad] == 0).all() and (g.dtopk_w[pad] == 0).all()
    assert torch.isfinite(g.dgate_up).all() and torch.isfinite(g.ddown).all()


def test_binding_refuses_what_it_cannot_address(gpu_lib):
    """Strided, misplaced and mistyped tensors never reach a kernel."""
    x, w = torch.zeros((4, 64), dtype=BF16, device="cuda"), torch.zeros((2, 32, 64), dtype=BF16,
                                                                         device="cuda")
    off, y = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros((4, 32), device="cuda")
    with pytest.raises(ValueError, match="w is not contiguous"):
        moe.moe_grouped_mm(x, torch.zeros((2, 64, 32), dtype=BF16, device="cuda").transpose(1, 2),
                           off, y)
    with pytest.raises(ValueError, match="offsets is on cpu"):
        moe.moe_grouped_mm(x, w, off.cpu(), y)
    with pytest.raises(ValueError, match="offsets has shape"):
        moe.moe_grouped_mm(x, w, off[:2], y)
    with pytest.raises(TypeError, match="rows is torch.int64"):
        moe.moe_grouped_mm(x, w, off, y, rows=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(moe.MoeError, match="MOE_ERR_SHAPE"):
        moe.moe_grouped_mm(x, w, off, y, rows_div=2)
    with pytest.raises(moe.MoeError, match="MOE_ERR_ALIGN"):
        moe.moe_grouped_mm(torch.zeros(4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(4, 64), w,
                           off, y)


def test_large_offsets(gpu_lib):
    """Rows whose byte offset passes 2^31 and 2^32: the last rows of a long x,
    y and dy against the same rows alone."""
    K, N, X = 4096, 8, 600_000  # x: 4.9 GB
    x = torch.zeros((X, K), dtype=BF16, device="cuda")
    g = gen(70)
    tail = rand(g, 40, K)
    x[X - 40:] = tail
    w = rand(g, 2, N, K, scale=0.1)
    rows = torch.arange(X - 40, X, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 25, 40], dtype=torch.int32, device="cuda")
    far, near = (torch.empty((40, N), device="cuda") for _ in range(2))
    moe.moe_grouped_mm(x, w, off, far, rows, 1)
    moe.moe_grouped_mm(tail, w, off, near)
    assert torch.equal(far, near)
    # the whole of it as positions of one group, and of the last of two
    y = torch.empty((X, N), device="cuda")
    ends = torch.tensor([0, X - 40, X], dtype=torch.int32, device="cuda")
    moe.moe_grouped_mm(x, w, ends, y)
    alone = torch.empty((40, N), device="cuda")
    moe.moe_grouped_mm(tail, w[1:].contiguous(), torch.tensor([0, 40], dtype=torch.int32,
                                                              device="cuda"), alone)
    want, mag = ref.grouped_mm(tail, w[1:], [0, 40], 40)
    check(y[X - 40:], want, K * U32 * mag + 1e-30, "last rows")
    assert (y[:X - 40] == 0).all()
    dw = torch.empty((2, N, K), device="cuda")
    ws = torch.empty(max(256, moe.moe_grouped_mm_dw_workspace_bytes(2, X, N, K)), dtype=torch.uint8,
                     device="cuda")
    dy = rand(g, 1, N).expand(X, N).contiguous()
    moe.moe_grouped_mm_dw(dy, x, ends, dw, ws)
    want, mag = ref.grouped_mm_dw(dy[X - 40:], tail, [0, 0, 40], 2)
    assert (dw[0] == 0).all()
    check(dw[1:], want[1:], (40 + 64) * U32 * mag[1:] + 2.0 ** -24 * want[1:].abs() + 1e-30, "dw")
