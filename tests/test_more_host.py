"""Host-side checks of the calls on 8-bit integers, of the layer for a few tokens
and of the AdamW step (no GPU needed): every call below has at least one defect,
or no work, so none reaches a kernel launch.  Then the plain forms the GPU
tests compare with, against differences, hand-worked values and torch's own
optimiser, and what layer.py sees to."""
import ctypes

import numpy as np
import pytest
import torch

import int4_routed_expert_logits_amd as moe
import more_ref as ref
from int4_routed_expert_logits_amd import _binding as B
from int4_routed_expert_logits_amd import layer as L

P = 1 << 20  # a 256-byte aligned stand-in address (never dereferenced)
MIS = P + 4
F, H = B.MOE_F32, B.MOE_BF16
NULL, SHAPE, DTYPE, ALIGN = B.MOE_ERR_NULL, B.MOE_ERR_SHAPE, B.MOE_ERR_DTYPE, B.MOE_ERR_ALIGN
UNSUPPORTED, WORKSPACE = B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def edit(args, **kw):
    out = dict(args)
    out.update(kw)
    return list(out.values())


# ----------------------------------------------------------------------------
# 8-bit integers
# ----------------------------------------------------------------------------

MM = dict(E=4, P=16, N=64, K=128, xq=P, xs=P, x_rows=16, rows=None, div=1, wq=P, ws=P, off=P, y=P,
          dt=H, s=None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), SHAPE), (dict(E=-1), SHAPE), (dict(P=-1), SHAPE), (dict(N=0), SHAPE),
    (dict(N=4), SHAPE), (dict(K=0), SHAPE), (dict(K=136), SHAPE), (dict(E=1025), UNSUPPORTED),
    (dict(P=(1 << 24) + 1), UNSUPPORTED), (dict(N=65544), UNSUPPORTED), (dict(K=65552), UNSUPPORTED),
    (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE), (dict(div=2), SHAPE), (dict(x_rows=15), SHAPE),
    (dict(x_rows=-1), SHAPE), (dict(rows=P, div=0), SHAPE), (dict(rows=P, div=257), UNSUPPORTED),
    (dict(rows=P, div=256, x_rows=65537), UNSUPPORTED), (dict(rows=P + 1), ALIGN),
    (dict(xq=None), NULL), (dict(xs=None), NULL), (dict(wq=None), NULL), (dict(ws=None), NULL),
    (dict(off=None), NULL), (dict(y=None), NULL), (dict(xq=MIS), ALIGN), (dict(wq=MIS), ALIGN),
    (dict(y=MIS), ALIGN), (dict(ws=MIS), ALIGN), (dict(xs=P + 2), ALIGN), (dict(off=P + 2), ALIGN)])
def test_rowscale_mm_refusals(lib, kw, status):
    assert lib.moe_rowscale_mm(*edit(MM, **kw)) == status


def test_rowscale_mm_of_no_rows(lib):
    assert lib.moe_rowscale_mm(*edit(MM, P=0, x_rows=0, xq=None, xs=None, wq=None, y=None)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), SHAPE), (dict(K=8), SHAPE), (dict(K=0), SHAPE), (dict(K=65552), UNSUPPORTED),
    (dict(dt=9), DTYPE), (dict(x=None), NULL), (dict(c=None), NULL), (dict(sc=None), NULL),
    (dict(x=MIS), ALIGN), (dict(c=MIS), ALIGN), (dict(sc=P + 2), ALIGN), (dict(R=0, x=None), 0)])
def test_rowscale_quantize_refusals(lib, kw, status):
    a = dict(R=4, K=128, x=P, dt=H, c=P, sc=P, s=None)
    assert lib.moe_rowscale_quantize(*edit(a, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(P=-1), SHAPE), (dict(f=0), SHAPE), (dict(f=24), SHAPE), (dict(f=32784), UNSUPPORTED),
    (dict(P=(1 << 24) + 1), UNSUPPORTED), (dict(dt=5), DTYPE), (dict(gu=None), NULL),
    (dict(c=None), NULL), (dict(sc=None), NULL), (dict(gu=MIS), ALIGN), (dict(c=MIS), ALIGN),
    (dict(sc=P + 2), ALIGN), (dict(n=P + 2), ALIGN), (dict(P=0, gu=None), 0)])
def test_swiglu_rowscale_refusals(lib, kw, status):
    a = dict(P=4, f=64, gu=P, dt=H, c=P, sc=P, n=None, s=None)
    assert lib.moe_swiglu_rowscale(*edit(a, **kw)) == status


def test_row_codes_by_hand():
    """absmax 127 gives a scale of one; half-way points go to the even code."""
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, -126.6, 2.49, 0, 0], [0.0] * 8])
    c, s = ref.row_quantize(x)
    one = np.float32(127) * np.float32(1 / 127)
    assert one == 1 and s.tolist() == [1.0, 1.0]
    assert c[0].tolist() == [127, 0, 2, -2, -127, 2, 0, 0] and not c[1].any()


def test_rowscale_mm_form_against_a_loop():
    g = torch.Generator().manual_seed(1)
    xq = torch.randint(-128, 128, (3, 16), generator=g).to(torch.int8)
    wq = torch.randint(-128, 128, (2, 8, 16), generator=g).to(torch.int8)
    xs, ws = torch.rand(3, generator=g), torch.rand((2, 8), generator=g)
    rows = torch.tensor([4, 0, -1, 2])
    y = ref.rowscale_mm(xq, xs, wq, ws, torch.tensor([0, 1, 4]), 4, torch.float32, rows, 2)
    for p, (e, r) in enumerate([(0, 2), (1, 0), (1, None), (1, 1)]):
        for n in range(8):
            want = 0.0 if r is None else np.float32(np.float32(
                int((xq[r].long() * wq[e, n].long()).sum())) * xs[r].numpy()) * ws[e, n].numpy()
            assert float(y[p, n]) == want


# ----------------------------------------------------------------------------
# the layer for a few tokens
# ----------------------------------------------------------------------------

def weights(gu=P, dn=P, gus=None, dns=None):
    return ctypes.byref(B.ExpertWeights(gu, dn, gus, dns))


CODES = weights(gus=P, dns=P)
OK = B.Shape(512, 256, 8, 2, 64, 0)
SHARED = B.Shape(512, 256, 8, 2, 64, 256)
FEW = dict(sh=ctypes.byref(OK), T=4, x=P, wr=None, bias=None, kind=0, ex=weights(), shared=None,
           idx=P, w=P, out=P, dt=H, ws=P, n=1 << 40, s=None)


@pytest.mark.parametrize("kw,status", [
    (dict(sh=None), NULL), (dict(T=-1), SHAPE), (dict(T=33), UNSUPPORTED),
    (dict(sh=ctypes.byref(B.Shape(512, 256, 64, 32, 64, 0)), T=9), UNSUPPORTED),
    (dict(sh=ctypes.byref(B.Shape(96, 256, 8, 2, 64, 0))), SHAPE),
    (dict(sh=ctypes.byref(B.Shape(512, 256, 8, 2, 64, 128))), UNSUPPORTED),
    (dict(dt=7), DTYPE), (dict(kind=3), DTYPE), (dict(kind=-1), DTYPE), (dict(x=None), NULL),
    (dict(ex=None), NULL), (dict(idx=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), NULL), (dict(bias=P), NULL), (dict(shared=weights()), NULL),
    (dict(sh=ctypes.byref(SHARED)), NULL), (dict(ex=weights(gu=None)), NULL),
    (dict(ex=weights(dn=None)), NULL), (dict(ex=CODES), NULL), (dict(kind=1), NULL),
    (dict(kind=2, ex=weights(gus=P)), NULL), (dict(kind=1, ex=weights(dns=P)), NULL),
    (dict(sh=ctypes.byref(SHARED), shared=weights(dn=None)), NULL),
    (dict(x=MIS), ALIGN), (dict(wr=MIS), ALIGN), (dict(wr=P, bias=P + 1), ALIGN),
    (dict(idx=P + 2), ALIGN), (dict(w=P + 1), ALIGN), (dict(out=MIS), ALIGN), (dict(ws=P + 64), ALIGN),
    (dict(ex=weights(gu=MIS)), ALIGN), (dict(ex=weights(dn=MIS)), ALIGN),
    (dict(kind=2, ex=weights(gus=MIS, dns=P)), ALIGN), (dict(kind=1, ex=weights(gus=P + 2, dns=P)), ALIGN),
    (dict(T=0, x=None, ex=None), 0)])
def test_layer_few_refusals(lib, kw, status):
    assert lib.moe_layer_few(*edit(FEW, **kw)) == status


def test_layer_few_workspace(lib):
    for sh, T in ((OK, 1), (SHARED, 32), (B.Shape(64, 8192, 4, 4, 64, 8192), 32)):
        n = moe.moe_layer_few_workspace_bytes(sh, T)
        assert 0 < n < 1 << 28 and n % 256 == 0
        a = dict(FEW, sh=ctypes.byref(sh), T=T, shared=weights() if sh.f_shared else None)
        assert lib.moe_layer_few(*edit(a, n=n - 1)) == WORKSPACE
    for T in (0, -1, 33, 2 ** 40, -2 ** 40):
        assert moe.moe_layer_few_workspace_bytes(OK, T) == 0
    assert moe.moe_layer_few_workspace_bytes(B.Shape(100, 64, 4, 2, 64, 0), 1) == 0


def test_layer_few_form_against_a_loop():
    """One token through two experts, scalar by scalar, on each kind of weights."""
    g = torch.Generator().manual_seed(2)
    d, f, n = 4, 3, 3
    x = torch.randn((1, d), generator=g).to(BF16)
    gu, dn = torch.randn((n, 2 * f, d), generator=g), torch.randn((n, d, f), generator=g)
    idx, w = torch.tensor([[2, 0]]), torch.tensor([[0.7, 0.3]])
    ints = [torch.randint(-99, 99, t.shape, generator=g).to(torch.int8) for t in (gu, dn)]
    scales = [torch.rand(t.shape[:2], generator=g) for t in (gu, dn)]
    codes = [t.to(torch.float8_e4m3fn) for t in (gu, dn)]
    one = [torch.rand((n, 1, 1), generator=g) for _ in range(2)]
    for weights_, val in (((gu.to(BF16), dn.to(BF16)), (gu.to(BF16).double(), dn.to(BF16).double())),
                          ((*ints, *scales), [i.double() * s.double()[:, :, None]
                                              for i, s in zip(ints, scales)]),
                          ((*codes, *one), [c.double() * s.double() for c, s in zip(codes, one)])):
        out, allow = ref.layer_few(x, idx, w, weights_, None, torch.float32)
        for c in range(d):
            want = 0.0
            for e, ww in ((2, float(w[0, 0])), (0, float(w[0, 1]))):
                for j in range(f):
                    gt = sum(float(val[0][e, j, i]) * float(x[0, i]) for i in range(d))
                    up = sum(float(val[0][e, f + j, i]) * float(x[0, i]) for i in range(d))
                    want += ww * float(val[1][e, c, j]) * gt / (1 + np.exp(-gt)) * up
            assert abs(float(out[0, c]) - want) < 1e-9 * (1 + abs(want))
            assert 0 < allow[0, c] < 1e-2 * (1 + abs(want))


# ----------------------------------------------------------------------------
# AdamW
# ----------------------------------------------------------------------------

def tensor(n=8, p=P, master=None, g=P, m=P, v=P, ms=None, vs=None, p_dt=F, g_dt=F):
    return B.AdamWTensor(n, p, master, g, m, v, ms, vs, p_dt, g_dt)


def call(lib, *tensors, n=None, step=P, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, gs=None):
    a = (B.AdamWTensor * max(len(tensors), 1))(*tensors)
    return lib.moe_adamw(a if tensors else None, len(tensors) if n is None else n, step, lr, b1, b2,
                         eps, wd, gs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(n=(1 << 40) + 1), UNSUPPORTED), (dict(p_dt=2), DTYPE),
    (dict(g_dt=-1), DTYPE), (dict(master=P), DTYPE), (dict(p=None), NULL), (dict(g=None), NULL),
    (dict(m=None), NULL), (dict(v=None), NULL), (dict(ms=P), NULL), (dict(vs=P), NULL),
    (dict(p=P + 2), ALIGN), (dict(p=P + 1, p_dt=H), ALIGN), (dict(master=P + 2, p_dt=H), ALIGN),
    (dict(g=P + 2), ALIGN), (dict(g=P + 1, g_dt=H), ALIGN), (dict(m=P + 2), ALIGN),
    (dict(v=P + 1), ALIGN), (dict(ms=P + 2, vs=P), ALIGN), (dict(ms=P, vs=P + 1), ALIGN)])
def test_adamw_refuses_a_tensor(lib, kw, status):
    assert call(lib, tensor(n=0), tensor(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(lr=-1e-3), SHAPE), (dict(lr=float("nan")), SHAPE), (dict(lr=float("inf")), SHAPE),
    (dict(lr=1e300), SHAPE), (dict(b1=1.0), SHAPE), (dict(b1=-0.1), SHAPE), (dict(b2=1.0), SHAPE),
    (dict(b2=float("nan")), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=1e-60), SHAPE),
    (dict(eps=1e60), SHAPE), (dict(wd=-1.0), SHAPE), (dict(wd=float("inf")), SHAPE),
    (dict(step=None), NULL), (dict(step=P + 4), ALIGN), (dict(gs=P + 2), ALIGN), (dict(n=-1), SHAPE),
    (dict(n=(1 << 20) + 1), UNSUPPORTED)])
def test_adamw_refusals(lib, kw, status):
    assert call(lib, tensor(), **kw) == status


def test_adamw_of_nothing(lib):
    assert call(lib) == 0 and call(lib, tensor(n=0, p=None, g=None, m=None, v=None), step=None) == 0
    assert call(lib, n=1) == NULL


def test_adamw_form_is_torchs():
    g = torch.Generator().manual_seed(3)
    new = lambda: torch.randn(50, generator=g, dtype=torch.float64)  # noqa: E731
    p = torch.nn.Parameter(new())
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.9), eps=1e-6, weight_decay=0.3)
    w, m, v = p.detach().clone(), torch.zeros(50, dtype=torch.float64), torch.zeros(50, dtype=torch.float64)
    for step in range(1, 6):
        p.grad = new()
        w, m, v = ref.adamw64(w, p.grad * 2, m, v, step, 1e-2, 0.8, 0.9, 1e-6, 0.3, gs=0.5)
        opt.step()
        assert torch.allclose(w, p.detach(), rtol=1e-12, atol=1e-14)
        q = ref.adamw32(*(t.float().numpy() for t in (w, p.grad, m, v)), step, 1e-2, 0.8, 0.9, 1e-6, 0.3)
        x = ref.adamw64(w, p.grad, m, v, step, 1e-2, 0.8, 0.9, 1e-6, 0.3)
        for a, b in zip(q, x):
            assert np.allclose(a, b.numpy(), rtol=1e-5, atol=1e-7)


def test_state_codes_by_hand():
    values = ref.root_values()
    assert (np.diff(values) > 0).all() and values[:3].tolist() == [0, 1, 2]
    assert values[63] == 63 and values[64] == 64 and values[65] == 66 and values[255] == 63 * 64
    # a block whose largest root is 4032 has a scale of one; 0.2 is held as 1, and
    # 65 lies half-way between codes 64 and 65
    c, s = ref.v_codes(np.array([4032, 0.2, 0, 65, 67, 31.5, 100], np.float32))
    assert s.tolist() == [1.0] and c.tolist() == [255, 1, 0, 64, 66, 32, 82]
    q, s = ref.m_codes(np.array([449, -0.001, 17], np.float32))
    assert s.tolist() == [2.0] and q.tolist() == [224, 0, 8]


# ----------------------------------------------------------------------------
# the binding's and layer.py's own checks, on tensors of the CPU
# ----------------------------------------------------------------------------

def z(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt)


def test_binding_refuses_tensors_before_the_library():
    i8, i32 = torch.int8, torch.int32
    with pytest.raises(ValueError, match="not on the GPU"):
        moe.moe_rowscale_quantize(z(2, 16), z(2, 16, dt=i8), z(2))
    with pytest.raises(TypeError, match="codes is torch.uint8"):
        moe.moe_rowscale_quantize(z(2, 16), z(2, 16, dt=torch.uint8), z(2))
    with pytest.raises(ValueError, match="scales has shape"):
        moe.moe_rowscale_quantize(z(3, 2, 16), z(3, 2, 16, dt=i8), z(6))
    with pytest.raises(ValueError, match="1 dimensions"):
        moe.moe_rowscale_quantize(z(16), z(16, dt=i8), z(1))
    a = dict(xq=z(4, 16, dt=i8), xs=z(4), wq=z(2, 8, 16, dt=i8), ws=z(2, 8), offsets=z(3, dt=i32),
             y=z(4, 8))
    for name, bad, err, match in (("xs", z(4, 1), ValueError, "xs has shape"),
                                  ("ws", z(2, 8, 1), ValueError, "ws has shape"),
                                  ("wq", z(2, 8, 32, dt=i8)[..., ::2], ValueError, "wq is not contiguous"),
                                  ("xq", z(4, 16), TypeError, "xq is torch.float32"),
                                  ("offsets", z(2, dt=i32), ValueError, "offsets has shape"),
                                  ("y", z(4, 8, dt=torch.float16), TypeError, "y is torch.float16")):
        with pytest.raises(err, match=match):
            moe.moe_rowscale_mm(**dict(a, **{name: bad}))
    with pytest.raises(ValueError, match="scales has shape"):
        moe.moe_swiglu_rowscale(z(4, 32), z(4, 16, dt=i8), z(4, 1))


def test_layer_few_binding_refusals():
    d, f, E, k, T = 64, 64, 4, 2, 3
    bf = lambda *s: z(*s, dt=BF16)  # noqa: E731
    a = dict(shape=(d, f, E, k, 64, 0), x=bf(T, d), w_router=None, bias=None,
             experts=(bf(E, 2 * f, d), bf(E, d, f)), shared=None, topk_idx=z(T, k, dt=torch.int32),
             topk_w=z(T, k), out=bf(T, d), workspace=z(4096, dt=torch.uint8))
    i8 = (z(E, 2 * f, d, dt=torch.int8), z(E, d, f, dt=torch.int8))
    f8 = (z(E, 2 * f, d, dt=torch.float8_e4m3fn), z(E, d, f, dt=torch.float8_e4m3fn))
    for kw, err, match in (
            (dict(), ValueError, "not on the GPU"), (dict(x=z(T, d)), TypeError, "x is"),
            (dict(x=bf(T, d + 64)), ValueError, "x has shape"),
            (dict(experts=(bf(E, 2 * f, d), z(E, d, f))), TypeError, "expert down is"),
            (dict(experts=(bf(E, f, d), bf(E, d, f))), ValueError, "expert gate_up has shape"),
            (dict(experts=(bf(E, 2 * f, d), bf(E, d, f), z(E, 2 * f), z(E, d))), ValueError, "no scales"),
            (dict(experts=i8), ValueError, "codes have no scales"),
            (dict(experts=(*i8, z(E, 2 * f), None)), ValueError, "codes have no scales"),
            (dict(experts=(*i8, z(E, f), z(E, d))), ValueError, "gate_up scales has shape"),
            (dict(experts=(*f8, z(E, 1, 1), z(E, 2, 1))), ValueError, "down scales has shape"),
            (dict(experts=(z(E, 2 * f, d), z(E, d, f))), TypeError, "expert gate_up is"),
            (dict(shared=(z(1, 2 * f, d, dt=torch.int8), z(1, d, f, dt=torch.int8), z(1, 2 * f), z(1, d))),
             TypeError, "another way"),
            (dict(shared=(bf(E, 2 * f, d), bf(E, d, f))), ValueError, "shared gate_up has shape"),
            (dict(topk_idx=z(T, k)), TypeError, "topk_idx is"),
            (dict(topk_w=z(T, k + 1)), ValueError, "topk_w has shape"),
            (dict(w_router=z(E, d + 1)), ValueError, "w_router has shape"),
            (dict(bias=z(E + 1)), ValueError, "bias has shape"),
            (dict(out=bf(T, 2 * d)[:, :d]), ValueError, "out is not contiguous")):
        with pytest.raises(err, match=match):
            moe.moe_layer_few(**dict(a, **kw))


def test_adamw_tensors_are_checked():
    n = 300
    a = dict(params=[z(n), z(n, dt=BF16)], grads=[z(n), z(n)], m=[z(n), z(n)], v=[z(n), z(n)],
             masters=[None, z(n)])
    q = moe.AdamWTensors(**a)
    assert q.n == 2 and q.array[1].n == n and q.array[0].master is None
    assert q.array[1].master == a["masters"][1].data_ptr() and q.array[1].p_dt == B.MOE_BF16
    flat = z(3 * n)
    codes = [z(n, dt=torch.float8_e4m3fn), z(n, dt=torch.uint8)]
    for kw, err, match in (
            (dict(grads=[z(n)]), ValueError, "1 grads for 2 params"),
            (dict(grads=None), ValueError, "grads is missing"),
            (dict(m=[z(n), None]), ValueError, r"m\[1\] is missing"),
            (dict(masters=[z(n), None]), TypeError, r"masters\[0\] stands beside"),
            (dict(grads=[z(n), z(n + 1)]), ValueError, r"grads\[1\] has shape"),
            (dict(v=[z(n), z(n, dt=BF16)]), TypeError, r"v\[1\] is"),
            (dict(m_scales=[z(2), None]), ValueError, r"only one of m_scales\[0\]"),
            (dict(m_scales=[z(2), None], v_scales=[z(2), None]), TypeError, r"m\[0\] is"),
            (dict(m=[codes[0], z(n)], v=[codes[1], z(n)], m_scales=[z(3), None],
                  v_scales=[z(2), None]), ValueError, r"m_scales\[0\] has shape"),
            (dict(params=[z(n, dt=torch.float16), z(n, dt=BF16)]), TypeError, r"params\[0\] is"),
            (dict(params=[z(2 * n)[::2], z(n, dt=BF16)]), ValueError, r"params\[0\] is not contiguous"),
            (dict(params=[a["params"][0], a["params"][0]], masters=None), ValueError, "tensors 0 and 1 overlap"),
            (dict(m=[flat[:n], flat[n - 1:2 * n - 1]]), ValueError, "overlap"),
            (dict(m=[flat[:n], flat[n:2 * n]], v=[flat[2 * n:], flat[1:n + 1]]), ValueError, "overlap"),
            (dict(grads=[z(n), a["params"][0]]), ValueError, "overlap")):
        with pytest.raises(err, match=match):
            moe.AdamWTensors(**dict(a, **kw))
    # neighbours do not overlap, gradients may be shared, empty tensors lie anywhere
    moe.AdamWTensors([flat[:n], z(n)], [a["grads"][0]] * 2, [flat[n:2 * n], z(n)], [flat[2 * n:], z(n)])
    moe.AdamWTensors([flat, flat[5:5]], [z(3 * n), z(0)], [z(3 * n), z(0)], [z(3 * n), z(0)])
    with pytest.raises(ValueError, match="not on the GPU"):
        moe.moe_adamw(q, torch.ones(1, dtype=torch.int64), 1e-3)
    with pytest.raises(TypeError, match="step is"):
        moe.moe_adamw(q, torch.ones(1), 1e-3)


def test_adamw_refuses_a_list_whose_memory_was_replaced():
    for name in ("params", "grads"):
        a = {q: [z(8), z(300)] for q in ("params", "grads", "m", "v")}
        q = moe.AdamWTensors(**a)
        a[name][1].data = z(300)
        with pytest.raises(ValueError, match="lies elsewhere"):
            moe.moe_adamw(q, torch.ones(1, dtype=torch.int64), 1e-3)


def test_a_refused_step_does_not_count():
    opt = L.AdamW([z(4)], [z(4)])
    for _ in range(2):
        with pytest.raises(ValueError, match="not on the GPU"):
            opt.step(1e-3)
    assert int(opt.count) == 0


def test_masters_are_no_part_of_a_graph():
    p = torch.nn.Parameter(z(4, dt=BF16))
    assert not L.AdamW([p], [z(4)]).masters[0].requires_grad


def test_optimiser_state_of_a_layer():
    bf = lambda *s: z(*s, dt=BF16)  # noqa: E731
    sh = moe.Shape(128, 64, 4, 2, 64, 64)
    ex = L.FloatExperts(bf(4, 128, 128), bf(4, 128, 64), bf(1, 128, 128), bf(1, 128, 64))
    buf = L.FloatLayerBuffers.allocate(sh, 3, device="cpu")
    grads = L.FloatLayerGrads.allocate(buf, ex)
    for bits in (32, 8):
        opt = L.AdamW.of_experts(ex, grads, bits)
        assert opt.tensors.n == 4 and opt.params[0] is ex.gate_up and opt.grads[3] is grads.dshared_down
        assert all(w.dtype == torch.float32 for w in opt.masters)
        assert opt.tensors.array[0].g == grads.dgate_up.data_ptr()
    assert all(w is None for w in L.AdamW.of_experts(ex, grads, masters=False).masters)
    with pytest.raises(ValueError, match="16 bits"):
        L.AdamW([z(4)], [z(4)], bits=16)
    with pytest.raises(ValueError, match="no parameters"):
        L.AdamW([], [])


def test_layer_refuses_integers_in_buffers_for_e4m3():
    sh = moe.Shape(128, 64, 4, 2, 64, 0)
    i8 = L.FloatExperts(z(4, 128, 128, dt=torch.int8), z(4, 128, 64, dt=torch.int8),
                        scales=(z(4, 128), z(4, 128)))
    f8 = L.FloatExperts(z(4, 128, 128, dt=torch.float8_e4m3fn), z(4, 128, 64, dt=torch.float8_e4m3fn),
                        scales=(z(4, 1, 1), z(4, 1, 1)))
    x, wr = z(3, 128, dt=BF16), z(4, 128)
    for ex, kw in ((i8, dict(codes=True)), (f8, dict(ints=True))):
        with pytest.raises(ValueError, match="int8 experts take buffers"):
            L.run_layer_float(x, wr, None, ex, L.FloatLayerBuffers.allocate(sh, 3, device="cpu", **kw))
    with pytest.raises(ValueError, match="8-bit experts take buffers"):
        L.run_layer_float(x, wr, None, i8, L.FloatLayerBuffers.allocate(sh, 3, device="cpu"))
