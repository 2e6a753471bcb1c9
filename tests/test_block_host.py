"""Host-side checks of the calls in include/moe_int4_block.h (no GPU needed).

Every call below has at least one defect, or no work, so none reaches a
kernel launch.  Then the float64 forms the GPU tests compare with, against
numerical differences and hand-worked values.
"""
import ctypes

import pytest
import torch

import block_ref as ref
import int4_routed_expert_logits_amd as moe
from int4_routed_expert_logits_amd import _binding as B
from int4_routed_expert_logits_amd import layer as L

P = 1 << 20  # a 256-byte aligned stand-in address (never dereferenced)
MIS = P + 4
F, H = B.MOE_F32, B.MOE_BF16


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def edit(args, **kw):
    out = dict(args)
    out.update(kw)
    return list(out.values())


MM = dict(E=4, P=16, N=64, K=128, x=P, x_rows=16, rows=None, div=1, w=P, off=P, y=P, dt=H, s=None)
DX = dict(E=4, P=16, N=64, K=128, dy=P, w=P, off=P, dx=P, dt=H, s=None)
DW = dict(E=4, P=16, N=64, K=128, dy=P, x=P, x_rows=16, rows=None, div=1, off=P, dw=P, dt=F, ws=P,
          n=1 << 40, s=None)
BS = dict(E=4, P=16, N=64, K=128, xq=P, xs=P, x_rows=16, rows=None, div=1, wq=P, ws=P, off=P, y=P,
          dt=H, s=None)
SIZES = [(dict(E=0), B.MOE_ERR_SHAPE), (dict(E=-1), B.MOE_ERR_SHAPE), (dict(P=-1), B.MOE_ERR_SHAPE),
         (dict(N=0), B.MOE_ERR_SHAPE), (dict(N=4), B.MOE_ERR_SHAPE), (dict(K=-8), B.MOE_ERR_SHAPE),
         (dict(K=12), B.MOE_ERR_SHAPE), (dict(E=1025), B.MOE_ERR_UNSUPPORTED),
         (dict(P=(1 << 24) + 1), B.MOE_ERR_UNSUPPORTED), (dict(N=65544), B.MOE_ERR_UNSUPPORTED),
         (dict(K=65552), B.MOE_ERR_UNSUPPORTED), (dict(dt=2), B.MOE_ERR_DTYPE),
         (dict(dt=-1), B.MOE_ERR_DTYPE), (dict(off=None), B.MOE_ERR_NULL),
         (dict(off=P + 2), B.MOE_ERR_ALIGN)]
ROWS = [(dict(div=2), B.MOE_ERR_SHAPE), (dict(x_rows=15), B.MOE_ERR_SHAPE),
        (dict(x_rows=-1), B.MOE_ERR_SHAPE), (dict(rows=P, div=0), B.MOE_ERR_SHAPE),
        (dict(rows=P, div=257), B.MOE_ERR_UNSUPPORTED),
        (dict(rows=P, div=256, x_rows=65537), B.MOE_ERR_UNSUPPORTED),
        (dict(rows=P + 1), B.MOE_ERR_ALIGN)]


@pytest.mark.parametrize("kw,status", SIZES + ROWS + [
    (dict(x=None), B.MOE_ERR_NULL), (dict(w=None), B.MOE_ERR_NULL), (dict(y=None), B.MOE_ERR_NULL),
    (dict(x=MIS), B.MOE_ERR_ALIGN), (dict(w=MIS), B.MOE_ERR_ALIGN), (dict(y=MIS), B.MOE_ERR_ALIGN)])
def test_grouped_mm_refusals(lib, kw, status):
    assert lib.moe_grouped_mm(*edit(MM, **kw)) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(dy=None), B.MOE_ERR_NULL), (dict(w=None), B.MOE_ERR_NULL), (dict(dx=None), B.MOE_ERR_NULL),
    (dict(dy=MIS), B.MOE_ERR_ALIGN), (dict(w=MIS), B.MOE_ERR_ALIGN), (dict(dx=MIS), B.MOE_ERR_ALIGN)])
def test_grouped_mm_dx_refusals(lib, kw, status):
    assert lib.moe_grouped_mm_dx(*edit(DX, **kw)) == status


@pytest.mark.parametrize("kw,status", SIZES + ROWS + [
    (dict(dy=None), B.MOE_ERR_NULL), (dict(x=None), B.MOE_ERR_NULL), (dict(dw=None), B.MOE_ERR_NULL),
    (dict(dy=MIS), B.MOE_ERR_ALIGN), (dict(x=MIS), B.MOE_ERR_ALIGN), (dict(dw=MIS), B.MOE_ERR_ALIGN),
    (dict(ws=P + 64), B.MOE_ERR_ALIGN)])
def test_grouped_mm_dw_refusals(lib, kw, status):
    assert lib.moe_grouped_mm_dw(*edit(DW, **kw)) == status


def test_grouped_mm_dw_workspace(lib):
    for sizes in ((1, 1 << 20, 64, 64), (1, 1 << 24, 8, 8), (4, 100, 64, 64), (1024, 1 << 24, 8, 8)):
        n = moe.moe_grouped_mm_dw_workspace_bytes(*sizes)
        assert n % 256 == 0 and n < 1 << 32
        if n:
            a = dict(DW, E=sizes[0], P=sizes[1], N=sizes[2], K=sizes[3], x_rows=sizes[1])
            assert lib.moe_grouped_mm_dw(*edit(a, n=n - 1)) == B.MOE_ERR_WORKSPACE
            assert lib.moe_grouped_mm_dw(*edit(a, ws=None)) == B.MOE_ERR_NULL
    assert moe.moe_grouped_mm_dw_workspace_bytes(0, 5, 8, 8) == 0
    assert moe.moe_grouped_mm_dw_workspace_bytes(1, 5, 9, 8) == 0


@pytest.mark.parametrize("kw,status", SIZES + ROWS + [
    (dict(K=136), B.MOE_ERR_SHAPE), (dict(xq=None), B.MOE_ERR_NULL), (dict(xs=None), B.MOE_ERR_NULL),
    (dict(wq=None), B.MOE_ERR_NULL), (dict(ws=None), B.MOE_ERR_NULL), (dict(y=None), B.MOE_ERR_NULL),
    (dict(xq=MIS), B.MOE_ERR_ALIGN), (dict(wq=MIS), B.MOE_ERR_ALIGN), (dict(y=MIS), B.MOE_ERR_ALIGN),
    (dict(xs=P + 2), B.MOE_ERR_ALIGN), (dict(ws=P + 1), B.MOE_ERR_ALIGN)])
def test_blockscale_mm_refusals(lib, kw, status):
    assert lib.moe_blockscale_mm(*edit(BS, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), B.MOE_ERR_SHAPE), (dict(R=-1), B.MOE_ERR_SHAPE), (dict(K=8), B.MOE_ERR_SHAPE),
    (dict(K=0), B.MOE_ERR_SHAPE), (dict(K=65552), B.MOE_ERR_UNSUPPORTED),
    (dict(br=64), B.MOE_ERR_UNSUPPORTED), (dict(br=0), B.MOE_ERR_UNSUPPORTED),
    (dict(n=70000, R=70000), B.MOE_ERR_UNSUPPORTED), (dict(R=2 ** 31 - 1, K=65536), B.MOE_ERR_UNSUPPORTED),
    (dict(dt=9), B.MOE_ERR_DTYPE), (dict(x=None), B.MOE_ERR_NULL), (dict(c=None), B.MOE_ERR_NULL),
    (dict(sc=None), B.MOE_ERR_NULL), (dict(x=MIS), B.MOE_ERR_ALIGN), (dict(c=MIS), B.MOE_ERR_ALIGN),
    (dict(sc=P + 2), B.MOE_ERR_ALIGN)])
def test_blockscale_quantize_refusals(lib, kw, status):
    a = dict(n=1, R=4, K=128, x=P, dt=H, br=1, c=P, sc=P, s=None)
    assert lib.moe_blockscale_quantize(*edit(a, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(P=-1), B.MOE_ERR_SHAPE), (dict(f=0), B.MOE_ERR_SHAPE), (dict(f=12), B.MOE_ERR_SHAPE),
    (dict(f=32784), B.MOE_ERR_UNSUPPORTED), (dict(P=(1 << 24) + 1), B.MOE_ERR_UNSUPPORTED),
    (dict(dt=5), B.MOE_ERR_DTYPE), (dict(a=None), B.MOE_ERR_NULL), (dict(a=MIS), B.MOE_ERR_ALIGN),
    (dict(b=None), B.MOE_ERR_NULL), (dict(b=MIS), B.MOE_ERR_ALIGN), (dict(n=P + 2), B.MOE_ERR_ALIGN)])
def test_swiglu_refusals(lib, kw, status):
    v = dict(P=4, f=64, a=P, b=P, dt=H, n=None)
    v.update(kw)
    assert lib.moe_swiglu(v["P"], v["f"], v["a"], v["b"], v["dt"], v["n"], None) == status
    assert lib.moe_swiglu_quantize(v["P"], v["f"], v["a"], v["dt"], v["b"], P, v["n"], None) == status
    assert lib.moe_swiglu_grad(v["P"], v["f"], v["a"], P, v["b"], v["dt"], v["n"], None) == status


def test_swiglu_quantize_wants_sixteen_columns(lib):
    assert lib.moe_swiglu_quantize(4, 72, P, H, P, P, None, None) == B.MOE_ERR_SHAPE
    assert lib.moe_swiglu_quantize(4, 64, P, H, P, None, None, None) == B.MOE_ERR_NULL
    assert lib.moe_swiglu_grad(4, 64, P, None, P, H, None, None) == B.MOE_ERR_NULL


def test_combine_grad_refusals(lib):
    ok = B.Shape(512, 256, 8, 2, 64, 0)
    a = dict(sh=ctypes.byref(ok), T=4, do=P, odt=H, y=P, ydt=H, inv=P, w=P, dy=P, dw=P, s=None)
    for kw, status in ((dict(sh=None), B.MOE_ERR_NULL), (dict(T=-1), B.MOE_ERR_SHAPE),
                       (dict(sh=ctypes.byref(B.Shape(96, 64, 8, 2, 64, 0))), B.MOE_ERR_SHAPE),
                       (dict(T=1 << 24), B.MOE_ERR_UNSUPPORTED), (dict(odt=3), B.MOE_ERR_DTYPE),
                       (dict(ydt=-2), B.MOE_ERR_DTYPE)):
        assert lib.moe_combine_grad(*edit(a, **kw)) == status
    for name in ("do", "y", "inv", "w", "dy", "dw"):
        assert lib.moe_combine_grad(*edit(a, **{name: None})) == B.MOE_ERR_NULL
    for name in ("do", "y", "dy"):
        assert lib.moe_combine_grad(*edit(a, **{name: MIS})) == B.MOE_ERR_ALIGN
    for name in ("inv", "w", "dw"):
        assert lib.moe_combine_grad(*edit(a, **{name: P + 2})) == B.MOE_ERR_ALIGN


NORM = dict(T=4, d=64, y=P, ydt=H, w1=P, gate=None, g=0, scale=1.0, res=P, rdt=H, out=P, w2=P,
            eps=1e-6, n=P, ndt=H, s=None)
NGRAD = dict(T=4, d=64, y=P, ydt=H, w1=P, gate=None, g=0, scale=1.0, res=P, rdt=H, w2=P, eps=1e-6,
             dr=P, dn=P, ndt=H, dy=P, dres=P, dgate=None, dw1=P, dw2=P, ws=P, nws=1 << 40, s=None)
NORM_BAD = [(dict(T=-1), B.MOE_ERR_SHAPE), (dict(d=0), B.MOE_ERR_SHAPE), (dict(d=12), B.MOE_ERR_SHAPE),
            (dict(d=8200), B.MOE_ERR_UNSUPPORTED), (dict(T=(1 << 24) + 1), B.MOE_ERR_UNSUPPORTED),
            (dict(ydt=4), B.MOE_ERR_DTYPE), (dict(rdt=4), B.MOE_ERR_DTYPE),
            (dict(ndt=-4), B.MOE_ERR_DTYPE), (dict(eps=0.0), B.MOE_ERR_SHAPE),
            (dict(eps=-1.0), B.MOE_ERR_SHAPE), (dict(eps=float("nan")), B.MOE_ERR_SHAPE),
            (dict(eps=float("inf")), B.MOE_ERR_SHAPE), (dict(scale=float("nan")), B.MOE_ERR_SHAPE),
            (dict(scale=float("inf")), B.MOE_ERR_SHAPE), (dict(g=1), B.MOE_ERR_SHAPE),
            (dict(gate=P, g=0), B.MOE_ERR_SHAPE), (dict(gate=P, g=3), B.MOE_ERR_SHAPE),
            (dict(y=None), B.MOE_ERR_NULL), (dict(y=None, res=None, w1=None), B.MOE_ERR_NULL),
            (dict(y=MIS), B.MOE_ERR_ALIGN), (dict(res=MIS), B.MOE_ERR_ALIGN),
            (dict(w1=MIS), B.MOE_ERR_ALIGN), (dict(w2=MIS), B.MOE_ERR_ALIGN),
            (dict(gate=MIS, g=1), B.MOE_ERR_ALIGN)]


@pytest.mark.parametrize("kw,status", NORM_BAD + [
    (dict(n=None), B.MOE_ERR_NULL), (dict(w2=None), B.MOE_ERR_NULL),
    (dict(w2=None, n=None, out=None), B.MOE_ERR_NULL), (dict(out=MIS), B.MOE_ERR_ALIGN),
    (dict(n=MIS), B.MOE_ERR_ALIGN)])
def test_block_norm_refusals(lib, kw, status):
    assert lib.moe_block_norm(*edit(NORM, **kw)) == status


@pytest.mark.parametrize("kw,status", [b for b in NORM_BAD if b[0] != dict(y=None)] + [
    (dict(dn=None), B.MOE_ERR_NULL), (dict(w2=None), B.MOE_ERR_NULL),
    (dict(w1=None), B.MOE_ERR_NULL), (dict(dgate=P), B.MOE_ERR_NULL), (dict(ws=None), B.MOE_ERR_NULL),
    (dict(y=None, w1=None, dw1=None), B.MOE_ERR_NULL), (dict(ws=P + 64), B.MOE_ERR_ALIGN),
    (dict(nws=4 * 2 * 64 * 4 - 1), B.MOE_ERR_WORKSPACE), (dict(dr=MIS), B.MOE_ERR_ALIGN),
    (dict(dn=MIS), B.MOE_ERR_ALIGN), (dict(dy=MIS), B.MOE_ERR_ALIGN), (dict(dres=MIS), B.MOE_ERR_ALIGN),
    (dict(dw1=P + 2), B.MOE_ERR_ALIGN), (dict(dw2=P + 2), B.MOE_ERR_ALIGN)])
def test_block_norm_grad_refusals(lib, kw, status):
    assert lib.moe_block_norm_grad(*edit(NGRAD, **kw)) == status


def test_block_norm_grad_workspace(lib):
    assert moe.moe_block_norm_grad_workspace_bytes(3, 64) == 3 * 2 * 64 * 4
    assert moe.moe_block_norm_grad_workspace_bytes(1 << 24, 8192) < 1 << 30
    for T, d in ((-1, 64), (4, 0), (4, 60), (4, 8200)):
        assert moe.moe_block_norm_grad_workspace_bytes(T, d) == 0


def test_calls_without_work_return_ok(lib):
    """No rows: nothing to enqueue, and no pointer is needed but the ones checked."""
    assert lib.moe_grouped_mm(*edit(MM, P=0, x=None, w=None, y=None, off=None)) == B.MOE_OK
    # an empty rows tensor has no address
    assert lib.moe_grouped_mm(*edit(MM, P=0, rows=None, div=2)) == B.MOE_OK
    assert lib.moe_grouped_mm_dx(*edit(DX, P=0, dy=None, w=None, dx=None, off=None)) == B.MOE_OK
    assert lib.moe_blockscale_mm(*edit(BS, P=0, xq=None, wq=None, y=None, off=None)) == B.MOE_OK
    assert lib.moe_blockscale_quantize(0, 5, 64, None, H, 1, None, None, None) == B.MOE_OK
    assert lib.moe_swiglu(0, 64, None, None, H, None, None) == B.MOE_OK
    assert lib.moe_block_norm(*edit(NORM, T=0)) == B.MOE_OK
    assert lib.moe_block_norm_grad(*edit(NGRAD, dy=None, dres=None, dw1=None, dw2=None)) == B.MOE_OK


def test_binding_checks_tensors():
    """Shapes, types, strides and places are checked before the library is called."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on the GPU"):
        moe.moe_grouped_mm(bf(4, 8), bf(2, 8, 8), off, bf(4, 8))
    with pytest.raises(TypeError, match="x is torch.float32"):
        moe.moe_grouped_mm(bf(4, 8).float(), bf(2, 8, 8), off, bf(4, 8))
    with pytest.raises(ValueError, match="w has 2 dimensions"):
        moe.moe_grouped_mm(bf(4, 8), bf(8, 8), off, bf(4, 8))
    with pytest.raises(ValueError, match="xq has 3 dimensions"):
        moe.moe_blockscale_mm(bf(4, 8, 2), None, bf(2, 8, 8), None, off, bf(4, 8))
    with pytest.raises(ValueError, match="neither y nor res"):
        moe.moe_block_norm(None, None, None, None)


def test_layer_checks_its_arguments():
    """Before anything is enqueued (these tensors are not on a GPU)."""
    E, d, f, T = 4, 64, 64, 3
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ex = L.FloatExperts(bf(E, 2 * f, d), bf(E, d, f))
    buf = L.FloatLayerBuffers.allocate(moe.Shape(d, f, E, 2, 64, 0), T, device="cpu")
    codes = L.FloatLayerBuffers.allocate(moe.Shape(d, f, E, 2, 64, 0), T, codes=True, device="cpu")
    grads = L.FloatLayerGrads.allocate(buf, ex)
    wr = torch.zeros(E, d)
    with pytest.raises(ValueError, match="x has shape"):
        L.run_layer_float(bf(T + 1, d), wr, None, ex, buf)
    with pytest.raises(ValueError, match="x has shape"):
        L.run_layer_float_grad(bf(T, d), bf(T - 1, d), ex, buf, grads)
    with pytest.raises(ValueError, match="codes=True"):
        L.run_layer_float(bf(T, d), wr, None, ex, codes)
    ex.scales = (torch.zeros(E, 1, 1), torch.zeros(E, 1, 1))
    with pytest.raises(ValueError, match="codes=True"):
        L.run_layer_float(bf(T, d), wr, None, ex, buf)
    with pytest.raises(ValueError, match="no gradient"):
        L.run_layer_float_grad(bf(T, d), bf(T, d), ex, codes, grads)
    ex.shared_gate_up = bf(1, 2 * f, d)
    with pytest.raises(ValueError, match="shared expert"):
        L.run_layer_float(bf(T, d), wr, None, ex, codes)
    norms = L.BlockNorms(torch.ones(d), torch.ones(d), eps=1e-5)
    with pytest.raises(ValueError, match="eps"):
        L.run_block(bf(T, d), norms, lambda n: n, bf(T, d), bf(T, d), L.BlockNorms(torch.ones(d)),
                    bf(T, d))


# ----------------------------------------------------------------------------
# the float64 forms themselves
# ----------------------------------------------------------------------------

def g64(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def differences(f, x, h=1e-6):
    """Gradient of the scalar f at x by central differences."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view(x.shape)
        g.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * h)
    return g


def close(a, b):
    assert torch.allclose(a, b, rtol=2e-7, atol=2e-8), (a - b).abs().max()


def test_grouped_gradients_by_differences():
    off, rows = [0, 2, 2, 5], torch.tensor([3, 0, 5, 2, 1])
    x, w, dy = g64(1, 3, 4), g64(2, 3, 6, 4), g64(3, 5, 6)
    f = lambda x, w: (ref.grouped_mm(x, w, off, 5, rows, 2)[0] * dy).sum()  # noqa: E731
    close(ref.grouped_mm_dw(dy, x, off, 3, rows, 2)[0], differences(lambda v: f(x, v), w))
    dx = ref.grouped_mm_dx(dy, w, off)[0]
    want = differences(lambda v: f(v, w), x)
    close(torch.zeros_like(x).index_add(0, rows // 2, dx), want)


def test_swiglu_gradient_by_differences():
    gu, dh = g64(4, 3, 10), g64(5, 3, 5)
    close(ref.swiglu_grad(gu, dh), differences(lambda v: (ref.swiglu(v) * dh).sum(), gu))


@pytest.mark.parametrize("form", [(1, 1, 1), (1, 1, 4), (0, 1, 1), (1, 0, 0), (0, 0, 4)])
def test_block_norm_gradient_by_differences(form):
    post, pre, gate = form
    T, d, s, eps = 4, 6, 0.7, 1e-3
    t = dict(y=g64(6, T, d), res=g64(7, T, d), w_post=g64(8, d) if post else None,
             w_pre=g64(9, d) if pre else None, gate=g64(10, gate, d) if gate else None)
    dr, dn = g64(11, T, d), g64(12, T, d) if pre else None

    def loss(**kw):
        r, n = ref.block_norm(**{**t, **kw}, scale=s, eps=eps)
        return (r * dr).sum() + (0 if n is None else (n * dn).sum())

    got = ref.block_norm_grad(**t, scale=s, eps=eps, dr=dr, dn=dn)
    for name, out in (("y", "dy"), ("res", "dres"), ("w_post", "dw_post"), ("w_pre", "dw_pre"),
                      ("gate", "dgate")):
        if t[name] is None:
            assert got[out] is None
        else:
            close(got[out], differences(lambda v: loss(**{name: v}), t[name]))


def test_combine_gradient_by_differences():
    inv = torch.tensor([2, 0, -1, 3])
    y, w, dout = g64(13, 4, 5), g64(14, 2, 2), g64(15, 2, 5)

    def loss(y, w):
        out = torch.zeros((2, 5), dtype=torch.float64)
        for s, p in enumerate(inv.tolist()):
            if p >= 0:
                out[s // 2] += w.view(-1)[s] * y[p]
        return (out * dout).sum()

    dy, dw, _ = ref.combine_grad(dout, y, inv, w)
    close(torch.nan_to_num(dy), differences(lambda v: loss(v, w), y))
    close(dw, differences(lambda v: loss(y, v), w))


def test_e4m3_values_are_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().to(torch.float64)
    assert torch.equal(ref.e4m3_values(), codes)
    x = torch.randn(4000, generator=torch.Generator().manual_seed(1)) * 90
    x = x.clamp(-448, 448)
    assert torch.equal(ref.e4m3_round(x.double()), x.to(torch.float8_e4m3fn).double())


def test_quantise_worked_blocks():
    x = torch.zeros(2, 256)
    x[0, 0], x[0, 1] = 448.0, 1.0625  # 1.0625 lies between 1 and 1.125: to the even code
    x[0, 128] = 449.0                 # over 448: the scale is 2
    v, s = ref.quantize(x, 1)
    assert s.tolist() == [[1.0, 2.0], [1.0, 1.0]]
    assert v[0, 0] == 448 and v[0, 1] == 1.0 and v[0, 128] == 224
    v, s = ref.quantize(x, 128)
    assert s.tolist() == [[1.0, 2.0]]
