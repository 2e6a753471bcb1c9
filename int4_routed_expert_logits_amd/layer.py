"""Device buffers for one layer call and the four-call sequence.

Plumbing only: torch allocates the caller-owned device memory the C ABI
expects, and ``run_layer`` issues moe_route_union -> moe_expert_ffn ->
moe_combine on one stream with no host synchronisation in between;
``run_layer_decode`` makes the single moe_layer_decode call instead (decode
batches of at most 8 tokens).

``run_layer_float`` is the layer on bfloat16 expert weights, on e4m3 codes with
block scales or on 8-bit integers with row scales, ``run_layer_few`` the same for a
few tokens in one call, ``run_layer_float_grad`` its gradient (the routing taken as
given), ``AdamW`` the step that applies such gradients, and ``run_block`` any of the
layers between its norms and residual.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional, Sequence

import torch

from . import _binding as B


@dataclasses.dataclass
class LayerBuffers:
    shape: B.Shape
    T: int
    path: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    perm: torch.Tensor
    inv_perm: torch.Tensor
    active: torch.Tensor
    n_active: torch.Tensor
    y: torch.Tensor
    y_shared: Optional[torch.Tensor]
    out: torch.Tensor
    workspace: torch.Tensor       # moe_route scratch
    ffn_workspace: torch.Tensor   # moe_expert_ffn scratch (the intermediate h)
    layer_workspace: torch.Tensor  # moe_layer_decode scratch (decode path only)

    @classmethod
    def allocate(cls, shape, T: int, path: int, device="cuda", out_dtype=None):
        sh = B._shape(shape)
        k, E, d = sh.top_k, sh.n_experts, sh.d
        i32 = dict(dtype=torch.int32, device=device)
        ydt = torch.float32 if path == B.MOE_PATH_DECODE_F32 else torch.bfloat16
        odt = out_dtype or ydt
        ws = max(B.moe_route_workspace_bytes(sh, T), 256)
        fws = max(B.moe_ffn_workspace_bytes(sh, T, path), 256)
        lws = max(B.moe_layer_decode_workspace_bytes(sh, T), 256) if path == B.MOE_PATH_DECODE_F32 else 256
        return cls(
            shape=sh, T=T, path=path,
            topk_idx=torch.empty((T, k), **i32),
            topk_w=torch.empty((T, k), dtype=torch.float32, device=device),
            counts=torch.empty((E,), **i32),
            offsets=torch.empty((E + 1,), **i32),
            perm=torch.empty((max(T * k, 1),), **i32),
            inv_perm=torch.empty((max(T * k, 1),), **i32),
            active=torch.empty((E,), **i32),
            n_active=torch.empty((1,), **i32),
            y=torch.empty((max(T * k, 1), d), dtype=ydt, device=device),
            y_shared=torch.empty((max(T, 1), d), dtype=ydt, device=device) if sh.f_shared else None,
            out=torch.empty((T, d), dtype=odt, device=device),
            workspace=torch.empty((ws,), dtype=torch.uint8, device=device),
            ffn_workspace=torch.empty((fws,), dtype=torch.uint8, device=device),
            layer_workspace=torch.empty((lws,), dtype=torch.uint8, device=device),
        )


def run_layer(x, w_router, bias, experts, shared, buf: LayerBuffers, stream=None):
    """All four steps of the layer for the batch x [T, d]: route and union in
    one call (moe_route_union), then the expert FFN and the combine."""
    sh = buf.shape
    B.moe_route_union(sh, x, w_router, bias, buf.topk_idx, buf.topk_w, buf.counts, buf.offsets,
                      buf.perm, buf.inv_perm, buf.active, buf.n_active, buf.workspace, stream)
    B.moe_expert_ffn(sh, x, experts, shared, buf.offsets, buf.perm, buf.active, buf.n_active,
                     buf.path, buf.y, buf.y_shared, buf.ffn_workspace, stream)
    B.moe_combine(sh, buf.y, buf.y_shared, buf.inv_perm, buf.topk_w, buf.out, stream)
    return buf.out


def run_layer_decode(x, w_router, bias, experts, shared, buf: LayerBuffers, stream=None):
    """The same layer for a decode batch of at most 8 tokens in one call
    (moe_layer_decode): four launches, the same outputs as run_layer."""
    B.moe_layer_decode(buf.shape, x, w_router, bias, experts, shared, buf.topk_idx, buf.topk_w,
                       buf.counts, buf.offsets, buf.perm, buf.inv_perm, buf.active, buf.n_active,
                       buf.y, buf.y_shared, buf.out, buf.layer_workspace, stream)
    return buf.out


# ----------------------------------------------------------------------------
# float and 8-bit experts (include/moe_int4_block.h)
# ----------------------------------------------------------------------------

@dataclasses.dataclass
class FloatExperts:
    """Expert weights of a layer: gate and up stacked [E, 2 f, d] (gate first),
    down [E, d, f], and the shared expert's as one-group tensors or None.  bf16,
    e4m3 codes with their scales per 128 x 128 ([E, 2 f / 128, d / 128] and
    [E, d / 128, f / 128], rounded up), or int8 codes with a scale per output
    channel ([E, 2 f] and [E, d])."""
    gate_up: torch.Tensor
    down: torch.Tensor
    shared_gate_up: Optional[torch.Tensor] = None
    shared_down: Optional[torch.Tensor] = None
    scales: Optional[tuple] = None         # (gate_up, down) of codes
    shared_scales: Optional[tuple] = None

    @classmethod
    def quantize(cls, e: "FloatExperts", stream=None, ints: bool = False) -> "FloatExperts":
        """e's bf16 weights as e4m3 codes and scales (moe_blockscale_quantize), or
        with `ints` as int8 ones (moe_rowscale_quantize), ready on `stream`.  Their
        memory is the current stream's: another one waits for what is queued
        there first, and holds on to all it touches."""
        side = _torch_stream(stream, e.gate_up.device)

        def q(w):
            if w is None:
                return None, None
            n, r, k = w.shape
            if ints:
                codes = torch.empty(w.shape, dtype=torch.int8, device=w.device)
                scales = torch.empty((n, r), device=w.device)
                B.moe_rowscale_quantize(w, codes, scales, stream)
            else:
                codes = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
                scales = torch.empty((n, -(-r // 128), -(-k // 128)), device=w.device)
                B.moe_blockscale_quantize(w, 128, codes, scales, stream)
            if side is not None:
                for t in (w, codes, scales):
                    t.record_stream(side)
            return codes, scales

        if side is not None:
            side.wait_stream(torch.cuda.current_stream(e.gate_up.device))
        (gu, gus), (dn, dns) = q(e.gate_up), q(e.down)
        (sgu, sgus), (sdn, sdns) = q(e.shared_gate_up), q(e.shared_down)
        return cls(gu, dn, sgu, sdn, (gus, dns), None if sgu is None else (sgus, sdns))


def _torch_stream(stream, device):
    """`stream` (a torch stream, a raw handle or None) as torch's own; None for None."""
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)


@dataclasses.dataclass
class FloatLayerBuffers:
    """Routing outputs and intermediates of one run_layer_float call; the
    gradient reads them.  The shared expert is one group of all T tokens."""
    shape: B.Shape
    T: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    n_rows: torch.Tensor          # offsets[E:]: the grouped rows in use
    perm: torch.Tensor
    inv_perm: torch.Tensor
    active: torch.Tensor
    n_active: torch.Tensor
    all_rows: torch.Tensor        # offsets {0, T} of the shared expert's group
    gu: torch.Tensor              # [T k, 2 f] bf16
    h: Optional[torch.Tensor]     # [T k, f] bf16 (bf16 experts)
    y: torch.Tensor               # [T k, d]
    gu_shared: Optional[torch.Tensor]
    h_shared: Optional[torch.Tensor]
    y_shared: Optional[torch.Tensor]
    codes: Optional[dict]         # (codes, scales) of x, h, h_shared (8-bit experts)
    out: torch.Tensor
    workspace: torch.Tensor
    ints: bool = False            # the codes are int8 with a scale per row

    @classmethod
    def allocate(cls, shape, T: int, codes: bool = False, device="cuda",
                 y_dtype=torch.bfloat16, out_dtype=torch.bfloat16, ints: bool = False):
        """codes: for 8-bit experts, e4m3 ones, or int8 ones with `ints`."""
        codes = codes or ints
        sh = B._shape(shape)
        k, E, d, f, P = sh.top_k, sh.n_experts, sh.d, sh.f, T * sh.top_k
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        i32 = torch.int32

        def pair(rows, cols):
            if ints:
                return new(rows, cols, dtype=torch.int8), new(rows, dtype=torch.float32)
            return (new(rows, cols, dtype=torch.float8_e4m3fn),
                    new(rows, -(-cols // 128), dtype=torch.float32))

        shared = bool(sh.f_shared)
        offsets = new(E + 1, dtype=i32)
        return cls(
            shape=sh, T=T, topk_idx=new(T, k, dtype=i32), topk_w=new(T, k, dtype=torch.float32),
            counts=new(E, dtype=i32), offsets=offsets, n_rows=offsets[E:], perm=new(P, dtype=i32),
            inv_perm=new(P, dtype=i32), active=new(E, dtype=i32), n_active=new(1, dtype=i32),
            all_rows=torch.tensor([0, T], dtype=i32, device=device),
            gu=new(P, 2 * f), h=None if codes else new(P, f), y=new(P, d, dtype=y_dtype),
            gu_shared=new(T, 2 * f) if shared else None,
            h_shared=new(T, f) if shared and not codes else None,
            y_shared=new(T, d, dtype=y_dtype) if shared else None,
            codes=dict(x=pair(T, d), h=pair(P, f), h_shared=pair(T, f) if shared else None)
            if codes else None,
            out=new(T, d, dtype=out_dtype),
            workspace=new(max(B.moe_route_workspace_bytes(sh, T), 256), dtype=torch.uint8),
            ints=ints)


def _check_float(fn: str, x, experts: FloatExperts, buf: FloatLayerBuffers):
    if tuple(x.shape) != (buf.T, buf.shape.d):
        raise ValueError(f"{fn}: x has shape {tuple(x.shape)}, the buffers hold "
                         f"{(buf.T, buf.shape.d)}")
    if (experts.shared_gate_up is None) != (buf.y_shared is None):
        raise ValueError(f"{fn}: the shape and the weights disagree about a shared expert")
    if (experts.scales is None) != (buf.codes is None):
        raise ValueError(f"{fn}: 8-bit experts take buffers allocated with codes=True, bf16 ones "
                         "without")
    if buf.codes is not None and (experts.gate_up.dtype == torch.int8) != buf.ints:
        raise ValueError(f"{fn}: int8 experts take buffers allocated with ints=True, e4m3 ones "
                         "without")
    _check_tensor(fn, "x", x, torch.bfloat16, x.shape, buf.gu.device)


def _gpu_of(t):
    """A context with t's GPU as the current one, for the calls that launch there
    (moe_route_union, moe_combine; the others go by their tensors)."""
    B._T or B._types()
    dev = t.get_device()
    if dev < 0 or dev == B._current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _check_tensor(fn: str, name: str, t, dtype, shape, device):
    """What moe_route_union, which takes addresses, cannot see of a tensor."""
    if t is None:
        raise ValueError(f"{fn}: {name} is missing")
    if t.dtype != dtype:
        raise TypeError(f"{fn}: {name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{fn}: {name} is on {t.device}, the buffers on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} is not contiguous")


def run_layer_float(x, w_router, bias, experts: FloatExperts, buf: FloatLayerBuffers, stream=None):
    """The layer for x [T, d] bf16 on float or 8-bit experts: route and union
    (w_router [E, d] and bias [E] or None, float32), gate and up products over
    the gathered tokens, SwiGLU, down products, combine.  Products with 8-bit
    experts take x and h quantised the same way."""
    fn, sh, b, k = "run_layer_float", buf.shape, buf, buf.shape.top_k
    _check_float(fn, x, experts, buf)
    _check_tensor(fn, "w_router", w_router, torch.float32, (sh.n_experts, sh.d), b.gu.device)
    if bias is not None:
        _check_tensor(fn, "bias", bias, torch.float32, (sh.n_experts,), b.gu.device)
    with _gpu_of(b.gu):
        B.moe_route_union(sh, x, w_router, bias, b.topk_idx, b.topk_w, b.counts, b.offsets, b.perm,
                          b.inv_perm, b.active, b.n_active, b.workspace, stream)
    if experts.scales is None:
        B.moe_grouped_mm(x, experts.gate_up, b.offsets, b.gu, b.perm, k, stream)
        B.moe_swiglu(b.gu, b.h, b.n_rows, stream)
        B.moe_grouped_mm(b.h, experts.down, b.offsets, b.y, stream=stream)
        if b.y_shared is not None:
            B.moe_grouped_mm(x, experts.shared_gate_up, b.all_rows, b.gu_shared, stream=stream)
            B.moe_swiglu(b.gu_shared, b.h_shared, stream=stream)
            B.moe_grouped_mm(b.h_shared, experts.shared_down, b.all_rows, b.y_shared, stream=stream)
    else:
        if buf.ints:
            quantize, mm, swiglu = (B.moe_rowscale_quantize, B.moe_rowscale_mm,
                                    B.moe_swiglu_rowscale)
        else:
            quantize, mm, swiglu = (lambda x, q, s, stream: B.moe_blockscale_quantize(  # noqa: E731
                x, 1, q, s, stream), B.moe_blockscale_mm, B.moe_swiglu_quantize)
        (xq, xs), (hq, hs) = b.codes["x"], b.codes["h"]
        gus, dns = experts.scales
        quantize(x, xq, xs, stream)
        mm(xq, xs, experts.gate_up, gus, b.offsets, b.gu, b.perm, k, stream)
        swiglu(b.gu, hq, hs, b.n_rows, stream)
        mm(hq, hs, experts.down, dns, b.offsets, b.y, stream=stream)
        if b.y_shared is not None:
            (hq, hs), (gus, dns) = b.codes["h_shared"], experts.shared_scales
            mm(xq, xs, experts.shared_gate_up, gus, b.all_rows, b.gu_shared, stream=stream)
            swiglu(b.gu_shared, hq, hs, stream=stream)
            mm(hq, hs, experts.shared_down, dns, b.all_rows, b.y_shared, stream=stream)
    with _gpu_of(b.gu):
        B.moe_combine(sh, b.y, b.y_shared, b.inv_perm, b.topk_w, b.out, stream)
    return b.out


@dataclasses.dataclass
class FewLayerBuffers:
    """Routing outputs, result and scratch of one run_layer_few call."""
    shape: B.Shape
    T: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    out: torch.Tensor
    workspace: torch.Tensor

    @classmethod
    def allocate(cls, shape, T: int, device="cuda", out_dtype=torch.bfloat16):
        sh = B._shape(shape)
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        return cls(sh, T, new(T, sh.top_k, dtype=torch.int32), new(T, sh.top_k, dtype=torch.float32),
                   new(T, sh.d, dtype=out_dtype),
                   new(max(B.moe_layer_few_workspace_bytes(sh, T), 256), dtype=torch.uint8))


def run_layer_few(x, w_router, bias, experts: FloatExperts, buf: FewLayerBuffers, stream=None):
    """The layer for a few tokens x [T, d] bf16 (T <= 32, T * top_k <= 256) on any
    of FloatExperts' weights in one call, moe_layer_few, and x and h are not
    quantised.  The faster one up to 8 tokens; beyond, run_layer_float is by up to a
    tenth where an expert of e4m3 codes has three tokens or more, or d is 8192.
    w_router None: buf.topk_idx and buf.topk_w are given."""
    sc, ssc = experts.scales or (None, None), experts.shared_scales or (None, None)
    shared = None
    if experts.shared_gate_up is not None:
        shared = (experts.shared_gate_up, experts.shared_down, *ssc)
    B.moe_layer_few(buf.shape, x, w_router, bias, (experts.gate_up, experts.down, *sc), shared,
                    buf.topk_idx, buf.topk_w, buf.out, buf.workspace, stream)
    return buf.out


@dataclasses.dataclass
class FloatLayerGrads:
    """Gradients of run_layer_float (bf16 experts) and their intermediates."""
    dx: torch.Tensor                      # [T, d], without the router's part
    dtopk_w: torch.Tensor                 # [T, k]
    dgate_up: torch.Tensor                # [E, 2 f, d] float32
    ddown: torch.Tensor                   # [E, d, f] float32
    dshared_gate_up: Optional[torch.Tensor]
    dshared_down: Optional[torch.Tensor]
    dy: torch.Tensor
    dh: torch.Tensor
    dgu: torch.Tensor
    dx_slots: torch.Tensor
    dh_shared: Optional[torch.Tensor]
    dgu_shared: Optional[torch.Tensor]
    dx_shared: Optional[torch.Tensor]
    ones: torch.Tensor
    workspace: torch.Tensor

    @classmethod
    def allocate(cls, buf: FloatLayerBuffers, experts: FloatExperts):
        sh, T, dev = buf.shape, buf.T, buf.gu.device
        P, f, d, E = T * sh.top_k, sh.f, sh.d, sh.n_experts
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
        f32 = torch.float32
        shared = buf.y_shared is not None
        ws = max([256] + [B.moe_grouped_mm_dw_workspace_bytes(*a) for a in (
            (E, P, 2 * f, d), (E, P, d, f), (1, T, 2 * f, d), (1, T, d, f))])
        return cls(
            dx=new(T, d), dtopk_w=new(T, sh.top_k, dtype=f32), dgate_up=new(E, 2 * f, d, dtype=f32),
            ddown=new(E, d, f, dtype=f32),
            dshared_gate_up=new(1, 2 * f, d, dtype=f32) if shared else None,
            dshared_down=new(1, d, f, dtype=f32) if shared else None,
            dy=new(P, d), dh=new(P, f), dgu=new(P, 2 * f), dx_slots=new(P, d),
            dh_shared=new(T, f) if shared else None, dgu_shared=new(T, 2 * f) if shared else None,
            dx_shared=new(T, d) if shared else None,
            ones=torch.ones((T, sh.top_k), device=dev), workspace=new(ws, dtype=torch.uint8))


def run_layer_float_grad(dout, x, experts: FloatExperts, buf: FloatLayerBuffers,
                         g: FloatLayerGrads, stream=None):
    """Gradient of the run_layer_float call that filled buf (bf16 experts and y)
    for dout [T, d] bf16 of its output: the experts' weights, topk_w, and x
    through the experts (x through the router is the caller's, from dtopk_w)."""
    _check_float("run_layer_float_grad", x, experts, buf)
    if experts.scales is not None:
        raise ValueError("run_layer_float_grad: 8-bit experts have no gradient")
    sh, b, k = buf.shape, buf, buf.shape.top_k
    B.moe_combine_grad(sh, dout, b.y, b.inv_perm, b.topk_w, g.dy, g.dtopk_w, stream)
    B.moe_grouped_mm_dw(g.dy, b.h, b.offsets, g.ddown, g.workspace, stream=stream)
    B.moe_grouped_mm_dx(g.dy, experts.down, b.offsets, g.dh, stream)
    B.moe_swiglu_grad(b.gu, g.dh, g.dgu, b.n_rows, stream)
    B.moe_grouped_mm_dw(g.dgu, x, b.offsets, g.dgate_up, g.workspace, b.perm, k, stream)
    B.moe_grouped_mm_dx(g.dgu, experts.gate_up, b.offsets, g.dx_slots, stream)
    if b.y_shared is not None:
        B.moe_grouped_mm_dw(dout, b.h_shared, b.all_rows, g.dshared_down, g.workspace, stream=stream)
        B.moe_grouped_mm_dx(dout, experts.shared_down, b.all_rows, g.dh_shared, stream)
        B.moe_swiglu_grad(b.gu_shared, g.dh_shared, g.dgu_shared, stream=stream)
        B.moe_grouped_mm_dw(g.dgu_shared, x, b.all_rows, g.dshared_gate_up, g.workspace,
                            stream=stream)
        B.moe_grouped_mm_dx(g.dgu_shared, experts.shared_gate_up, b.all_rows, g.dx_shared, stream)
    # a token's gradient is the sum over its slots: the combine with weights of 1
    with _gpu_of(b.gu):
        B.moe_combine(sh, g.dx_slots, g.dx_shared, b.inv_perm, g.ones, g.dx, stream)
    return g


class AdamW:
    """AdamW over a list of tensors and their gradients (buffers that later
    backward passes fill again): moments in float32 or, with bits=8, in codes, a
    float32 master of each bf16 parameter (masters=False: none), and the step's
    number on the device, so that a captured step counts on.  A saved state (count,
    masters, m, v and the scales) is copied into these tensors: a step refuses ones
    that were given other memory."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 bits: int = 32, masters: bool = True):
        if bits not in (8, 32):
            raise ValueError(f"AdamW: moments of {bits} bits; 8 or 32")
        if not params:
            raise ValueError("AdamW: no parameters")
        self.params, self.grads = tuple(params), tuple(grads)
        dev = self.params[0].device
        new = lambda p, dt: torch.zeros(p.shape, dtype=dt, device=p.device)  # noqa: E731
        # tuples: an entry put in later would not be the step's
        self.masters = tuple(p.detach().float() if masters and p.dtype == torch.bfloat16 else None
                             for p in self.params)
        each = lambda make: tuple(make(p) for p in self.params)  # noqa: E731
        if bits == 32:
            self.m, self.v = (each(lambda p: new(p, torch.float32)) for _ in range(2))
            self.m_scales = self.v_scales = None
        else:
            self.m = each(lambda p: new(p, torch.float8_e4m3fn))
            self.v = each(lambda p: new(p, torch.uint8))
            ones = lambda p: torch.ones(-(-p.numel() // 256), device=p.device)  # noqa: E731
            self.m_scales, self.v_scales = (each(ones) for _ in range(2))
        self.count = torch.zeros(1, dtype=torch.int64, device=dev)
        self.tensors = B.AdamWTensors(self.params, self.grads, self.m, self.v, self.masters,
                                      self.m_scales, self.v_scales)

    @classmethod
    def of_experts(cls, experts: FloatExperts, grads: "FloatLayerGrads", bits: int = 32,
                   masters: bool = True) -> "AdamW":
        """The bf16 weights of a layer with run_layer_float_grad's gradients."""
        pairs = [(experts.gate_up, grads.dgate_up), (experts.down, grads.ddown),
                 (experts.shared_gate_up, grads.dshared_gate_up),
                 (experts.shared_down, grads.dshared_down)]
        pairs = [(p, g) for p, g in pairs if p is not None]
        return cls([p for p, _ in pairs], [g for _, g in pairs], bits, masters)

    def step(self, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             weight_decay: float = 0.0, grad_scale=None, stream=None):
        """One step on `stream`, or the current one (moe_adamw)."""
        side = _torch_stream(stream, self.count.device)
        turn = lambda: contextlib.nullcontext() if side is None else torch.cuda.stream(side)  # noqa: E731
        with turn():
            self.count += 1
        try:
            B.moe_adamw(self.tensors, self.count, lr, beta1, beta2, eps, weight_decay, grad_scale,
                        stream)
        except Exception:
            with turn():
                self.count -= 1  # a step that was refused is none
            raise


@dataclasses.dataclass
class BlockNorms:
    """A block's norm weights [d] float32 (None: no such norm), its gate ([1 or
    T, d] of the layer output's type, or None) and its residual scale."""
    w_pre: torch.Tensor
    w_post: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    scale: float = 1.0
    eps: float = 1e-6


def run_block(res, norms: BlockNorms, layer, normed, res_out, next_norms=None, next_normed=None,
              stream=None, normed_ready=False):
    """res_out = res + scale * gate * norm(layer(norm(res))) for the residual
    stream res [T, d]; layer: a function of the normed tokens [T, d] (normed, a
    buffer of the type it takes), such as run_layer or run_layer_float with the
    rest bound; it is called with `stream` as the current one.  With next_norms,
    next_normed gets the next block's pre norm in the same pass: hand it to that
    block as its `normed`, with normed_ready, and its first norm is not done
    again.  The post norm and the next pre norm share their eps; without a post
    norm the next one's holds."""
    eps = norms.eps
    if next_norms is not None and next_norms.eps != eps:
        if norms.w_post is not None:
            raise ValueError(f"run_block: a post norm with eps {eps} and a next pre norm with "
                             f"{next_norms.eps} are not one pass")
        eps = next_norms.eps
    if not normed_ready:
        B.moe_block_norm(None, res, None, normed, w_pre=norms.w_pre, eps=norms.eps, stream=stream)
    side = _torch_stream(stream, res.device)
    with contextlib.nullcontext() if side is None else torch.cuda.stream(side):
        out = layer(normed)
    B.moe_block_norm(out, res, res_out, next_normed, norms.w_post,
                     None if next_norms is None else next_norms.w_pre, norms.gate, norms.scale,
                     eps, stream)
    return res_out
