"""Device buffers for one layer call and the four-call sequence.

Plumbing only: torch allocates the caller-owned device memory the C ABI
expects, and ``run_layer`` issues moe_route_union -> moe_expert_ffn ->
moe_combine on one stream with no host synchronisation in between;
``run_layer_decode`` makes the single moe_layer_decode call instead (decode
batches of at most 8 tokens).

``run_layer_float`` is the layer on bfloat16 expert weights, or on e4m3 codes
with block scales, ``run_layer_float_grad`` its gradient (the routing taken as
given), and ``run_block`` any of them between its norms and residual.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

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
    or e4m3 codes with their scales per 128 x 128 ([E, 2 f / 128, d / 128] and
    [E, d / 128, f / 128], rounded up)."""
    gate_up: torch.Tensor
    down: torch.Tensor
    shared_gate_up: Optional[torch.Tensor] = None
    shared_down: Optional[torch.Tensor] = None
    scales: Optional[tuple] = None         # (gate_up, down) of codes
    shared_scales: Optional[tuple] = None

    @classmethod
    def quantize(cls, e: "FloatExperts", stream=None) -> "FloatExperts":
        """e's bf16 weights as codes and scales (moe_blockscale_quantize), ready
        on `stream`.  Their memory is the current stream's: another one waits for
        what is queued there first, and holds on to all it touches."""
        side = _torch_stream(stream, e.gate_up.device)

        def q(w):
            if w is None:
                return None, None
            n, r, k = w.shape
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

    @classmethod
    def allocate(cls, shape, T: int, codes: bool = False, device="cuda",
                 y_dtype=torch.bfloat16, out_dtype=torch.bfloat16):
        sh = B._shape(shape)
        k, E, d, f, P = sh.top_k, sh.n_experts, sh.d, sh.f, T * sh.top_k
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        i32 = torch.int32

        def pair(rows, cols):
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
            workspace=new(max(B.moe_route_workspace_bytes(sh, T), 256), dtype=torch.uint8))


def _check_float(fn: str, x, experts: FloatExperts, buf: FloatLayerBuffers):
    if tuple(x.shape) != (buf.T, buf.shape.d):
        raise ValueError(f"{fn}: x has shape {tuple(x.shape)}, the buffers hold "
                         f"{(buf.T, buf.shape.d)}")
    if (experts.shared_gate_up is None) != (buf.y_shared is None):
        raise ValueError(f"{fn}: the shape and the weights disagree about a shared expert")
    if (experts.scales is None) != (buf.codes is None):
        raise ValueError(f"{fn}: 8-bit experts take buffers allocated with codes=True, bf16 ones "
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
    the gathered tokens, SwiGLU, down products, combine."""
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
        (xq, xs), (hq, hs) = b.codes["x"], b.codes["h"]
        gus, dns = experts.scales
        B.moe_blockscale_quantize(x, 1, xq, xs, stream)
        B.moe_blockscale_mm(xq, xs, experts.gate_up, gus, b.offsets, b.gu, b.perm, k, stream)
        B.moe_swiglu_quantize(b.gu, hq, hs, b.n_rows, stream)
        B.moe_blockscale_mm(hq, hs, experts.down, dns, b.offsets, b.y, stream=stream)
        if b.y_shared is not None:
            (hq, hs), (gus, dns) = b.codes["h_shared"], experts.shared_scales
            B.moe_blockscale_mm(xq, xs, experts.shared_gate_up, gus, b.all_rows, b.gu_shared,
                                stream=stream)
            B.moe_swiglu_quantize(b.gu_shared, hq, hs, stream=stream)
            B.moe_blockscale_mm(hq, hs, experts.shared_down, dns, b.all_rows, b.y_shared,
                                stream=stream)
    with _gpu_of(b.gu):
        B.moe_combine(sh, b.y, b.y_shared, b.inv_perm, b.topk_w, b.out, stream)
    return b.out


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
