"""ctypes binding of libmoe_int4.so: one Python function per C entry point,
with the same name.  Argument marshalling only -- every step of the layer
runs in the library's HIP kernels.  PyTorch supplies device memory and the
current HIP stream.

Loading fails loudly when the library has not been built; there is no other
implementation behind these functions.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_int32, c_size_t, c_void_p, POINTER

LIB_NAME = "libmoe_int4.so"
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), LIB_NAME)

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_ALIGN = 0, 1, 2, 3, 4
MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 5, 6, 7
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_DTYPE",
                4: "MOE_ERR_ALIGN", 5: "MOE_ERR_UNSUPPORTED", 6: "MOE_ERR_WORKSPACE",
                7: "MOE_ERR_HIP"}
MOE_F32, MOE_BF16 = 0, 1
MOE_PATH_DECODE_F32, MOE_PATH_PREFILL_BF16 = 0, 1
MOE_QUANT_GS64, MOE_QUANT_ROW = 0, 1
MOE_WEIGHTS_BF16, MOE_WEIGHTS_E4M3, MOE_WEIGHTS_INT8 = 0, 1, 2

# every function include/moe_int4.h declares
EXPORTS = ("moe_expert_bytes", "moe_pack_experts", "moe_quantize", "moe_route_workspace_bytes",
           "moe_route", "moe_union", "moe_route_union", "moe_ffn_workspace_bytes",
           "moe_expert_ffn", "moe_combine", "moe_layer_decode_workspace_bytes",
           "moe_layer_decode", "moe_layer_decode_static", "moe_layer_decode_static_max_bytes",
           "moe_cache_create", "moe_cache_destroy", "moe_cache_pin",
           "moe_cache_plan", "moe_cache_stats", "moe_cache_last_fetch", "moe_cache_unplan_last",
           "moe_cache_workspace_bytes",
           "moe_cache_layer_decode", "moe_status_str", "moe_measure_stream_read",
           "moe_grouped_mm", "moe_grouped_mm_dx", "moe_grouped_mm_dw",
           "moe_grouped_mm_dw_workspace_bytes", "moe_blockscale_quantize", "moe_blockscale_mm",
           "moe_rowscale_quantize", "moe_rowscale_mm", "moe_swiglu_rowscale",
           "moe_layer_few", "moe_layer_few_workspace_bytes", "moe_adamw",
           "moe_swiglu", "moe_swiglu_quantize", "moe_swiglu_grad", "moe_combine_grad",
           "moe_block_norm", "moe_block_norm_grad", "moe_block_norm_grad_workspace_bytes")


class Shape(ctypes.Structure):
    """moe_shape: d, f, n_experts, top_k, group, f_shared (all int32)."""
    _fields_ = [("d", c_int32), ("f", c_int32), ("n_experts", c_int32), ("top_k", c_int32),
                ("group", c_int32), ("f_shared", c_int32)]

    def __repr__(self):
        return (f"Shape(d={self.d}, f={self.f}, n_experts={self.n_experts}, top_k={self.top_k}, "
                f"group={self.group}, f_shared={self.f_shared})")


class ExpertWeights(ctypes.Structure):
    """moe_expert_weights: device addresses."""
    _fields_ = [(name, c_void_p) for name in ("gate_up", "down", "gate_up_scales", "down_scales")]


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor: an element count, device addresses, two moe_dtypes."""
    _fields_ = ([("n", ctypes.c_int64)] +
                [(name, c_void_p) for name in ("p", "master", "g", "m", "v", "m_scales",
                                               "v_scales")] +
                [("p_dt", c_int32), ("g_dt", c_int32)])


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({_status_text(status)})")


_lib = None


def load():
    """Load the shared library (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m int4_routed_expert_logits_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    sp = POINTER(Shape)
    lib.moe_expert_bytes.argtypes = [c_int32, c_int32, c_int32]
    lib.moe_expert_bytes.restype = c_size_t
    lib.moe_route_workspace_bytes.argtypes = [sp, c_int32]
    lib.moe_route_workspace_bytes.restype = c_size_t
    lib.moe_ffn_workspace_bytes.argtypes = [sp, c_int32, c_int32]
    lib.moe_ffn_workspace_bytes.restype = c_size_t
    lib.moe_route.argtypes = [sp, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_void_p, c_size_t, c_void_p]
    lib.moe_route.restype = c_int32
    lib.moe_union.argtypes = [sp, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_void_p, c_void_p]
    lib.moe_union.restype = c_int32
    lib.moe_route_union.argtypes = [sp, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_size_t, c_void_p]
    lib.moe_route_union.restype = c_int32
    lib.moe_expert_ffn.argtypes = [sp, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
                                   c_void_p, c_size_t, c_void_p]
    lib.moe_expert_ffn.restype = c_int32
    lib.moe_combine.argtypes = [sp, c_int32, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
                                c_void_p, c_int32, c_void_p]
    lib.moe_combine.restype = c_int32
    lib.moe_layer_decode_workspace_bytes.argtypes = [sp, c_int32]
    lib.moe_layer_decode_workspace_bytes.restype = c_size_t
    lib.moe_layer_decode.argtypes = ([sp, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                      c_void_p] + [c_void_p] * 11 + [c_int32, c_void_p, c_size_t,
                                                                     c_void_p])
    lib.moe_layer_decode.restype = c_int32
    lib.moe_layer_decode_static.argtypes = ([sp, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                             c_void_p, c_void_p] + [c_void_p] * 11 +
                                            [c_int32, c_void_p])
    lib.moe_layer_decode_static.restype = c_int32
    lib.moe_measure_stream_read.argtypes = [c_void_p, c_int32, c_size_t, c_int32, c_void_p,
                                            c_void_p]
    lib.moe_measure_stream_read.restype = c_int32
    lib.moe_layer_decode_static_max_bytes.argtypes = []
    lib.moe_layer_decode_static_max_bytes.restype = c_size_t
    vp = c_void_p
    lib.moe_cache_create.argtypes = [sp, c_int32, vp, vp, POINTER(vp)]
    lib.moe_cache_create.restype = c_int32
    lib.moe_cache_destroy.argtypes = [vp]
    lib.moe_cache_destroy.restype = None
    lib.moe_cache_pin.argtypes = [vp, c_int32, c_int32]
    lib.moe_cache_pin.restype = c_int32
    lib.moe_cache_plan.argtypes = [vp, c_int32, vp, vp, vp, vp, vp]
    lib.moe_cache_plan.restype = c_int32
    lib.moe_cache_stats.argtypes = [vp, vp, vp, vp]
    lib.moe_cache_stats.restype = c_int32
    lib.moe_cache_last_fetch.argtypes = [vp, c_int32, vp, vp, vp]
    lib.moe_cache_last_fetch.restype = c_int32
    lib.moe_cache_unplan_last.argtypes = [vp]
    lib.moe_cache_unplan_last.restype = c_int32
    lib.moe_cache_workspace_bytes.argtypes = [sp, c_int32, c_int32]
    lib.moe_cache_workspace_bytes.restype = c_size_t
    lib.moe_cache_layer_decode.argtypes = [vp, c_int32, vp, c_int32, vp, vp, vp, vp, vp, vp, vp,
                                           vp, c_int32, vp, c_size_t, vp, vp]
    lib.moe_cache_layer_decode.restype = c_int32
    lib.moe_pack_experts.argtypes = [sp, ctypes.c_int64, c_void_p, c_void_p, c_void_p]
    lib.moe_pack_experts.restype = c_int32
    lib.moe_quantize.argtypes = [c_int32, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                 c_void_p]
    lib.moe_quantize.restype = c_int32
    i32, f32, sz = c_int32, ctypes.c_float, c_size_t
    for name, args, res in (
            ("moe_grouped_mm", [i32] * 4 + [vp, i32, vp, i32, vp, vp, vp, i32, vp], i32),
            ("moe_grouped_mm_dx", [i32] * 4 + [vp, vp, vp, vp, i32, vp], i32),
            ("moe_grouped_mm_dw_workspace_bytes", [i32] * 4, sz),
            ("moe_grouped_mm_dw", [i32] * 4 + [vp, vp, i32, vp, i32, vp, vp, i32, vp, sz, vp], i32),
            ("moe_blockscale_quantize", [i32] * 3 + [vp, i32, i32, vp, vp, vp], i32),
            ("moe_blockscale_mm",
             [i32] * 4 + [vp, vp, i32, vp, i32, vp, vp, vp, vp, i32, vp], i32),
            ("moe_swiglu", [i32, i32, vp, vp, i32, vp, vp], i32),
            ("moe_swiglu_quantize", [i32, i32, vp, i32, vp, vp, vp, vp], i32),
            ("moe_rowscale_quantize", [i32, i32, vp, i32, vp, vp, vp], i32),
            ("moe_rowscale_mm", [i32] * 4 + [vp, vp, i32, vp, i32, vp, vp, vp, vp, i32, vp], i32),
            ("moe_swiglu_rowscale", [i32, i32, vp, i32, vp, vp, vp, vp], i32),
            ("moe_layer_few_workspace_bytes", [sp, i32], sz),
            ("moe_layer_few", [sp, i32, vp, vp, vp, i32, POINTER(ExpertWeights),
                               POINTER(ExpertWeights), vp, vp, vp, i32, vp, sz, vp], i32),
            ("moe_adamw", [POINTER(AdamWTensor), i32, vp] + [ctypes.c_double] * 5 + [vp, vp], i32),
            ("moe_swiglu_grad", [i32, i32, vp, vp, vp, i32, vp, vp], i32),
            ("moe_combine_grad", [sp, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp], i32),
            ("moe_block_norm", [i32, i32, vp, i32, vp, vp, i32, f32, vp, i32, vp, vp, f32, vp, i32,
                                vp], i32),
            ("moe_block_norm_grad_workspace_bytes", [i32, i32], sz),
            ("moe_block_norm_grad", [i32, i32, vp, i32, vp, vp, i32, f32, vp, i32, vp, f32, vp, vp,
                                     i32, vp, vp, vp, vp, vp, vp, sz, vp], i32)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    lib.moe_status_str.argtypes = [c_int32]
    lib.moe_status_str.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _status_text(status: int) -> str:
    try:
        return load().moe_status_str(status).decode()
    except Exception:  # pragma: no cover - only when the library itself is missing
        return "?"


# ----------------------------------------------------------------------------
# marshalling helpers
# ----------------------------------------------------------------------------

def _ptr(t):
    """Device address of a tensor (None -> NULL).  Raw integers pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dtype(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def _shape(shape):
    if isinstance(shape, Shape):
        return shape
    return Shape(*shape)


# ----------------------------------------------------------------------------
# the C entry points, one to one
# ----------------------------------------------------------------------------

def moe_expert_bytes(d: int, f: int, group: int = 64) -> int:
    return load().moe_expert_bytes(d, f, group)


def moe_pack_experts(shape, n_blocks: int, src, dst, stream=None):
    """Canonical expert blocks (uint8 device tensor) -> packed blocks."""
    sh = _shape(shape)
    _check("moe_pack_experts", load().moe_pack_experts(ctypes.byref(sh), n_blocks, _ptr(src),
                                                       _ptr(dst), _stream(stream)))


def moe_quantize(w, mode, codes, scales, stream=None):
    """w [N, K] bf16/f32 -> codes [N, K/2] uint8 and float16 scales
    ([N, K/64] for MOE_QUANT_GS64, [N] for MOE_QUANT_ROW)."""
    n, k = w.shape
    _check("moe_quantize", load().moe_quantize(n, k, _ptr(w), _dtype(w), mode, _ptr(codes),
                                               _ptr(scales), _stream(stream)))


def moe_route_workspace_bytes(shape, T: int) -> int:
    return load().moe_route_workspace_bytes(ctypes.byref(_shape(shape)), T)


def moe_ffn_workspace_bytes(shape, T: int, path: int) -> int:
    return load().moe_ffn_workspace_bytes(ctypes.byref(_shape(shape)), T, path)


def moe_layer_decode_workspace_bytes(shape, T: int) -> int:
    return load().moe_layer_decode_workspace_bytes(ctypes.byref(_shape(shape)), T)


def moe_status_str(status: int) -> str:
    return load().moe_status_str(status).decode()


def moe_route(shape, x, w_router, bias, topk_idx, topk_w, workspace, stream=None):
    """x [T, d] bf16/f32; writes topk_idx [T, k] int32 and topk_w [T, k] f32."""
    sh = _shape(shape)
    _check("moe_route", load().moe_route(
        ctypes.byref(sh), x.shape[0], _ptr(x), _dtype(x), _ptr(w_router), _ptr(bias),
        _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_union(shape, T, topk_idx, counts, offsets, perm, inv_perm, active, n_active, stream=None):
    sh = _shape(shape)
    _check("moe_union", load().moe_union(
        ctypes.byref(sh), T, _ptr(topk_idx), _ptr(counts), _ptr(offsets), _ptr(perm),
        _ptr(inv_perm), _ptr(active), _ptr(n_active), _stream(stream)))


def moe_route_union(shape, x, w_router, bias, topk_idx, topk_w, counts, offsets, perm, inv_perm,
                    active, n_active, workspace, stream=None):
    """moe_route then moe_union in one call (same outputs)."""
    sh = _shape(shape)
    _check("moe_route_union", load().moe_route_union(
        ctypes.byref(sh), x.shape[0], _ptr(x), _dtype(x), _ptr(w_router), _ptr(bias),
        _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv_perm),
        _ptr(active), _ptr(n_active), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_expert_ffn(shape, x, experts, shared, offsets, perm, active, n_active, path, y, y_shared,
                   workspace, stream=None):
    sh = _shape(shape)
    _check("moe_expert_ffn", load().moe_expert_ffn(
        ctypes.byref(sh), x.shape[0], _ptr(x), _dtype(x), _ptr(experts), _ptr(shared),
        _ptr(offsets), _ptr(perm), _ptr(active), _ptr(n_active), path, _ptr(y), _ptr(y_shared),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_combine(shape, y, y_shared, inv_perm, topk_w, out, stream=None):
    sh = _shape(shape)
    _check("moe_combine", load().moe_combine(
        ctypes.byref(sh), out.shape[0], _ptr(y), _ptr(y_shared), _dtype(y), _ptr(inv_perm),
        _ptr(topk_w), _ptr(out), _dtype(out), _stream(stream)))


def moe_layer_decode(shape, x, w_router, bias, experts, shared, topk_idx, topk_w, counts, offsets,
                     perm, inv_perm, active, n_active, y, y_shared, out, workspace, stream=None):
    """The whole layer for a decode batch of T <= 8 tokens (route, union,
    expert FFN, combine): the same outputs as the separate calls."""
    sh = _shape(shape)
    _check("moe_layer_decode", load().moe_layer_decode(
        ctypes.byref(sh), x.shape[0], _ptr(x), _dtype(x), _ptr(w_router), _ptr(bias),
        _ptr(experts), _ptr(shared), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
        _ptr(perm), _ptr(inv_perm), _ptr(active), _ptr(n_active), _ptr(y), _ptr(y_shared),
        _ptr(out), _dtype(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_layer_decode_static_max_bytes() -> int:
    return load().moe_layer_decode_static_max_bytes()


def moe_layer_decode_static(shape, x, w_router, bias, experts, shared, topk_idx, topk_w, counts,
                            offsets, perm, inv_perm, active, n_active, y, y_shared, out,
                            stream=None):
    """moe_layer_decode without a workspace: the library's static per-GPU
    scratch array stands in for it (include/moe_int4_static.h)."""
    sh = _shape(shape)
    _check("moe_layer_decode_static", load().moe_layer_decode_static(
        ctypes.byref(sh), x.shape[0], _ptr(x), _dtype(x), _ptr(w_router), _ptr(bias),
        _ptr(experts), _ptr(shared), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
        _ptr(perm), _ptr(inv_perm), _ptr(active), _ptr(n_active), _ptr(y), _ptr(y_shared),
        _ptr(out), _dtype(out), _stream(stream)))


def moe_measure_stream_read(block_ptrs, block_bytes: int, workgroups: int, sink, stream=None):
    """Calibration read of the device blocks at block_ptrs (ints) once
    (include/moe_int4_measure.h); sink: a device int32 tensor of at least
    `workgroups` entries."""
    arr = (c_void_p * len(block_ptrs))(*block_ptrs)
    _check("moe_measure_stream_read", load().moe_measure_stream_read(
        arr, len(block_ptrs), block_bytes, workgroups, _ptr(sink), _stream(stream)))


# ----------------------------------------------------------------------------
# per-layer expert cache
# ----------------------------------------------------------------------------

def moe_cache_create(shape, n_slots: int, device_slots=None, host_blocks=None) -> int:
    """Handle of a new cache (device_slots / host_blocks: tensors or None
    for a planning-only cache)."""
    h = c_void_p()
    _check("moe_cache_create", load().moe_cache_create(
        ctypes.byref(_shape(shape)), n_slots, _ptr(device_slots), _ptr(host_blocks),
        ctypes.byref(h)))
    return h.value


def moe_cache_destroy(cache: int):
    load().moe_cache_destroy(cache)


def moe_cache_pin(cache: int, expert: int, pinned: bool = True):
    _check("moe_cache_pin", load().moe_cache_pin(cache, expert, 1 if pinned else 0))


def moe_cache_plan(cache: int, experts):
    """One policy step on a planning-only cache: experts (host ints) ->
    (slot_of per entry, fetched experts in placement order, the expert each
    displaced or -1)."""
    import numpy as np
    e = np.ascontiguousarray(np.asarray(experts, dtype=np.int32))
    n = e.size
    slot_of = np.empty(max(n, 1), np.int32)
    fetched = np.empty(max(n, 1), np.int32)
    evicted = np.empty(max(n, 1), np.int32)
    nf = c_int32(0)
    _check("moe_cache_plan", load().moe_cache_plan(
        cache, n, e.ctypes.data, slot_of.ctypes.data, fetched.ctypes.data, evicted.ctypes.data,
        ctypes.addressof(nf)))
    k = nf.value
    return slot_of[:n].copy(), fetched[:k].copy(), evicted[:k].copy()


def moe_cache_stats(cache: int):
    """(hits, misses, bytes fetched) since creation."""
    h, m, b = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check("moe_cache_stats", load().moe_cache_stats(cache, ctypes.addressof(h),
                                                     ctypes.addressof(m), ctypes.addressof(b)))
    return h.value, m.value, b.value


def moe_cache_last_fetch(cache: int, capacity: int):
    """The latest step's fetched experts in placement order and the expert
    each displaced (-1 for an empty slot): (fetched, evicted) lists."""
    f = (ctypes.c_int32 * max(capacity, 1))()
    e = (ctypes.c_int32 * max(capacity, 1))()
    n = ctypes.c_int32()
    _check("moe_cache_last_fetch", load().moe_cache_last_fetch(
        cache, capacity, ctypes.addressof(f), ctypes.addressof(e), ctypes.addressof(n)))
    return list(f[:n.value]), list(e[:n.value])


def moe_cache_unplan_last(cache: int) -> None:
    """Undo the latest step's placements (its fetched slots become empty)."""
    _check("moe_cache_unplan_last", load().moe_cache_unplan_last(cache))


def moe_cache_workspace_bytes(shape, T: int, n_slots: int) -> int:
    return load().moe_cache_workspace_bytes(ctypes.byref(_shape(shape)), T, n_slots)


def moe_cache_layer_decode(cache: int, x, w_router, bias, shared, topk_idx, topk_w, y, y_shared,
                           out, workspace, stream=None, copy_stream=None):
    """One decode step of the layer through the cache (copies of missing
    experts on copy_stream, overlapped with the resident experts' FFN)."""
    _check("moe_cache_layer_decode", load().moe_cache_layer_decode(
        cache, x.shape[0], _ptr(x), _dtype(x), _ptr(w_router), _ptr(bias), _ptr(shared),
        _ptr(topk_idx), _ptr(topk_w), _ptr(y), _ptr(y_shared), _ptr(out), _dtype(out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream),
        _stream(copy_stream) if copy_stream is not None else _stream(stream)))


# ----------------------------------------------------------------------------
# float and 8-bit expert weights, gradients, block norms
# (include/moe_int4_block.h)
#
# These take whole tensors and check them first: each on the GPU of the first
# one, without gaps, of the named type and shape (TypeError, ValueError); the
# sizes' limits are the library's (MoeError).  A call runs on the tensors'
# GPU, on `stream` or on that GPU's current stream.
# ----------------------------------------------------------------------------

# set by _types(), which every call below makes first (once: `_T or _types()`)
_T = _raw_stream = _current_device = _INT8 = _INT64 = _same_memory = _written = None
_CODES = {}  # torch type -> moe_dtype


def _types():
    """(bf16, f32, either, int32, e4m3 code) as tuples of torch types."""
    global _T, _raw_stream, _current_device, _INT8, _INT64, _same_memory, _written
    if _T is None:
        import torch
        # the stream's handle and the device's index themselves: building a torch
        # Stream takes as long as a launch
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _current_device = _current_device or torch._C._cuda_getDevice
        _INT8, _INT64 = (torch.int8,), (torch.int64,)
        _same_memory = torch._C._tensors_data_ptrs_at_indices_equal
        _written = torch.autograd.graph.increment_version
        _CODES.update({torch.bfloat16: MOE_BF16, torch.float32: MOE_F32})
        _T = ((torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32), (torch.int32,),
              (torch.float8_e4m3fn, torch.uint8))
    return _T


def _take(fn: str, dev: int, name: str, t, dtypes, shape):
    """t's address, after checking it (None passes as NULL)."""
    if t is None:
        return None
    if t.dtype in dtypes and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{fn}: {name} is {t.dtype}, not {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on the first tensor's GPU ({dev})")
    raise ValueError(f"{fn}: {name} is not contiguous")


_INT32_MAX = 2 ** 31 - 1


def _dim(fn: str, name: str, t, n: int):
    """t's shape, of n sizes that int32 holds (ctypes would wrap larger ones)."""
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{fn}: {name} has {len(shape)} dimensions, not {n}")
    if max(shape) > _INT32_MAX:
        raise MoeError(fn, MOE_ERR_UNSUPPORTED)
    return shape


def _int32(fn: str, v: int) -> int:
    if not -_INT32_MAX <= v <= _INT32_MAX:
        raise MoeError(fn, MOE_ERR_UNSUPPORTED)
    return v


def _workspace(fn: str, dev: int, t):
    """(address, bytes) of a workspace tensor of any type; (NULL, 0) for None."""
    if t is None:
        return None, 0
    return _take(fn, dev, "workspace", t, (t.dtype,), t.shape), t.numel() * t.element_size()


def _run(fn: str, dev: int, stream, *args):
    """One C call with GPU dev current, on `stream` or dev's current stream."""
    if dev < 0:
        raise ValueError(f"{fn}: the tensors are not on the GPU")
    call = getattr(_lib or load(), fn)
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current_device() == dev:
        status = call(*args, stream)
    else:
        import torch
        with torch.cuda.device(dev):
            status = call(*args, stream)
    if status != MOE_OK:
        raise MoeError(fn, status)


def _rows_args(fn, dev, P, rows):
    return None if rows is None else _take(fn, dev, "rows", rows, (_T or _types())[3], (P,))


def moe_grouped_mm(x, w, offsets, y, rows=None, rows_div: int = 1, stream=None):
    """y[p] = w[e] x[rows[p] // rows_div] (x[p] without rows): x [X, K] bf16,
    w [E, N, K] bf16, offsets [E + 1] and rows [P] int32, y [P, N] bf16/f32."""
    fn, dev = "moe_grouped_mm", x.get_device()
    bf16, _, floats, i32, _ = _T or _types()
    E, N, K = _dim(fn, "w", w, 3)
    P, X = _dim(fn, "y", y, 2)[0], _dim(fn, "x", x, 2)[0]
    _run(fn, dev, stream, E, P, N, K, _take(fn, dev, "x", x, bf16, (X, K)), X,
         _rows_args(fn, dev, P, rows), _int32(fn, rows_div),
         _take(fn, dev, "w", w, bf16, (E, N, K)),
         _take(fn, dev, "offsets", offsets, i32, (E + 1,)),
         _take(fn, dev, "y", y, floats, (P, N)), _code(y.dtype))


def moe_grouped_mm_dx(dy, w, offsets, dx, stream=None):
    """dx[p] = w[e]^T dy[p]: dy [P, N] bf16, w [E, N, K] bf16, dx [P, K] bf16/f32."""
    fn, dev = "moe_grouped_mm_dx", dy.get_device()
    bf16, _, floats, i32, _ = _T or _types()
    E, N, K = _dim(fn, "w", w, 3)
    P = _dim(fn, "dx", dx, 2)[0]
    _run(fn, dev, stream, E, P, N, K, _take(fn, dev, "dy", dy, bf16, (P, N)),
         _take(fn, dev, "w", w, bf16, (E, N, K)),
         _take(fn, dev, "offsets", offsets, i32, (E + 1,)),
         _take(fn, dev, "dx", dx, floats, (P, K)), _code(dx.dtype))


def moe_grouped_mm_dw_workspace_bytes(E: int, P: int, N: int, K: int) -> int:
    if max(E, P, N, K) > _INT32_MAX or min(E, P, N, K) < 0:
        return 0
    return load().moe_grouped_mm_dw_workspace_bytes(E, P, N, K)


def moe_grouped_mm_dw(dy, x, offsets, dw, workspace=None, rows=None, rows_div: int = 1,
                      stream=None):
    """dw[e] = sum over e's positions of dy[p] x[row(p)]^T: dy [P, N] and
    x [X, K] bf16, dw [E, N, K] bf16/f32 (all of it written)."""
    fn, dev = "moe_grouped_mm_dw", dy.get_device()
    bf16, _, floats, i32, _ = _T or _types()
    E, N, K = _dim(fn, "dw", dw, 3)
    P, X = _dim(fn, "dy", dy, 2)[0], _dim(fn, "x", x, 2)[0]
    ws, nws = _workspace(fn, dev, workspace)
    _run(fn, dev, stream, E, P, N, K, _take(fn, dev, "dy", dy, bf16, (P, N)),
         _take(fn, dev, "x", x, bf16, (X, K)), X,
         _rows_args(fn, dev, P, rows), _int32(fn, rows_div),
         _take(fn, dev, "offsets", offsets, i32, (E + 1,)),
         _take(fn, dev, "dw", dw, floats, (E, N, K)), _code(dw.dtype), ws, nws)


def moe_blockscale_quantize(x, block_rows: int, codes, scales, stream=None):
    """x [R, K] or [n, R, K] bf16/f32 -> e4m3 codes of x's shape
    (float8_e4m3fn or uint8) and float32 scales per 128 columns: [.., R, K/128]
    for block_rows 1, [.., R/128, K/128] for 128 (rounded up)."""
    fn, dev = "moe_blockscale_quantize", x.get_device()
    _, f32, floats, _, codes_t = _T or _types()
    if x.dim() not in (2, 3):
        raise ValueError(f"{fn}: x has {x.dim()} dimensions, not 2 or 3")
    *lead, R, K = _dim(fn, "x", x, x.dim())
    sr = R if block_rows == 1 else -(-R // 128)
    _run(fn, dev, stream, lead[0] if lead else 1, R, K, _take(fn, dev, "x", x, floats, x.shape),
         _code(x.dtype), _int32(fn, block_rows), _take(fn, dev, "codes", codes, codes_t, x.shape),
         _take(fn, dev, "scales", scales, f32, (*lead, sr, -(-K // 128))))


def moe_blockscale_mm(xq, xs, wq, ws, offsets, y, rows=None, rows_div: int = 1, stream=None):
    """moe_grouped_mm over e4m3 codes: xq [X, K] with xs [X, K/128], wq
    [E, N, K] with ws [E, N/128, K/128] (rounded up), y [P, N] bf16/f32."""
    fn, dev = "moe_blockscale_mm", xq.get_device()
    _, f32, floats, i32, codes_t = _T or _types()
    E, N, K = _dim(fn, "wq", wq, 3)
    P, X, kb = _dim(fn, "y", y, 2)[0], _dim(fn, "xq", xq, 2)[0], -(-K // 128)
    _run(fn, dev, stream, E, P, N, K, _take(fn, dev, "xq", xq, codes_t, (X, K)),
         _take(fn, dev, "xs", xs, f32, (X, kb)), X,
         _rows_args(fn, dev, P, rows), _int32(fn, rows_div),
         _take(fn, dev, "wq", wq, codes_t, (E, N, K)),
         _take(fn, dev, "ws", ws, f32, (E, -(-N // 128), kb)),
         _take(fn, dev, "offsets", offsets, i32, (E + 1,)),
         _take(fn, dev, "y", y, floats, (P, N)), _code(y.dtype))


def moe_rowscale_quantize(x, codes, scales, stream=None):
    """x [R, K] or [n, R, K] bf16/f32 -> int8 codes of x's shape and a float32
    scale per row ([R] or [n, R])."""
    fn, dev = "moe_rowscale_quantize", x.get_device()
    _, f32, floats, _, _ = _T or _types()
    if x.dim() not in (2, 3):
        raise ValueError(f"{fn}: x has {x.dim()} dimensions, not 2 or 3")
    shape = _dim(fn, "x", x, x.dim())
    rows = 1
    for n in shape[:-1]:
        rows *= n
    _run(fn, dev, stream, _int32(fn, rows), shape[-1], _take(fn, dev, "x", x, floats, shape),
         _code(x.dtype), _take(fn, dev, "codes", codes, _INT8, shape),
         _take(fn, dev, "scales", scales, f32, shape[:-1]))


def moe_rowscale_mm(xq, xs, wq, ws, offsets, y, rows=None, rows_div: int = 1, stream=None):
    """moe_grouped_mm over 8-bit integers: xq [X, K] int8 with xs [X], wq [E, N, K]
    int8 with ws [E, N], y [P, N] bf16/f32."""
    fn, dev = "moe_rowscale_mm", xq.get_device()
    _, f32, floats, i32, _ = _T or _types()
    E, N, K = _dim(fn, "wq", wq, 3)
    P, X = _dim(fn, "y", y, 2)[0], _dim(fn, "xq", xq, 2)[0]
    _run(fn, dev, stream, E, P, N, K, _take(fn, dev, "xq", xq, _INT8, (X, K)),
         _take(fn, dev, "xs", xs, f32, (X,)), X,
         _rows_args(fn, dev, P, rows), _int32(fn, rows_div),
         _take(fn, dev, "wq", wq, _INT8, (E, N, K)), _take(fn, dev, "ws", ws, f32, (E, N)),
         _take(fn, dev, "offsets", offsets, i32, (E + 1,)),
         _take(fn, dev, "y", y, floats, (P, N)), _code(y.dtype))


def moe_swiglu_rowscale(gu, codes, scales, n_rows=None, stream=None):
    """moe_swiglu's result as int8 codes [P, f] and a scale per row [P]."""
    fn, dev = "moe_swiglu_rowscale", gu.get_device()
    _, f32, floats, _, _ = _T or _types()
    P, f = _dim(fn, "codes", codes, 2)
    _run(fn, dev, stream, P, f, _take(fn, dev, "gu", gu, floats, (P, 2 * f)), _code(gu.dtype),
         _take(fn, dev, "codes", codes, _INT8, (P, f)),
         _take(fn, dev, "scales", scales, f32, (P,)), _n_rows(fn, dev, n_rows))


def _n_rows(fn, dev, n_rows):
    return None if n_rows is None else _take(fn, dev, "n_rows", n_rows, (_T or _types())[3], (1,))


def moe_swiglu(gu, h, n_rows=None, stream=None):
    """h = silu(gu[:, :f]) * gu[:, f:]: gu [P, 2 f], h [P, f], both bf16 or both
    f32; n_rows: device int32 [1], rows from it on are left as they were."""
    fn, dev = "moe_swiglu", gu.get_device()
    P, f = _dim(fn, "h", h, 2)
    _run(fn, dev, stream, P, f, _take(fn, dev, "gu", gu, (_T or _types())[2], (P, 2 * f)),
         _take(fn, dev, "h", h, (gu.dtype,), (P, f)), _code(gu.dtype), _n_rows(fn, dev, n_rows))


def moe_swiglu_quantize(gu, codes, scales, n_rows=None, stream=None):
    """moe_swiglu's result as e4m3 codes [P, f] and scales [P, f/128] (rounded up)."""
    fn, dev = "moe_swiglu_quantize", gu.get_device()
    _, f32, floats, _, codes_t = _T or _types()
    P, f = _dim(fn, "codes", codes, 2)
    _run(fn, dev, stream, P, f, _take(fn, dev, "gu", gu, floats, (P, 2 * f)), _code(gu.dtype),
         _take(fn, dev, "codes", codes, codes_t, (P, f)),
         _take(fn, dev, "scales", scales, f32, (P, -(-f // 128))), _n_rows(fn, dev, n_rows))


def moe_swiglu_grad(gu, dh, dgu, n_rows=None, stream=None):
    """moe_swiglu's gradient: gu, dgu [P, 2 f], dh [P, f], one type; dgu may be gu."""
    fn, dev = "moe_swiglu_grad", gu.get_device()
    P, f = _dim(fn, "dh", dh, 2)
    _run(fn, dev, stream, P, f, _take(fn, dev, "gu", gu, (_T or _types())[2], (P, 2 * f)),
         _take(fn, dev, "dh", dh, (gu.dtype,), (P, f)),
         _take(fn, dev, "dgu", dgu, (gu.dtype,), (P, 2 * f)), _code(gu.dtype), _n_rows(fn, dev, n_rows))


def moe_combine_grad(shape, dout, y, inv_perm, topk_w, dy, dtopk_w, stream=None):
    """moe_combine's gradient: dout [T, d], y and dy [T * k, d] (bf16/f32, one
    type; dy may be y), inv_perm [T * k] int32, topk_w and dtopk_w [T, k] f32."""
    fn, dev = "moe_combine_grad", dout.get_device()
    _, f32, floats, i32, _ = _T or _types()
    sh = _shape(shape)
    k, d, ydt = sh.top_k, sh.d, y.dtype
    T = _dim(fn, "dout", dout, 2)[0]
    n, by_slot = T * k, (T, k)
    _run(fn, dev, stream, ctypes.byref(sh), T, _take(fn, dev, "dout", dout, floats, (T, d)),
         _code(dout.dtype), _take(fn, dev, "y", y, floats, (n, d)), _code(ydt),
         _take(fn, dev, "inv_perm", inv_perm, i32, (n,)),
         _take(fn, dev, "topk_w", topk_w, f32, by_slot), _take(fn, dev, "dy", dy, (ydt,), (n, d)),
         _take(fn, dev, "dtopk_w", dtopk_w, f32, by_slot))


def _norm_args(fn, y, res, w_post, w_pre, gate, scale):
    """The first arguments of the block norm calls and the sizes they check by."""
    bf16, f32, floats, _, _ = _T or _types()
    first = y if y is not None else res
    if first is None:
        raise ValueError(f"{fn}: neither y nor res")
    name = "y" if y is not None else "res"
    dev, (T, d) = first.get_device(), _dim(fn, name, first, 2)
    ydt = bf16[0] if y is None else y.dtype
    rdt = ydt if res is None else res.dtype
    g = 0 if gate is None else _dim(fn, "gate", gate, 2)[0]
    head = (T, d, _take(fn, dev, "y", y, floats, (T, d)), _code(ydt),
            _take(fn, dev, "w_post", w_post, f32, (d,)),
            _take(fn, dev, "gate", gate, (ydt,), (g, d)), g, scale,
            _take(fn, dev, "res", res, (rdt,) if rdt in floats else floats, (T, d)))
    return dev, T, d, ydt, rdt, head, _take(fn, dev, "w_pre", w_pre, f32, (d,))


def moe_block_norm(y, res, res_out, normed, w_post=None, w_pre=None, gate=None, scale=1.0,
                   eps=1e-6, stream=None):
    """r = res + scale * gate * norm(y) * w_post -> res_out, norm(r) * w_pre ->
    normed: y, res, res_out, normed [T, d] bf16/f32 (res_out of res's type, or
    y's without res), w_post, w_pre [d] f32, gate [1 or T, d] of y's type.  Any
    of y, res, res_out, w_post, gate and (w_pre with normed) may be None."""
    fn = "moe_block_norm"
    _, _, floats, _, _ = _T or _types()
    dev, T, d, _, rdt, head, w2 = _norm_args(fn, y, res, w_post, w_pre, gate, scale)
    if res is None and res_out is not None:
        rdt = res_out.dtype
    _run(fn, dev, stream, *head, _code(rdt), _take(fn, dev, "res_out", res_out, (rdt,), (T, d)),
         w2, eps, _take(fn, dev, "normed", normed, floats, (T, d)),
         MOE_F32 if normed is None else _code(normed.dtype))


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def moe_block_norm_grad_workspace_bytes(T: int, d: int) -> int:
    if max(T, d) > _INT32_MAX or min(T, d) < 0:
        return 0
    return load().moe_block_norm_grad_workspace_bytes(T, d)


def moe_block_norm_grad(y, res, dr, dn, dy, dres, dw_post, dw_pre, dgate, w_post=None, w_pre=None,
                        gate=None, scale=1.0, eps=1e-6, workspace=None, stream=None):
    """moe_block_norm's gradient at the same inputs, given dr (of res_out, of
    its type; or None) and dn (of normed): dy, dres [T, d], dw_post, dw_pre [d],
    dgate of gate's shape, each None where not wanted."""
    fn = "moe_block_norm_grad"
    _, f32, floats, _, _ = _T or _types()
    dev, T, d, ydt, rdt, head, w2 = _norm_args(fn, y, res, w_post, w_pre, gate, scale)
    if res is None:
        rdt = dr.dtype if dr is not None else dres.dtype if dres is not None else rdt
    ws, nws = _workspace(fn, dev, workspace)
    _run(fn, dev, stream, *head, _code(rdt), w2, eps, _take(fn, dev, "dr", dr, (rdt,), (T, d)),
         _take(fn, dev, "dn", dn, floats, (T, d)), MOE_F32 if dn is None else _code(dn.dtype),
         _take(fn, dev, "dy", dy, (ydt,), (T, d)), _take(fn, dev, "dres", dres, (rdt,), (T, d)),
         _take(fn, dev, "dgate", dgate, (ydt,), (head[6], d)),
         _take(fn, dev, "dw_post", dw_post, f32, (d,)),
         _take(fn, dev, "dw_pre", dw_pre, f32, (d,)), ws, nws)


# ----------------------------------------------------------------------------
# the layer for a few tokens (include/moe_int4_few.h)
# ----------------------------------------------------------------------------

def moe_layer_few_workspace_bytes(shape, T: int) -> int:
    if not 0 <= T <= _INT32_MAX:
        return 0
    return load().moe_layer_few_workspace_bytes(ctypes.byref(_shape(shape)), T)


def _expert_weights(fn, dev, who, w, n, d, f):
    """(kind, moe_expert_weights) of a tuple (gate_up, down[, gate_up_scales,
    down_scales]) for n experts."""
    bf16, f32, _, _, codes = _T or _types()
    gu, dn, gus, dns = w if len(w) == 4 else (*w, None, None)
    if gu.dtype == bf16[0]:
        kind, dt, sizes = MOE_WEIGHTS_BF16, bf16, None
        if gus is not None or dns is not None:
            raise ValueError(f"{fn}: bfloat16 {who} weights have no scales")
    elif gu.dtype == _INT8[0]:
        kind, dt, sizes = MOE_WEIGHTS_INT8, _INT8, ((n, 2 * f), (n, d))
    elif gu.dtype in codes:
        b = lambda v: -(-v // 128)  # noqa: E731
        kind, dt, sizes = MOE_WEIGHTS_E4M3, codes, ((n, b(2 * f), b(d)), (n, b(d), b(f)))
    else:
        raise TypeError(f"{fn}: {who} gate_up is {gu.dtype}, not bfloat16, int8 or e4m3 codes")
    s = ExpertWeights(_take(fn, dev, f"{who} gate_up", gu, dt, (n, 2 * f, d)),
                      _take(fn, dev, f"{who} down", dn, dt, (n, d, f)))
    if sizes is not None:
        if gus is None or dns is None:
            raise ValueError(f"{fn}: {who} codes have no scales")
        s.gate_up_scales = _take(fn, dev, f"{who} gate_up scales", gus, f32, sizes[0])
        s.down_scales = _take(fn, dev, f"{who} down scales", dns, f32, sizes[1])
    return kind, s


def moe_layer_few(shape, x, w_router, bias, experts, shared, topk_idx, topk_w, out, workspace,
                  stream=None):
    """The whole layer for x [T, d] bf16, T <= 32 and T * top_k <= 256.  experts:
    (gate_up [E, 2 f, d], down [E, d, f]) in bf16, or with their scales behind them
    in e4m3 codes or int8; shared: one expert's the same way, or None.  w_router
    [E, d] f32 (bias [E] or None): the routing goes to topk_idx and topk_w [T, k];
    None: they are given.  out [T, d] bf16/f32."""
    fn, dev = "moe_layer_few", x.get_device()
    bf16, f32, floats, i32, _ = _T or _types()
    sh = _shape(shape)
    T, d, f, E, k = _dim(fn, "x", x, 2)[0], sh.d, sh.f, sh.n_experts, sh.top_k
    kind, w = _expert_weights(fn, dev, "expert", experts, E, d, f)
    ws = None
    if shared is not None:
        other, ws = _expert_weights(fn, dev, "shared", shared, 1, d, f)
        if other != kind:
            raise TypeError(f"{fn}: the shared expert's weights are held another way")
        ws = ctypes.byref(ws)
    scratch, n_scratch = _workspace(fn, dev, workspace)
    _run(fn, dev, stream, ctypes.byref(sh), T, _take(fn, dev, "x", x, bf16, (T, d)),
         _take(fn, dev, "w_router", w_router, f32, (E, d)), _take(fn, dev, "bias", bias, f32, (E,)),
         kind, ctypes.byref(w), ws, _take(fn, dev, "topk_idx", topk_idx, i32, (T, k)),
         _take(fn, dev, "topk_w", topk_w, f32, (T, k)), _take(fn, dev, "out", out, floats, (T, d)),
         _code(out.dtype), scratch, n_scratch)


# ----------------------------------------------------------------------------
# one AdamW step over many tensors (include/moe_int4_adamw.h)
# ----------------------------------------------------------------------------

class AdamWTensors:
    """The tensors of moe_adamw, checked once and held: lists, entry by entry, of
    the parameters (bf16/f32), their gradients (bf16/f32, of the same shape) and
    the moments: float32 of the same shape, or with m_scales and v_scales 8-bit
    codes (m float8_e4m3fn or uint8, v uint8) and a float32 scale per 256 elements.
    masters: a float32 copy of each bf16 parameter, or None for all or for one.
    All on one GPU, without gaps, none overlapping one that the step writes.  A step
    goes by the addresses taken here; it refuses a list of which a tensor has been
    given other memory since (`p.data = ...`, moments moved away and back)."""

    def __init__(self, params, grads, m, v, masters=None, m_scales=None, v_scales=None):
        fn = "AdamWTensors"
        _, f32, floats, _, codes = _T or _types()
        n = len(params)
        lists = [params, masters, grads, m, v, m_scales, v_scales]
        names = ("params", "masters", "grads", "m", "v", "m_scales", "v_scales")
        for i, (name, q) in enumerate(zip(names, lists)):
            if q is None:
                if name in ("grads", "m", "v"):
                    raise ValueError(f"{fn}: {name} is missing")
                lists[i] = [None] * n
            elif len(q) != n:
                raise ValueError(f"{fn}: {len(q)} {name} for {n} params")
        self.tensors = lists = [list(q) for q in lists]  # held: the step goes by address
        self.device = params[0].get_device() if n else -1
        self.array = (AdamWTensor * n)()
        self.n = n
        # their memory, also of one that is given another later
        self.held = [t.untyped_storage() for q in lists for t in q if t is not None]
        spans, dev = [], self.device
        bf16, byte = _T[0][0], codes[1:]

        def take(name, i, t, dtypes, shape, count):
            """t's address, checked, of `count` elements; its span is kept."""
            dt = t.dtype
            if not (dt in dtypes and t.shape == shape and t.get_device() == dev and
                    t.is_contiguous()):
                _take(fn, dev, f"{name}[{i}]", t, dtypes, shape)  # raises
            at = t.data_ptr()
            if count:
                spans.append((at, at + count * dt.itemsize, name != "grads", i))
            return at

        for i, (p, w, g, a, b, sa, sb) in enumerate(zip(*lists)):
            for name, t in (("params", p), ("grads", g), ("m", a), ("v", b)):
                if t is None:
                    raise ValueError(f"{fn}: {name}[{i}] is missing")
            if (sa is None) != (sb is None):
                raise ValueError(f"{fn}: only one of m_scales[{i}] and v_scales[{i}] is given")
            shape, s = p.shape, self.array[i]
            s.n = count = p.numel()
            s.p, s.p_dt = take("params", i, p, floats, shape, count), _code(p.dtype)
            s.g, s.g_dt = take("grads", i, g, floats, shape, count), _code(g.dtype)
            if w is not None:
                if p.dtype != bf16:
                    raise TypeError(f"{fn}: masters[{i}] stands beside a parameter of {p.dtype}")
                s.master = take("masters", i, w, f32, shape, count)
            if sa is None:
                s.m, s.v = take("m", i, a, f32, shape, count), take("v", i, b, f32, shape, count)
            else:
                blocks = (-(-count // 256),)
                s.m, s.v = take("m", i, a, codes, shape, count), take("v", i, b, byte, shape, count)
                s.m_scales = take("m_scales", i, sa, f32, blocks, blocks[0])
                s.v_scales = take("v_scales", i, sb, f32, blocks, blocks[0])
        live = [t for q in lists for t in q if t is not None]
        # what a graph of autograd may have saved
        self.kept = [t for q in lists[:2] for t in q if t is not None]
        self.live = (live, [t.data_ptr() for t in live], list(range(len(live))))
        # two spans overlap only if one of them does with the one that reaches
        # furthest among those that begin before it: of the written and of all
        end = [(0, -1), (0, -1)]
        for lo, hi, written, i in sorted(spans):
            for reach, j in (end if written else end[:1]):
                if lo < reach:
                    raise ValueError(f"{fn}: tensors {j} and {i} overlap")
            if written:
                end[0] = max(end[0], (hi, i))
            end[1] = max(end[1], (hi, i))


def moe_adamw(tensors: AdamWTensors, step, lr: float, beta1: float = 0.9, beta2: float = 0.999,
              eps: float = 1e-8, weight_decay: float = 0.0, grad_scale=None, stream=None):
    """One step, in place.  step: device int64 [1], 1 for the first (the caller
    advances it; the parameters and masters count as modified in place, but not by
    a captured step's replays; the codes of 8-bit moments are drawn by it
    but for betas like 0.9 and 0.95); grad_scale: device f32 [1] that gradients are multiplied by."""
    fn = "moe_adamw"
    if not _same_memory(*tensors.live):  # 60 ns each: a step over many small ones waits for it
        raise ValueError(f"{fn}: a tensor lies elsewhere than when the list was made")
    dev = tensors.device if tensors.n else step.get_device()
    _run(fn, dev, stream, tensors.array, tensors.n,
         _take(fn, dev, "step", step, _INT64, (1,)), lr, beta1, beta2, eps, weight_decay,
         _take(fn, dev, "grad_scale", grad_scale, _T[1], (1,)))
    _written(tensors.kept)  # a backward pass over values of before the step is refused
