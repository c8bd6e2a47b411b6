"""A16W4 mixture-of-experts layer for AMD MI355X (gfx950).

Thin ctypes binding over libmoe_a16w4.so (include/moe_a16w4.h). Every step
of the layer runs in the library's HIP kernels; this module only checks
tensor dtypes/devices, passes device pointers and the current HIP stream,
and turns a non-OK status into MoeError. PyTorch provides device memory and
streams. There is no CPU fallback: importing this package fails if the
library has not been built.

Functions mirror the C ABI names:
  moe_route_topk, moe_align_sort_capacity, moe_default_block_m,
  moe_align_sort, moe_route_align, moe_a16w4_workspace_size, moe_a16w4_forward,
  moe_a16w4_forward_stages, moe_a16w4_forward_ex, moe_a16w4_forward_monolithic,
  moe_a16w4_forward_noalloc,
  mxfp4_to_int4g32_requant, moe_last_error,
  moe_rms_norm, moe_lora_linear, moe_ffn_forward, moe_ffn_forward_mxfp8,
  moe_ffn_backward (the dense operators around the routed experts)
plus compositions: moe_ffn (the shared expert as a differentiable function),
moe_a16w4_block (norm -> router -> routed experts + shared expert),
moe_a16w4_layer (route -> sort -> forward, the
in-kernel routing path of apply_monolithic on the vLLM mxfp4 API page) and
requantize_mxfp4_experts (the chunked MXFP4 -> int4-g32 load-time
conversion, eight experts per call).
"""
import contextlib
import ctypes
import os
import warnings
from typing import NamedTuple, Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_a16w4.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP = 0, 1, 2, 3
MOE_W_MXFP4, MOE_W_INT4G32 = 0, 1
MOE_ACT_SWIGLU = 0
MOE_DT_BF16, MOE_DT_F32 = 0, 1
MOE_STAGE_GATE_UP, MOE_STAGE_DOWN, MOE_STAGE_COMBINE, MOE_STAGE_ALL = 1, 2, 4, 7

# Every symbol include/moe_a16w4.h declares.
EXPORTS = (
    "moe_last_error", "moe_route_topk", "moe_align_sort_capacity", "moe_default_block_m",
    "moe_align_sort", "moe_route_align", "moe_a16w4_workspace_size", "moe_a16w4_forward",
    "moe_a16w4_forward_stages", "moe_a16w4_forward_ex", "moe_a16w4_forward_monolithic",
    "moe_a16w4_forward_noalloc",
    "mxfp4_to_int4g32_requant",
    "moe_rms_norm", "moe_lora_linear_workspace_size", "moe_lora_linear", "moe_ffn_workspace_size",
    "moe_ffn_forward", "moe_ffn_mxfp8_workspace_size", "moe_ffn_forward_mxfp8",
    "moe_ffn_backward_workspace_size", "moe_ffn_backward",
)
# Scratch of the allocation-free forward (MOE_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 64 << 20


class _CLora(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("index", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("n", ctypes.c_int),
                ("rank", ctypes.c_int)]


class MoeError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"[status {status}] {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the HIP library first "
            "(python -c 'import __graft_entry__ as g; g.build()'). There is no CPU fallback.")
    L = ctypes.CDLL(LIB_PATH)
    p, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_last_error.argtypes = []
    L.moe_route_topk.restype = i
    L.moe_route_topk.argtypes = [p, i, i, i, i, p, p, p]
    L.moe_align_sort_capacity.restype = i64
    L.moe_align_sort_capacity.argtypes = [i, i, i, i]
    L.moe_default_block_m.restype = i
    L.moe_default_block_m.argtypes = [i, i, i]
    L.moe_align_sort.restype = i
    L.moe_align_sort.argtypes = [p, i, i, i, i, p, p, p, p, p]
    L.moe_route_align.restype = i
    L.moe_route_align.argtypes = [p, i, i, i, i, i, p, p, p, p, p, p, p]
    L.moe_a16w4_workspace_size.restype = i64
    L.moe_a16w4_workspace_size.argtypes = [i, i, i, i, i, i]
    L.moe_a16w4_forward.restype = i
    L.moe_a16w4_forward.argtypes = [p, p, p, p, p, i, i, p, p, p, p, p, i, i, i, i, i, i, p, p, sz, p]
    L.moe_a16w4_forward_stages.restype = i
    L.moe_a16w4_forward_stages.argtypes = [p, p, p, p, p, i, i, p, p, p, p, p, i, i, i, i, i, i, p, p, sz,
                                           ctypes.c_uint, p]
    L.moe_a16w4_forward_ex.restype = i
    L.moe_a16w4_forward_ex.argtypes = [p, p, p, p, p, p, p, i, i, ctypes.c_float, p, p, p, p, p, i, i, i, i,
                                       i, i, p, p, sz, ctypes.c_uint, p]
    L.moe_a16w4_forward_monolithic.restype = i
    L.moe_a16w4_forward_monolithic.argtypes = [p, p, p, p, p, p, p, p, i, i, ctypes.c_float, i, i, i, i, i,
                                               i, i, p, p, p, p, p, p, p, p, sz, ctypes.c_uint, p]
    L.moe_a16w4_forward_noalloc.restype = i
    L.moe_a16w4_forward_noalloc.argtypes = [p, p, p, p, p, i, i, p, p, p, p, p, i, i, i, i, i, i, p, p]
    L.mxfp4_to_int4g32_requant.restype = i
    L.mxfp4_to_int4g32_requant.argtypes = [p, p, i, i, i, i, i, p, p, p]
    f, lo = ctypes.c_float, ctypes.POINTER(_CLora)
    L.moe_rms_norm.restype = i
    L.moe_rms_norm.argtypes = [p, i64, p, i64, i, p, i, f, f, i, i, p, i64, p, i64, p, i64, p, i64, p]
    L.moe_lora_linear_workspace_size.restype = i64
    L.moe_lora_linear_workspace_size.argtypes = [i, i, i, i]
    L.moe_lora_linear.restype = i
    L.moe_lora_linear.argtypes = [p, i64, p, lo, i, i, i, p, i64, i, p, sz, p]
    L.moe_ffn_workspace_size.restype = i64
    L.moe_ffn_workspace_size.argtypes = [i, i, i, i, i]
    L.moe_ffn_forward.restype = i
    L.moe_ffn_forward.argtypes = [p, i64, p, p, i, p, i64, lo, lo, i, i, i, p, i64, p, p, sz, p]
    L.moe_ffn_mxfp8_workspace_size.restype = i64
    L.moe_ffn_mxfp8_workspace_size.argtypes = [i, i, i]
    L.moe_ffn_forward_mxfp8.restype = i
    L.moe_ffn_forward_mxfp8.argtypes = [p, p, p, p, p, p, i, p, i64, i, i, i, p, i64, p, sz, p]
    L.moe_ffn_backward_workspace_size.restype = i64
    L.moe_ffn_backward_workspace_size.argtypes = [i, i, i]
    L.moe_ffn_backward.restype = i
    L.moe_ffn_backward.argtypes = [p, i64, p, i64, p, p, p, i, i, i, i, p, i64, p, p, p, sz, p]
    return L


lib = _load()


def moe_last_error() -> str:
    return lib.moe_last_error().decode()


def _check(status):
    if status != MOE_OK:
        raise MoeError(status, moe_last_error())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Allocation context for the tensors a call creates: with an explicit
    stream they are allocated on it, so the caching allocator does not hand
    their memory to other work while the call's kernels still use it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _dev(t, name, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def moe_route_topk(logits, topk, renormalize=True, topk_ids=None, topk_weights=None, stream=None):
    """Softmax top-k routing of fp32 logits [T, E] -> (ids int32, weights fp32) [T, topk]."""
    _dev(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    with _on(stream):
        if topk_ids is None:
            topk_ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
        if topk_weights is None:
            topk_weights = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    _dev(topk_ids, "topk_ids", torch.int32)
    _dev(topk_weights, "topk_weights", torch.float32)
    _check(lib.moe_route_topk(_ptr(logits), T, E, int(topk), int(bool(renormalize)),
                              _ptr(topk_ids), _ptr(topk_weights), _stream(stream)))
    return topk_ids, topk_weights


def moe_align_sort_capacity(T, topk, E, block_m) -> int:
    return int(lib.moe_align_sort_capacity(int(T), int(topk), int(E), int(block_m)))


def moe_default_block_m(T, topk, E) -> int:
    return int(lib.moe_default_block_m(int(T), int(topk), int(E)))


def moe_align_sort(topk_ids, E, block_m, out=None, stream=None):
    """Group pairs by expert -> (sorted_ids, block_expert, expert_offsets, num_post_pad)."""
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, topk = topk_ids.shape
    cap = moe_align_sort_capacity(T, topk, E, block_m)
    if cap < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, f"invalid align/sort sizes T={T} topk={topk} E={E} block_m={block_m}")
    dev = topk_ids.device
    if out is None:
        with _on(stream):
            out = (torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
                   torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev),
                   torch.empty(E + 1, dtype=torch.int32, device=dev),
                   torch.empty(1, dtype=torch.int32, device=dev))
    sorted_ids, block_expert, offsets, npp = out
    if sorted_ids.numel() < cap or block_expert.numel() < cap // block_m or offsets.numel() < E + 1:
        raise ValueError("align/sort output buffers too small")
    _check(lib.moe_align_sort(_ptr(topk_ids), T, topk, int(E), int(block_m), _ptr(sorted_ids),
                              _ptr(block_expert), _ptr(offsets), _ptr(npp), _stream(stream)))
    return sorted_ids, block_expert, offsets, npp


def moe_route_align(logits, topk, E, block_m, renormalize=True, ids=None, weights=None, out=None,
                    stream=None):
    """Routing + align/sort in one call -> (ids, weights, sorted_ids, block_expert,
    expert_offsets, num_post_pad); identical to moe_route_topk then moe_align_sort."""
    _dev(logits, "logits", torch.float32, 2)
    T, El = logits.shape
    if El != E:
        raise ValueError(f"logits have {El} experts, expected {E}")
    dev = logits.device
    with _on(stream):
        if ids is None:
            ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
        if weights is None:
            weights = torch.empty((T, topk), dtype=torch.float32, device=dev)
    _dev(ids, "ids", torch.int32)
    _dev(weights, "weights", torch.float32)
    cap = moe_align_sort_capacity(T, topk, E, block_m)
    if cap < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, f"invalid sizes T={T} topk={topk} E={E} block_m={block_m}")
    if out is None:
        with _on(stream):
            out = (torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
                   torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev),
                   torch.empty(E + 1, dtype=torch.int32, device=dev),
                   torch.empty(1, dtype=torch.int32, device=dev))
    sorted_ids, block_expert, offsets, npp = out
    if sorted_ids.numel() < cap or block_expert.numel() < cap // block_m or offsets.numel() < E + 1:
        raise ValueError("align/sort output buffers too small")
    _check(lib.moe_route_align(_ptr(logits), T, int(E), int(topk), int(bool(renormalize)),
                               int(block_m), _ptr(ids), _ptr(weights), _ptr(sorted_ids),
                               _ptr(block_expert), _ptr(offsets), _ptr(npp), _stream(stream)))
    return ids, weights, sorted_ids, block_expert, offsets, npp


def moe_a16w4_workspace_size(T, H, I, E, topk, block_m) -> int:
    return int(lib.moe_a16w4_workspace_size(int(T), int(H), int(I), int(E), int(topk), int(block_m)))


def _weights(w13, w13_scale, w2, w2_scale, fmt):
    sdt = torch.uint8 if fmt == MOE_W_MXFP4 else (torch.int16, torch.uint16, torch.bfloat16)
    _dev(w13, "w13", torch.uint8, 3)
    _dev(w2, "w2", torch.uint8, 3)
    _dev(w13_scale, "w13_scale", sdt, 3)
    _dev(w2_scale, "w2_scale", sdt, 3)
    E, I2, Hh = w13.shape
    H, I = Hh * 2, I2 // 2
    if (w2.shape != (E, H, I // 2) or w13_scale.shape != (E, 2 * I, H // 32)
            or w2_scale.shape != (E, H, I // 32)):
        raise ValueError(
            f"weight shapes disagree: w13 {tuple(w13.shape)}, w13_scale {tuple(w13_scale.shape)}, "
            f"w2 {tuple(w2.shape)}, w2_scale {tuple(w2_scale.shape)}")
    return E, H, I


def _bias(b, name, shape):
    if b is None:
        return None
    _dev(b, name, (torch.bfloat16, torch.int16, torch.uint16), 2)
    if tuple(b.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(b.shape)}")
    return b


def moe_a16w4_forward(x, w13, w13_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids,
                      block_expert, num_post_pad, block_m, fmt=MOE_W_MXFP4, act=MOE_ACT_SWIGLU,
                      out=None, workspace=None, stream=None, stages=MOE_STAGE_ALL,
                      w13_bias=None, w2_bias=None, swiglu_limit=0.0):
    """Fused MoE forward with precomputed routing. x bf16 [T, H] -> out bf16 [T, H].
    `stages` selects a subset of the launches (moe_a16w4_forward_stages).
    Optional expert biases w13_bias bf16 [E, 2I] and w2_bias bf16 [E, H], and
    swiglu_limit > 0 clamping gate and up to [-limit, limit]
    (moe_a16w4_forward_ex)."""
    _dev(x, "x", torch.bfloat16, 2)
    E, H, I = _weights(w13, w13_scale, w2, w2_scale, fmt)
    T = x.shape[0]
    if x.shape[1] != H:
        raise ValueError(f"x has {x.shape[1]} columns, weights expect H={H}")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    _dev(topk_weights, "topk_weights", torch.float32, 2)
    topk = topk_ids.shape[1]
    need = moe_a16w4_workspace_size(T, H, I, E, topk, block_m)
    if need < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "invalid forward sizes")
    with _on(stream):
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    _dev(out, "out", torch.bfloat16)
    _bias(w13_bias, "w13_bias", (E, 2 * I))
    _bias(w2_bias, "w2_bias", (E, H))
    if w13_bias is not None or w2_bias is not None or swiglu_limit:
        _check(lib.moe_a16w4_forward_ex(
            _ptr(x), _ptr(w13), _ptr(w13_scale), _ptr(w13_bias), _ptr(w2), _ptr(w2_scale), _ptr(w2_bias),
            int(fmt), int(act), float(swiglu_limit), _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_ids),
            _ptr(block_expert), _ptr(num_post_pad), T, H, I, E, topk, int(block_m), _ptr(out),
            _ptr(workspace), workspace.numel(), int(stages), _stream(stream)))
        return out
    args = (_ptr(x), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), int(fmt), int(act),
            _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_ids), _ptr(block_expert),
            _ptr(num_post_pad), T, H, I, E, topk, int(block_m), _ptr(out), _ptr(workspace),
            workspace.numel())
    if stages == MOE_STAGE_ALL:
        _check(lib.moe_a16w4_forward(*args, _stream(stream)))
    else:
        _check(lib.moe_a16w4_forward_stages(*args, int(stages), _stream(stream)))
    return out


def moe_a16w4_forward_noalloc(x, w13, w13_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids,
                              block_expert, num_post_pad, block_m, out, fmt=MOE_W_MXFP4,
                              act=MOE_ACT_SWIGLU, stream=None):
    """moe_a16w4_forward into a caller-given `out`, with the library's own
    device scratch as the workspace: neither this function nor the library
    allocates device memory (for callers that cannot allocate). Calls that
    overlap in time on one GPU share that scratch and race."""
    _dev(x, "x", torch.bfloat16, 2)
    E, H, I = _weights(w13, w13_scale, w2, w2_scale, fmt)
    T = x.shape[0]
    if x.shape[1] != H:
        raise ValueError(f"x has {x.shape[1]} columns, weights expect H={H}")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    _dev(topk_weights, "topk_weights", torch.float32, 2)
    _dev(out, "out", torch.bfloat16, 2)
    topk = topk_ids.shape[1]
    _check(lib.moe_a16w4_forward_noalloc(
        _ptr(x), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), int(fmt), int(act),
        _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_ids), _ptr(block_expert), _ptr(num_post_pad),
        T, H, I, E, topk, int(block_m), _ptr(out), _stream(stream)))
    return out


class MonolithicBuffers:
    """Every device buffer of moe_a16w4_forward_monolithic for one shape:
    the routing and align/sort outputs, the workspace and the output."""

    def __init__(self, T, H, I, E, topk, block_m, device, stream=None):
        cap = moe_align_sort_capacity(T, topk, E, block_m)
        need = moe_a16w4_workspace_size(T, H, I, E, topk, block_m)
        if cap < 0 or need < 0:
            raise MoeError(MOE_ERR_INVALID_ARG, f"invalid sizes T={T} H={H} I={I} E={E} topk={topk} "
                           f"block_m={block_m}")
        self.block_m = block_m
        with _on(stream):
            self.ids = torch.empty((T, topk), dtype=torch.int32, device=device)
            self.weights = torch.empty((T, topk), dtype=torch.float32, device=device)
            self.sorted_ids = torch.empty(max(cap, 1), dtype=torch.int32, device=device)
            self.block_expert = torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=device)
            self.expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
            self.num_post_pad = torch.empty(1, dtype=torch.int32, device=device)
            self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
            self.out = torch.empty((T, H), dtype=torch.bfloat16, device=device)


def moe_a16w4_forward_monolithic(x, router_logits, w13, w13_scale, w2, w2_scale, topk, fmt=MOE_W_MXFP4,
                                 act=MOE_ACT_SWIGLU, renormalize=True, block_m=None, bufs=None,
                                 w13_bias=None, w2_bias=None, swiglu_limit=0.0, stages=MOE_STAGE_ALL,
                                 stream=None):
    """The layer from router logits in one call (apply_monolithic): routing,
    align/sort and the forward. `bufs` (MonolithicBuffers) holds every
    device buffer; one is allocated on `stream` when not given. Returns
    bufs (bufs.out is the layer output; bufs.ids / bufs.weights the routing)."""
    _dev(x, "x", torch.bfloat16, 2)
    _dev(router_logits, "router_logits", torch.float32, 2)
    E, H, I = _weights(w13, w13_scale, w2, w2_scale, fmt)
    T = x.shape[0]
    if x.shape[1] != H or tuple(router_logits.shape) != (T, E):
        raise ValueError(f"x {tuple(x.shape)} / router_logits {tuple(router_logits.shape)} do not match "
                         f"H={H}, E={E}")
    bm = moe_default_block_m(T, topk, E) if block_m is None else int(block_m)
    if bufs is None:
        bufs = MonolithicBuffers(T, H, I, E, topk, bm, x.device, stream)
    elif bufs.block_m != bm:
        raise ValueError(f"buffers were sized for block_m={bufs.block_m}, not {bm}")
    _bias(w13_bias, "w13_bias", (E, 2 * I))
    _bias(w2_bias, "w2_bias", (E, H))
    b = bufs
    _check(lib.moe_a16w4_forward_monolithic(
        _ptr(x), _ptr(router_logits), _ptr(w13), _ptr(w13_scale), _ptr(w13_bias), _ptr(w2), _ptr(w2_scale),
        _ptr(w2_bias), int(fmt), int(act), float(swiglu_limit), int(bool(renormalize)), T, H, I, E, int(topk),
        bm, _ptr(b.ids), _ptr(b.weights), _ptr(b.sorted_ids), _ptr(b.block_expert), _ptr(b.expert_offsets),
        _ptr(b.num_post_pad), _ptr(b.out), _ptr(b.workspace), b.workspace.numel(), int(stages),
        _stream(stream)))
    return bufs


def moe_a16w4_layer(x, router_logits, w13, w13_scale, w2, w2_scale, topk, fmt=MOE_W_MXFP4,
                    renormalize=True, block_m=None, stream=None, w13_bias=None, w2_bias=None,
                    swiglu_limit=0.0):
    """route -> align/sort -> forward on one stream (no host synchronisation),
    through moe_a16w4_forward_monolithic. With an explicit `stream` every
    tensor the call creates is allocated on that stream (the routing and
    sort arrays, the workspace and the output), so their memory stays
    reserved until the stream's work is done; the caller orders any use of
    the output on another stream as usual."""
    return moe_a16w4_forward_monolithic(x, router_logits, w13, w13_scale, w2, w2_scale, topk, fmt=fmt,
                                        renormalize=renormalize, block_m=block_m, w13_bias=w13_bias,
                                        w2_bias=w2_bias, swiglu_limit=swiglu_limit, stream=stream).out


def mxfp4_to_int4g32_requant(w, scale_e8m0, expert_lo, expert_hi, w_int4, scale_bf16, stream=None):
    """Requantize experts [lo, hi) of MXFP4 w [E, N, K/2] into preallocated outputs."""
    _dev(w, "w", torch.uint8, 3)
    _dev(scale_e8m0, "scale_e8m0", torch.uint8, 3)
    _dev(w_int4, "w_int4", torch.uint8, 3)
    _dev(scale_bf16, "scale_bf16", (torch.int16, torch.uint16, torch.bfloat16), 3)
    E, N, Kh = w.shape
    K = Kh * 2
    if (scale_e8m0.shape != (E, N, K // 32) or w_int4.shape != w.shape
            or scale_bf16.shape != (E, N, K // 32)):
        raise ValueError("requant tensor shapes disagree")
    _check(lib.mxfp4_to_int4g32_requant(_ptr(w), _ptr(scale_e8m0), E, N, K, int(expert_lo),
                                        int(expert_hi), _ptr(w_int4), _ptr(scale_bf16),
                                        _stream(stream)))
    return w_int4, scale_bf16


_warned_lossy = False


def requantize_mxfp4_experts(w, scale_e8m0, chunk=8, stream=None):
    """Convert a whole MXFP4 expert tensor to int4-g32, `chunk` experts per call,
    into preallocated outputs (the conversion loop of the MXFP4-to-int4 pull
    request). Returns (codes uint8 [E, N, K/2], scales bf16 [E, N, K/32])."""
    global _warned_lossy
    if not _warned_lossy:
        warnings.warn("Requantizing MXFP4 experts to groupwise int4 (int4_per_group_32): "
                      "this conversion is lossy.", stacklevel=2)
        _warned_lossy = True
    E, N, Kh = w.shape
    with _on(stream):
        codes = torch.empty_like(w)
        scales = torch.empty((E, N, Kh * 2 // 32), dtype=torch.bfloat16, device=w.device)
    for lo in range(0, E, chunk):
        mxfp4_to_int4g32_requant(w, scale_e8m0, lo, min(lo + chunk, E), codes, scales, stream=stream)
    return codes, scales


# ---------------------------------------------------------------------------
# Dense operators around the routed experts.
#
# moe_ffn is the one that autograd sees. The others compute and record nothing,
# as the routed layer does: what they return has no graph, also for inputs that
# require gradients.

class LoraAdapters(NamedTuple):
    """A stack of low-rank adapters beside one projection [N, K]: token t adds
    B[i] (scale[i] * (A[i] x[t])) for i = index[t] (outside [0, n): nothing).
    a bf16 [n, rank, K]; b bf16 [n, N, rank]; index int32 [T]; ranks int32 [n]
    (adapter i uses its first ranks[i]) and scale fp32 [n], each optional."""
    a: torch.Tensor
    b: torch.Tensor
    index: torch.Tensor
    ranks: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None


_CODES = (torch.uint8, torch.float8_e4m3fn)
_SCALES = (torch.uint8, torch.float8_e8m0fnu)


def _fail_tensor(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


# A decode step calls these functions back to back, so what they do on the
# host counts: one pass of cheap checks a tensor, and the messages only where
# one fails. `device` is the device of a tensor that is known to be on a GPU.
def _full(t, name, dtype, shape, device):
    """The address of a contiguous tensor of this type (or one of these),
    shape and device."""
    try:
        if t.shape == shape and t.device == device and t.is_contiguous() and (
                t.dtype in dtype if type(dtype) is tuple else t.dtype is dtype):
            return t.data_ptr()
    except AttributeError:
        pass
    _fail_tensor(t, name, dtype, shape, device)


def _rows(t, name, dtype, shape, device):
    """A matrix whose rows are contiguous -> (address, row stride)."""
    try:
        if t.shape == shape and t.device == device and (
                t.dtype in dtype if type(dtype) is tuple else t.dtype is dtype):
            if t.is_contiguous():
                return t.data_ptr(), shape[1]
            T, cols = shape
            if cols > 1 and t.stride(1) != 1:
                raise ValueError(f"{name} must have contiguous rows, got strides {t.stride()}")
            return t.data_ptr(), t.stride(0) if T > 1 else cols
    except AttributeError:
        pass
    _fail_tensor(t, name, dtype, shape, device)


def _matrix(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def _run(device, stream, fn, *args):
    """fn(*args, stream address) with `device` current, on `stream` or that
    device's current stream."""
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return _run(device, stream, fn, *args)
    if stream is None:
        at = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    else:
        at = stream.cuda_stream
    status = fn(*args, at)
    if status != MOE_OK:
        _check(status)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t, stride, cols, stream):
    """A contiguous tensor of t's shape and type."""
    if stream is None and stride == cols:
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _workspace(given, need, device, stream):
    """-> (address, bytes, the tensor that holds them)."""
    if need < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "invalid sizes")
    if given is None:
        if need == 0:
            return None, 0, None
        given = _empty(need, torch.uint8, device, stream)
    elif given.dtype != torch.uint8 or not given.is_contiguous() or given.device != device:
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return given.data_ptr(), given.numel(), given


def _lora(lora, name, T, K, N, device):
    """-> (ctypes struct or None, rank)."""
    if lora is None:
        return None, 0
    a, b, index, ranks, scale = lora if len(lora) == 5 else LoraAdapters(*lora)
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError(f"{name}.a must be a tensor [n, rank, {K}]")
    n, rank, _ = a.shape
    return _CLora(_full(a, name + ".a", torch.bfloat16, (n, rank, K), device),
                  _full(b, name + ".b", torch.bfloat16, (n, N, rank), device),
                  _full(index, name + ".index", torch.int32, (T,), device),
                  None if ranks is None else _full(ranks, name + ".ranks", torch.int32, (n,), device),
                  None if scale is None else _full(scale, name + ".scale", torch.float32, (n,), device),
                  n, rank), rank


def moe_rms_norm(x, weight, residual=None, eps=1e-6, weight_offset=0.0, mxfp8=False, y=None,
                 residual_out=None, q=None, q_scale=None, stream=None):
    """Residual addition and RMS norm of x bf16 [T, H]:
    s = x + residual, v = s / sqrt(mean(s^2) + eps) * (weight_offset + weight).
    residual bf16 or fp32 [T, H] (None: s = x, and no residual_out unless a
    buffer is given); weight bf16 or fp32 [H]. mxfp8: also the MXFP8 output,
    for moe_ffn_forward_mxfp8. -> (y bf16, residual_out of residual's type or
    None, q float8_e4m3fn or None, q_scale float8_e8m0fnu [T, H/32] or None),
    without a graph for gradients.
    Buffers may be given; y=x and residual_out=residual work in place."""
    T, H = _matrix(x, "x")
    device = x.device
    px, ldx = _rows(x, "x", torch.bfloat16, (T, H), device)
    pr, ldr, rdt = None, H, None
    if residual is not None:
        pr, ldr = _rows(residual, "residual", (torch.bfloat16, torch.float32), (T, H), device)
        rdt = residual.dtype
    pw = _full(weight, "weight", (torch.bfloat16, torch.float32), (H,), device)
    if y is None:
        y = _like(x, ldx, H, stream)
        py, ldy = y.data_ptr(), H
    else:
        py, ldy = _rows(y, "y", torch.bfloat16, (T, H), device)
    po, ldo = None, H
    if residual_out is None and residual is not None:
        residual_out = _like(residual, ldr, H, stream)
        po = residual_out.data_ptr()
    elif residual_out is not None:
        po, ldo = _rows(residual_out, "residual_out", rdt or (torch.bfloat16, torch.float32), (T, H), device)
        rdt = residual_out.dtype
    pq, ldq, ps, lds = None, H, None, max(H // 32, 1)
    if mxfp8 or q is not None or q_scale is not None:
        if H % 32:
            raise ValueError(f"H={H} must be a multiple of 32 for the MXFP8 output")
        if q is None:
            q = _empty((T, H), torch.float8_e4m3fn, device, stream)
        if q_scale is None:
            q_scale = _empty((T, H // 32), torch.float8_e8m0fnu, device, stream)
        pq, ldq = _rows(q, "q", _CODES, (T, H), device)
        ps, lds = _rows(q_scale, "q_scale", _SCALES, (T, H // 32), device)
    _run(device, stream, lib.moe_rms_norm,
         px, ldx, pr, ldr, MOE_DT_F32 if rdt is torch.float32 else MOE_DT_BF16, pw,
         MOE_DT_F32 if weight.dtype is torch.float32 else MOE_DT_BF16, eps, weight_offset, T, H, po, ldo,
         py, ldy, pq, ldq, ps, lds)
    return y, residual_out, q, q_scale


def moe_lora_linear_workspace_size(T, K, N, rank=0) -> int:
    return int(lib.moe_lora_linear_workspace_size(T, K, N, rank))


def moe_lora_linear(x, w, lora=None, out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """x bf16 [T, K] times w bf16 [N, K] transposed, plus each token's low-rank
    adapter (LoraAdapters, or a tuple of its fields) -> out [T, N] in bf16 or
    fp32 (without adapters and in fp32: a router's logits), without a graph for
    gradients."""
    T, K = _matrix(x, "x")
    N = _matrix(w, "w")[0]
    device = x.device
    px, ldx = _rows(x, "x", torch.bfloat16, (T, K), device)
    pw = _full(w, "w", torch.bfloat16, (N, K), device)
    cl, rank = _lora(lora, "lora", T, K, N, device)
    if out is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        out = _empty((T, N), out_dtype, device, stream)
    po, ldo = _rows(out, "out", (torch.bfloat16, torch.float32), (T, N), device)
    pws, nws, _ws = _workspace(workspace, lib.moe_lora_linear_workspace_size(T, K, N, rank), device, stream)
    _run(device, stream, lib.moe_lora_linear,
         px, ldx, pw, cl, T, K, N, po, ldo, MOE_DT_F32 if out.dtype is torch.float32 else MOE_DT_BF16,
         pws, nws)
    return out


def moe_ffn_workspace_size(T, H, I, rank13=0, rank2=0) -> int:
    return int(lib.moe_ffn_workspace_size(T, H, I, rank13, rank2))


def _ffn_sizes(x, w13, w2):
    T, H = _matrix(x, "x")
    I2 = _matrix(w13, "w13")[0]
    if I2 % 2:
        raise ValueError(f"w13 must have 2I rows (gate rows, then up rows), got {I2}")
    return T, H, I2 // 2


def moe_ffn_forward(x, w13, w2, addend=None, lora13=None, lora2=None, save_gate_up=False, gate_up=None,
                    act=MOE_ACT_SWIGLU, out=None, workspace=None, stream=None):
    """Gated feed-forward block (the shared expert): [gate; up] = w13 x,
    h = silu(gate) * up, out = w2 h (+ addend). x bf16 [T, H], w13 bf16
    [2I, H], w2 bf16 [H, I], addend bf16 [T, H]; lora13 / lora2: adapters of
    the two projections. save_gate_up (or a gate_up buffer): -> (out, gate_up
    bf16 [T, 2I], what moe_ffn_backward needs), else out. No graph is recorded
    for gradients: moe_ffn does that (without adapters)."""
    T, H, I = _ffn_sizes(x, w13, w2)
    device = x.device
    px, ldx = _rows(x, "x", torch.bfloat16, (T, H), device)
    p13 = _full(w13, "w13", torch.bfloat16, (2 * I, H), device)
    p2 = _full(w2, "w2", torch.bfloat16, (H, I), device)
    pa, lda = (None, H) if addend is None else _rows(addend, "addend", torch.bfloat16, (T, H), device)
    c13, r13 = _lora(lora13, "lora13", T, H, 2 * I, device)
    c2, r2 = _lora(lora2, "lora2", T, I, H, device)
    if out is None:
        out = _like(x, ldx, H, stream)
        po, ldo = out.data_ptr(), H
    else:
        po, ldo = _rows(out, "out", torch.bfloat16, (T, H), device)
    if gate_up is None and save_gate_up:
        gate_up = _empty((T, 2 * I), torch.bfloat16, device, stream)
    pg = None if gate_up is None else _full(gate_up, "gate_up", torch.bfloat16, (T, 2 * I), device)
    pws, nws, _ws = _workspace(workspace, lib.moe_ffn_workspace_size(T, H, I, r13, r2), device, stream)
    _run(device, stream, lib.moe_ffn_forward,
         px, ldx, p13, p2, act, pa, lda, c13, c2, T, H, I, po, ldo, pg,
         pws, nws)
    return out if gate_up is None else (out, gate_up)


def moe_ffn_mxfp8_workspace_size(T, H, I) -> int:
    return int(lib.moe_ffn_mxfp8_workspace_size(T, H, I))


def moe_ffn_forward_mxfp8(x, x_scale, w13, w13_scale, w2, w2_scale, addend=None, act=MOE_ACT_SWIGLU,
                          out=None, workspace=None, stream=None):
    """moe_ffn_forward with MXFP8 activations and weights: codes e4m3 x [T, H],
    w13 [2I, H], w2 [H, I] (float8_e4m3fn or uint8) and e8m0 scales [rows,
    columns / 32] (float8_e8m0fnu or uint8) -> out bf16 [T, H], without a graph
    for gradients."""
    T, H, I = _ffn_sizes(x, w13, w2)
    device = x.device
    if H % 32 or I % 32:
        raise ValueError(f"H={H} and I={I} must be multiples of 32")
    px = _full(x, "x", _CODES, (T, H), device)
    pxs = _full(x_scale, "x_scale", _SCALES, (T, H // 32), device)
    p13 = _full(w13, "w13", _CODES, (2 * I, H), device)
    p13s = _full(w13_scale, "w13_scale", _SCALES, (2 * I, H // 32), device)
    p2 = _full(w2, "w2", _CODES, (H, I), device)
    p2s = _full(w2_scale, "w2_scale", _SCALES, (H, I // 32), device)
    pa, lda = (None, H) if addend is None else _rows(addend, "addend", torch.bfloat16, (T, H), device)
    if out is None:
        out = _empty((T, H), torch.bfloat16, device, stream)
        po, ldo = out.data_ptr(), H
    else:
        po, ldo = _rows(out, "out", torch.bfloat16, (T, H), device)
    pws, nws, _ws = _workspace(workspace, lib.moe_ffn_mxfp8_workspace_size(T, H, I), device, stream)
    _run(device, stream, lib.moe_ffn_forward_mxfp8,
         px, pxs, p13, p13s, p2, p2s, act, pa, lda, T, H, I, po, ldo,
         pws, nws)
    return out


def moe_ffn_backward_workspace_size(T, H, I) -> int:
    return int(lib.moe_ffn_backward_workspace_size(T, H, I))


def moe_ffn_backward(dout, x, gate_up, w13, w2, need_dx=True, need_dw13=True, need_dw2=True, dx=None,
                     dw13=None, dw2=None, act=MOE_ACT_SWIGLU, workspace=None, stream=None):
    """Backward of moe_ffn_forward (without adapters) from its gate_up ->
    (dx bf16 [T, H], dw13 bf16 [2I, H], dw2 bf16 [H, I]); a gradient that is
    not needed is None. The gradient of addend is dout itself."""
    T, H, I = _ffn_sizes(x, w13, w2)
    device = x.device
    pd, ldd = _rows(dout, "dout", torch.bfloat16, (T, H), device)
    px, ldx = _rows(x, "x", torch.bfloat16, (T, H), device)
    pg = _full(gate_up, "gate_up", torch.bfloat16, (T, 2 * I), device)
    p13 = _full(w13, "w13", torch.bfloat16, (2 * I, H), device)
    p2 = _full(w2, "w2", torch.bfloat16, (H, I), device)
    if not (need_dx or need_dw13 or need_dw2):
        return None, None, None
    if need_dx and dx is None:
        dx = _empty((T, H), torch.bfloat16, device, stream)
    if need_dw13 and dw13 is None:
        dw13 = _empty((2 * I, H), torch.bfloat16, device, stream)
    if need_dw2 and dw2 is None:
        dw2 = _empty((H, I), torch.bfloat16, device, stream)
    pdx, lddx = (None, H) if not need_dx else _rows(dx, "dx", torch.bfloat16, (T, H), device)
    pd13 = None if not need_dw13 else _full(dw13, "dw13", torch.bfloat16, (2 * I, H), device)
    pd2 = None if not need_dw2 else _full(dw2, "dw2", torch.bfloat16, (H, I), device)
    pws, nws, _ws = _workspace(workspace, lib.moe_ffn_backward_workspace_size(T, H, I), device, stream)
    _run(device, stream, lib.moe_ffn_backward,
         pd, ldd, px, ldx, pg, p13, p2, act, T, H, I, pdx, lddx, pd13, pd2,
         pws, nws)
    return dx if need_dx else None, dw13 if need_dw13 else None, dw2 if need_dw2 else None


class _Ffn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2, addend):
        needs = any(ctx.needs_input_grad[:3])
        r = moe_ffn_forward(x, w13, w2, addend=addend, save_gate_up=needs)
        out, gate_up = r if needs else (r, None)
        ctx.save_for_backward(x, w13, w2, gate_up)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, w13, w2, gate_up = ctx.saved_tensors
        nx, n13, n2, na = ctx.needs_input_grad
        if not (nx or n13 or n2):
            return None, None, None, dout
        # A gradient may come expanded or transposed.
        dense = dout.contiguous()
        if dense.data_ptr() % 16:
            dense = dense.clone()
        dx, dw13, dw2 = moe_ffn_backward(dense, x, gate_up, w13, w2, nx, n13, n2)
        return dx, dw13, dw2, dout if na else None


def moe_ffn(x, w13, w2, addend=None):
    """The shared expert as a differentiable function of bf16 x [T, H], w13
    [2I, H], w2 [H, I] and addend [T, H]: moe_ffn_forward, with
    moe_ffn_backward for the gradients that are asked for. There is no second
    derivative, and there are no gradients of adapters."""
    return _Ffn.apply(x, w13, w2, addend)


def moe_a16w4_block(x, norm_weight, router_w, w13, w13_scale, w2, w2_scale, topk, residual=None, eps=1e-6,
                    weight_offset=0.0, shared=None, shared_mxfp8=None, lora13=None, lora2=None,
                    renormalize=True, fmt=MOE_W_MXFP4, block_m=None, stream=None, w13_bias=None, w2_bias=None,
                    swiglu_limit=0.0):
    """The feed-forward half of a decoder layer on one stream: residual
    addition and norm (moe_rms_norm), router logits (moe_lora_linear in fp32
    with router_w bf16 [E, H]), the routed experts (moe_a16w4_layer, with the
    expert biases and the clamp if given) and the shared expert added to their
    output: shared = (w13, w2) in bf16 (moe_ffn_forward, with its adapters), or
    shared_mxfp8 = (w13, w13_scale, w2, w2_scale) (moe_ffn_forward_mxfp8 on the
    norm's MXFP8 output).
    The projection computes logits in eights: where E is no multiple of 8,
    router_w is padded in every call, or may be given with its rows padded to
    the next multiple (what these hold does not matter).
    -> (out bf16 [T, H], the residual for the next layer), without a graph for
    gradients (of its parts only the bf16 shared expert has one: moe_ffn)."""
    if shared is not None and shared_mxfp8 is not None:
        raise ValueError("shared and shared_mxfp8 exclude each other")
    if shared is None and (lora13 is not None or lora2 is not None):
        raise ValueError("lora13 and lora2 belong to the bf16 shared expert")
    E, rows = w13.shape[0], _matrix(router_w, "router_w")[0]
    if rows not in (E, -(-E // 8) * 8):
        raise ValueError(f"router_w has {rows} rows for {E} experts")
    with torch.cuda.device(x.device), _on(stream):
        y, res, q, qs = moe_rms_norm(x, norm_weight, residual=residual, eps=eps, weight_offset=weight_offset,
                                     mxfp8=shared_mxfp8 is not None, stream=stream)
        if rows % 8:
            router_w = torch.nn.functional.pad(router_w, (0, 0, 0, -E % 8))
        logits = moe_lora_linear(y, router_w, out_dtype=torch.float32, stream=stream)
        if logits.shape[1] != E:
            logits = logits[:, :E].contiguous()
        out = moe_a16w4_layer(y, logits, w13, w13_scale, w2, w2_scale, topk, fmt=fmt, renormalize=renormalize,
                              block_m=block_m, stream=stream, w13_bias=w13_bias, w2_bias=w2_bias,
                              swiglu_limit=swiglu_limit)
        if shared is not None:
            out = moe_ffn_forward(y, *shared, addend=out, out=out, lora13=lora13, lora2=lora2, stream=stream)
        elif shared_mxfp8 is not None:
            out = moe_ffn_forward_mxfp8(q, qs, *shared_mxfp8, addend=out, out=out, stream=stream)
    return out, x if residual is None else res
