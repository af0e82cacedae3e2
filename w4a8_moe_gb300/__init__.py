"""W4A8 mixture-of-experts FFN, FP8 projections, and key/value caches of 8 and of 4
bits with their decode attention, page tables and query/key rotation for GB300
(sm_103a).

Thin Python binding over the C ABI in include/w4a8_moe.h: each function has
the C entry point's name, takes torch CUDA tensors, allocates outputs and
workspaces with torch when the caller passes none, and forwards pointers, sizes
and the current CUDA stream. Every arithmetic step runs in the library's CUDA
kernels (libw4a8_moe.so, built in-tree by w4a8_moe_gb300/build.py); there is
no other implementation, and a missing library raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from collections import namedtuple

import torch

__all__ = [
    "w4a8_quantize_experts", "w4a8_quantize_act", "moe_route", "moe_w4a8_forward",
    "fp8_block_linear", "w4a8_device_error", "w4a8_selftest_wait_timeout", "w4a8_set_profile_events", "moe_w4a8_workspace_size",
    "moe_route_workspace_size", "fp8_block_linear_workspace_size", "moe_route_gate",
    "moe_route_gate_workspace_size", "fp8_linear", "fp8_linear_workspace_size",
    "moe_w4a8_forward_dynamic", "moe_w4a8_dynamic_workspace_size", "moe_w4a8_workspace_layout",
    "moe_w4a8_plan",
    "w4a8_quantize_act_workspace_size", "kv8_write", "kv8_read", "kv8_prefix_attention",
    "kv8_prefix_attention_workspace_size", "kv8_prefix_attention_plan", "RouteResult", "library_path", "W4A8Error",
    "rope_table", "RopeTable", "qk_norm_rope", "kv8_norm_rope_write", "kv_pages_extend", "kv_pages_truncate", "PageStep",
    "kv_pages_workspace_size", "kv4_write", "kv4_read", "kv4_attention", "kv4_attention_workspace_size",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libw4a8_moe.so")
_lib = None

RouteResult = namedtuple("RouteResult", "topk_ids topk_w counts offsets sorted_ids inv_perm")
RopeTable = namedtuple("RopeTable", "turns magnitude")
PageStep = namedtuple("PageStep", "starts seqs positions seen slots lens")


class W4A8Error(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise W4A8Error(f"CUDA library {_LIB_PATH} is not built; run "
                        "`python -m w4a8_moe_gb300.build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(_LIB_PATH)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    f32, f64 = ctypes.c_float, ctypes.c_double
    sig = {
        "w4a8_status_string": (ctypes.c_char_p, [i32]),
        "w4a8_version": (i32, []),
        "w4a8_quantize_experts": (i32, [P, i32, i32, i32, P, P, P]),
        "w4a8_quantize_act": (i32, [P, i64, P, i32, P, P, sz, P]),
        "w4a8_quantize_act_workspace_size": (sz, [i64]),
        "moe_route": (i32, [P, i32, i32, i32, i32, P, P, P, P, P, P, P, sz, P]),
        "moe_route_workspace_size": (sz, [i32, i32, i32]),
        "moe_route_gate": (i32, [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, sz, P]),
        "moe_route_gate_workspace_size": (sz, [i32, i32, i32, i32]),
        "moe_w4a8_forward": (i32, [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, i32, P, P, P, P, P,
                                   P, P, P, sz, P]),
        "moe_w4a8_workspace_size": (sz, [i32, i32, i32, i32, i32]),
        "moe_w4a8_plan": (i32, [i32, i32, i32, i32, i32, i32, i32, P]),
        "moe_w4a8_workspace_layout": (i32, [i32, i32, i32, i32, i32, P]),
        "moe_w4a8_forward_dynamic": (i32, [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, i32, P, P, P, P, P,
                                           P, P, P, sz, P]),
        "moe_w4a8_dynamic_workspace_size": (sz, [i32, i32, i32, i32, i32]),
        "fp8_block_linear": (i32, [P, i32, i32, i32, P, P, P, P, P, P, sz, P]),
        "fp8_block_linear_workspace_size": (sz, [i32, i32, i32]),
        "fp8_linear": (i32, [P, P, i32, i32, i32, P, P, P, P, sz, P]),
        "fp8_linear_workspace_size": (sz, [i32, i32, i32]),
        "kv8_write": (i32, [P, P, i32, i64, i64, P, i32, i32, i32, i32, i32, f32, P, P, P, P, P]),
        "kv8_read": (i32, [P, P, P, P, P, i32, i32, i32, i32, i32, i32, P, i64, P, i64, P]),
        "kv8_prefix_attention": (i32, [P, i64, i32, i32, i32, i32, P, P, P, P, i32, i32, i32, P, i32, P, i64, i32, P,
                                       f32, f32, P, P, P, sz, P]),
        "kv8_prefix_attention_workspace_size": (sz, [i32] * 7),
        "kv8_prefix_attention_plan": (i32, [i32] * 8 + [f32, i32, P]),
        "rope_table": (i32, [i32, P, f64, i32, f64, f64, f64, f64, P, P]),
        "qk_norm_rope": (i32, [P, i64, i32, P, i64, i32, i32, i32, P, P, i32, f32, i32, P, P, f32, P, i64, P, i64, P]),
        "kv8_norm_rope_write": (i32, [P, i64, i32, P, i64, P, i64, i32, i32, i32, P, P, P, i32, f32, i32, P, P, f32,
                                      i32, i32, i32, f32, P, i64, P, P, P, P, P]),
        "kv_pages_extend": (i32, [P, P, i32, P, i64, i32, i32, P, P, i32, i32, P, P, P, P, P, P, P, sz, P]),
        "kv_pages_truncate": (i32, [P, P, i32, P, i64, i32, i32, P, P, i32, P, P, sz, P]),
        "kv_pages_workspace_size": (sz, []),
        "kv4_write": (i32, [P, P, i32, i64, i64, P, i32, i32, i32, i32, P, P, P, P, P]),
        "kv4_read": (i32, [P, P, P, P, P, i32, i32, i32, i32, i32, P, i64, P, i64, P]),
        "kv4_attention": (i32, [P, i64, i32, i32, i32, i32, P, P, P, P, i32, i32, P, i64, i32, i32, P, P, f32, f32, P,
                                P, P, sz, P]),
        "kv4_attention_workspace_size": (sz, [i32] * 6),
        "w4a8_device_error": (i32, [P, P, P]),
        "w4a8_selftest_wait_timeout": (i32, [P, P]),
        "w4a8_set_profile_events": (i32, [P, i32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise W4A8Error(_load().w4a8_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """What is allocated inside belongs to `stream` (the current one when None)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _u8(t):
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


def _ws(nbytes: int, device, ws=None):
    if ws is not None:
        return ws
    buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    buf[:256].zero_()  # device error word
    return buf


# --------------------------------------------------------------------------- sizes
def moe_w4a8_workspace_size(T, H, I, E, k) -> int:
    return int(_load().moe_w4a8_workspace_size(T, H, I, E, k))


_PLAN_KEYS = ("token_tile", "k_per_stage", "down_ksplit", "down_streamk", "down_slots", "one_launch",
              "launches", "partials")


def moe_w4a8_plan(T, H, I, E, k, dynamic=False, num_sms=None) -> dict:
    """The launch plan of the MoE forward for this shape (host only; see
    moe_w4a8_plan in include/w4a8_moe.h). num_sms defaults to the current
    device's SM count."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    plan = (ctypes.c_int32 * 8)()
    _check(_load().moe_w4a8_plan(T, H, I, E, k, 1 if dynamic else 0, num_sms, plan))
    return dict(zip(_PLAN_KEYS, list(plan)))


def moe_w4a8_workspace_layout(T, H, I, E, k) -> dict:
    """Byte offsets of the intermediate tensors a forward call leaves in its
    workspace (see moe_w4a8_workspace_layout in include/w4a8_moe.h)."""
    off = (ctypes.c_int64 * 2)()
    _check(_load().moe_w4a8_workspace_layout(T, H, I, E, k, off))
    return {"hq": int(off[0]), "xp": int(off[1])}


def moe_w4a8_dynamic_workspace_size(T, H, I, E, k) -> int:
    return int(_load().moe_w4a8_dynamic_workspace_size(T, H, I, E, k))


def moe_route_workspace_size(T, E, k) -> int:
    return int(_load().moe_route_workspace_size(T, E, k))


def moe_route_gate_workspace_size(T, H, E, k) -> int:
    return int(_load().moe_route_gate_workspace_size(T, H, E, k))


def fp8_linear_workspace_size(M, N, K) -> int:
    return int(_load().fp8_linear_workspace_size(M, N, K))


def fp8_block_linear_workspace_size(M, N, K) -> int:
    return int(_load().fp8_block_linear_workspace_size(M, N, K))


def w4a8_quantize_act_workspace_size(numel) -> int:
    return int(_load().w4a8_quantize_act_workspace_size(numel))


def kv8_prefix_attention_workspace_size(B, Hq, Hkv, D, prefix_len, max_pages, page_size) -> int:
    return int(_load().kv8_prefix_attention_workspace_size(B, Hq, Hkv, D, prefix_len, max_pages, page_size))


def kv8_prefix_attention_plan(B, Hq, Hkv, D, prefix_len, max_pages, page_size, scale_mode=0, logit_cap=0.0,
                              num_sms=None) -> dict:
    """How a kv8_prefix_attention call of this shape is cut up (host only; see kv8_prefix_attention_plan in
    include/w4a8_moe.h). num_sms defaults to the current device's SM count."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    plan = (ctypes.c_int32 * 6)()
    _check(_load().kv8_prefix_attention_plan(B, Hq, Hkv, D, prefix_len, max_pages, page_size, scale_mode, logit_cap,
                                             num_sms, plan))
    return dict(zip(("ranges", "tiles_per_range", "prefix_blocks", "launches", "own_blocks_per_sm", "join_warps"),
                    list(plan)))


def kv4_attention_workspace_size(T, Hq, Hkv, D, max_pages, page_size) -> int:
    return int(_load().kv4_attention_workspace_size(T, Hq, Hkv, D, max_pages, page_size))


def kv_pages_workspace_size() -> int:
    return int(_load().kv_pages_workspace_size())


# --------------------------------------------------------------------------- calls
def w4a8_quantize_experts(w_bf16: torch.Tensor, packed=None, scale=None, stream=None):
    """bf16 [E, N, K] -> (packed int32 [E, N, K/8], scale fp32 [E, N])."""
    assert w_bf16.dtype == torch.bfloat16 and w_bf16.is_contiguous() and w_bf16.dim() == 3
    E, N, K = w_bf16.shape
    dev = w_bf16.device
    packed = packed if packed is not None else torch.empty(E, N, K // 8, dtype=torch.int32, device=dev)
    scale = scale if scale is not None else torch.empty(E, N, dtype=torch.float32, device=dev)
    _check(_load().w4a8_quantize_experts(_ptr(w_bf16), E, N, K, _ptr(packed), _ptr(scale),
                                         _stream(stream)))
    return packed, scale


def w4a8_quantize_act(x_bf16: torch.Tensor, scale=None, compute_scale: bool = True, out=None,
                      ws=None, stream=None):
    """bf16 tensor -> (E4M3 codes uint8 of the same shape, fp32 scale [1])."""
    assert x_bf16.dtype == torch.bfloat16 and x_bf16.is_contiguous()
    dev = x_bf16.device
    n = x_bf16.numel()
    if scale is None:
        if not compute_scale:
            raise ValueError("a static scale tensor is required when compute_scale=False")
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    out = out if out is not None else torch.empty(x_bf16.shape, dtype=torch.uint8, device=dev)
    nbytes = w4a8_quantize_act_workspace_size(n)
    ws = _ws(nbytes, dev, ws) if compute_scale else ws
    _check(_load().w4a8_quantize_act(_ptr(x_bf16), n, _ptr(scale), int(bool(compute_scale)),
                                     _ptr(_u8(out)), _ptr(ws), 0 if ws is None else ws.numel(),
                                     _stream(stream)))
    return out, scale


def moe_route(logits: torch.Tensor, k: int, renormalize: bool = True, out: RouteResult = None,
              ws=None, stream=None) -> RouteResult:
    """fp32 router logits [T, E] -> RouteResult (top-k ids/weights, histogram, permutation)."""
    assert logits.dtype == torch.float32 and logits.is_contiguous() and logits.dim() == 2
    T, E = logits.shape
    dev = logits.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = RouteResult(torch.empty(T, k, **i32), torch.empty(T, k, dtype=torch.float32, device=dev),
                          torch.empty(E, **i32), torch.empty(E + 1, **i32),
                          torch.empty(T * k, **i32), torch.empty(T * k, **i32))
    ws = _ws(moe_route_workspace_size(T, E, k), dev, ws)
    _check(_load().moe_route(_ptr(logits), T, E, k, int(bool(renormalize)), *map(_ptr, out), _ptr(ws),
                             ws.numel(), _stream(stream)))
    return out


def moe_route_gate(hidden: torch.Tensor, gate: torch.Tensor, k: int, renormalize: bool = True,
                   out: RouteResult = None, logits=None, ws=None, stream=None):
    """bf16 hidden [T, H] and bf16 router gate [E, H] -> (RouteResult, fp32 logits [T, E] or None).
    Pass `logits` (an fp32 [T, E] tensor, or True to allocate one) to receive the logits."""
    assert hidden.dtype == torch.bfloat16 and hidden.is_contiguous() and hidden.dim() == 2
    assert gate.dtype == torch.bfloat16 and gate.is_contiguous() and gate.dim() == 2
    T, H = hidden.shape
    E = gate.shape[0]
    dev = hidden.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = RouteResult(torch.empty(T, k, **i32), torch.empty(T, k, dtype=torch.float32, device=dev),
                          torch.empty(E, **i32), torch.empty(E + 1, **i32),
                          torch.empty(T * k, **i32), torch.empty(T * k, **i32))
    if logits is True:
        logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    ws = _ws(moe_route_gate_workspace_size(T, H, E, k), dev, ws)
    _check(_load().moe_route_gate(_ptr(hidden), _ptr(gate), T, H, E, k, int(bool(renormalize)),
                                  None if logits is None else _ptr(logits), *map(_ptr, out), _ptr(ws),
                                  ws.numel(), _stream(stream)))
    return out, logits


def moe_w4a8_forward(x_e4m3, a1_scale, w_gu, s_gu, w_d, s_d, a2_scale, act: int,
                     route: RouteResult, out=None, ws=None, stream=None):
    """W4A8 MoE FFN: E4M3 x [T, H] -> bf16 [T, H] (act 0 = SiLU-gated, 1 = GELU-tanh-gated)."""
    x = _u8(x_e4m3)
    T, H = x.shape
    E, I2, _ = w_gu.shape
    I = I2 // 2
    k = route.topk_ids.shape[1]
    dev = x.device
    out = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    ws = _ws(moe_w4a8_workspace_size(T, H, I, E, k), dev, ws)
    _check(_load().moe_w4a8_forward(
        _ptr(x), _ptr(a1_scale), T, H, I, E, k, _ptr(w_gu), _ptr(s_gu), _ptr(w_d), _ptr(s_d),
        _ptr(a2_scale), int(act), _ptr(route.topk_ids), _ptr(route.topk_w), _ptr(route.counts),
        _ptr(route.offsets), _ptr(route.sorted_ids), _ptr(route.inv_perm), _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


def moe_w4a8_forward_dynamic(x_e4m3, a1_scale, w_gu, s_gu, w_d, s_d, act: int, route: RouteResult,
                             out=None, a2_out=None, ws=None, stream=None):
    """moe_w4a8_forward with the intermediate scale computed from this call's h:
    returns (bf16 out [T, H], fp32 a2 [1])."""
    x = _u8(x_e4m3)
    T, H = x.shape
    E, I2, _ = w_gu.shape
    I = I2 // 2
    k = route.topk_ids.shape[1]
    dev = x.device
    out = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    a2_out = a2_out if a2_out is not None else torch.empty(1, dtype=torch.float32, device=dev)
    ws = _ws(moe_w4a8_dynamic_workspace_size(T, H, I, E, k), dev, ws)
    _check(_load().moe_w4a8_forward_dynamic(
        _ptr(x), _ptr(a1_scale), T, H, I, E, k, _ptr(w_gu), _ptr(s_gu), _ptr(w_d), _ptr(s_d),
        _ptr(a2_out), int(act), _ptr(route.topk_ids), _ptr(route.topk_w), _ptr(route.counts),
        _ptr(route.offsets), _ptr(route.sorted_ids), _ptr(route.inv_perm), _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out, a2_out


def fp8_linear(x_e4m3, x_scale, w_e4m3, w_scale, out=None, ws=None, stream=None):
    """Per-tensor FP8: E4M3 x [M, K] (scale [1]) x E4M3 W [N, K] (scale [1]) -> bf16 y [M, N].
    A workspace passed in must have been zero-filled before its first use here."""
    x = _u8(x_e4m3)
    w = _u8(w_e4m3)
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    out = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = torch.zeros(max(fp8_linear_workspace_size(M, N, K), 256), dtype=torch.uint8, device=dev)
    _check(_load().fp8_linear(_ptr(x), _ptr(x_scale), M, N, K, _ptr(w), _ptr(w_scale), _ptr(out), _ptr(ws),
                              ws.numel(), _stream(stream)))
    return out


def fp8_block_linear(x_bf16, w_e4m3, w_scale_inv, out=None, xq_out=None, xs_out=None, ws=None,
                     stream=None):
    """bf16 x [M, K] x (E4M3 W [N, K], Wsi [N/128, K/128]) -> bf16 y [M, N]."""
    assert x_bf16.dtype == torch.bfloat16 and x_bf16.is_contiguous()
    M, K = x_bf16.shape
    w = _u8(w_e4m3)
    N = w.shape[0]
    dev = x_bf16.device
    out = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    ws = _ws(fp8_block_linear_workspace_size(M, N, K), dev, ws)
    _check(_load().fp8_block_linear(_ptr(x_bf16), M, N, K, _ptr(w), _ptr(w_scale_inv), _ptr(out),
                                    _ptr(None if xq_out is None else _u8(xq_out)), _ptr(xs_out),
                                    _ptr(ws), ws.numel(), _stream(stream)))
    return out


# The kv8_* calls are made once per layer and decode step, where a call takes a few microseconds on the GPU, so their
# checks are written to cost little: every tensor attribute is read once (some 0.1 us each), and what went wrong is told
# apart only after a check has failed.
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_CODES = (torch.uint8, torch.float8_e4m3fn)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_gpus = 0   # how many there are, once known: with one, tensors on a GPU are on the current one


def _count_gpus():
    global _gpus
    _gpus = torch.cuda.device_count()
    return _gpus


def _cache_refused(k_cache, v_cache, k_scale, v_scale):
    if k_cache.dtype not in _CODES or v_cache.dtype not in _CODES or k_cache.dim() != 4 \
            or k_cache.shape != v_cache.shape or not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        return ValueError("k_cache and v_cache must be contiguous uint8 or float8_e4m3fn [pages, kv heads, page size, D]")
    return ValueError("k_scale and v_scale must be contiguous float32, both [kv heads] or both [pages, kv heads, page size]")


def _devices_refused(*tensors):
    if any(not t.is_cuda for t in tensors):
        return ValueError("tensors must be on the GPU")
    if len({t.get_device() for t in tensors}) > 1:
        return ValueError("tensors must be on one GPU")
    return ValueError(f"tensors are on cuda:{tensors[0].get_device()}, but the current device, on which the library "
                      f"launches, is cuda:{_current_device()}")


def _handle(stream, device):
    """The handle of the caller's stream, which has to belong to the tensors' GPU."""
    if stream.device_index != device:
        raise ValueError(f"stream is of cuda:{stream.device_index}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _row_stride(t, rows, heads, d, what):
    """The row stride of a bf16 [rows, heads, D] tensor whose rows may lie apart."""
    if t.dtype is not _BF16 or t.shape != (rows, heads, d):
        raise ValueError(f"{what} must be bf16 of shape {[rows, heads, d]}")
    row, head, one = t.stride()
    if one != 1 or (head != d and heads != 1):
        raise ValueError(f"{what}: each token's heads must be contiguous")
    return row if rows > 1 else heads * d   # one row may report any row stride


def _vector_refused(what):
    return ValueError(f"{what} must be a contiguous int32 vector")


def kv8_write(k, v, slots, k_cache, v_cache, k_scale, v_scale, min_scale: float = 0.0, stream=None) -> None:
    """Quantize bf16 keys and values [T, kv heads, D] (rows may lie apart, as in a fused projection's output) into
    slots [T] (int32; out of range: skipped) of the cache. k_scale / v_scale of shape [kv heads] are read; of shape
    [pages, kv heads, page size] they are computed and written."""
    shape, scales = k_cache.shape, k_scale.shape
    if k_cache.dtype not in _CODES or v_cache.dtype not in _CODES or len(shape) != 4 or v_cache.shape != shape \
            or k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or v_scale.shape != scales \
            or (scales != shape[1:2] and scales != shape[:3]) or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous() or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        raise _cache_refused(k_cache, v_cache, k_scale, v_scale)
    n, h, page, d = shape
    if slots.dtype is not _I32 or slots.dim() != 1 or not slots.is_contiguous():
        raise _vector_refused("slots")
    T = slots.numel()
    k_stride, v_stride = _row_stride(k, T, h, d, "k"), _row_stride(v, T, h, d, "v")
    device = k_cache.get_device()
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == k.get_device() == v.get_device() == slots.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, k, v, slots)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv8_write(
        k.data_ptr(), v.data_ptr(), T, k_stride, v_stride, slots.data_ptr(), h, d, n, page, len(scales) == 3, float(min_scale),
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        to_stream)
    if status:
        _check(status)


def kv8_read(k_cache, v_cache, k_scale, v_scale, slots, k_out=None, v_out=None, stream=None):
    """The cache's slots [T] (int32; out of range: zeros) as bf16 keys and values, each [T, kv heads, D]."""
    shape, scales = k_cache.shape, k_scale.shape
    if k_cache.dtype not in _CODES or v_cache.dtype not in _CODES or len(shape) != 4 or v_cache.shape != shape \
            or k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or v_scale.shape != scales \
            or (scales != shape[1:2] and scales != shape[:3]) or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous() or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        raise _cache_refused(k_cache, v_cache, k_scale, v_scale)
    n, h, page, d = shape
    if slots.dtype is not _I32 or slots.dim() != 1 or not slots.is_contiguous():
        raise _vector_refused("slots")
    T = slots.numel()
    if k_out is None or v_out is None:
        with _on(stream):
            k_out = k_out if k_out is not None else torch.empty(T, h, d, dtype=_BF16, device=k_cache.device)
            v_out = v_out if v_out is not None else torch.empty(T, h, d, dtype=_BF16, device=k_cache.device)
    k_stride, v_stride = _row_stride(k_out, T, h, d, "k_out"), _row_stride(v_out, T, h, d, "v_out")
    device = k_cache.get_device()
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == slots.get_device() == k_out.get_device() == v_out.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv8_read(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), slots.data_ptr(), T, h, d, n,
        page, len(scales) == 3, k_out.data_ptr(), k_stride, v_out.data_ptr(), v_stride,
        to_stream)
    if status:
        _check(status)
    return k_out, v_out


def kv8_prefix_attention(q, k_cache, v_cache, k_scale, v_scale, prefix_pages, prefix_len: int, page_table, suffix_lens,
                         sm_scale=None, logit_cap: float = 0.0, out=None, lse=None, ws=None, stream=None):
    """Decode attention of bf16 q [B, query heads, D] over a shared prefix (prefix_pages, the first prefix_len tokens;
    None with 0) and each sequence's own tokens (page_table [B, max pages], suffix_lens [B]; both None: no own tokens);
    returns (bf16 out [B, query heads, D], fp32 lse [B, query heads] or None). Pass `lse` (a tensor, or True to allocate one) to receive it.
    sm_scale defaults to D ** -0.5; logit_cap 0 is no cap."""
    shape, scales = k_cache.shape, k_scale.shape
    if k_cache.dtype not in _CODES or v_cache.dtype not in _CODES or len(shape) != 4 or v_cache.shape != shape \
            or k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or v_scale.shape != scales \
            or (scales != shape[1:2] and scales != shape[:3]) or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous() or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        raise _cache_refused(k_cache, v_cache, k_scale, v_scale)
    n, h, page, d = shape
    q_shape = q.shape
    if len(q_shape) != 3:
        raise ValueError("q must be bf16 [B, query heads, D of the cache]")
    B, hq, _ = q_shape
    q_stride = _row_stride(q, B, hq, d, "q")
    device = k_cache.get_device()
    if page_table is None and suffix_lens is None:
        row = most = 0
        table = lens = None
        own_device = device
    else:
        if page_table is None or page_table.dtype is not _I32 or page_table.dim() != 2:
            raise ValueError("page_table must be int32 [B, max pages]; None only with suffix_lens None")
        rows, most = page_table.shape
        row, one = page_table.stride()
        if rows != B or (one != 1 and most > 1):
            raise ValueError("page_table must be int32 [B, max pages], each sequence's pages contiguous")
        if suffix_lens is None or suffix_lens.dtype is not _I32 or suffix_lens.shape != (B,) \
                or not suffix_lens.is_contiguous():
            raise _vector_refused("suffix_lens")
        table, lens, own_device = page_table.data_ptr(), suffix_lens.data_ptr(), page_table.get_device()
        if suffix_lens.get_device() != own_device:
            raise _devices_refused(k_cache, page_table, suffix_lens)
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == q.get_device() == own_device) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, q, *(() if table is None else (page_table,)))
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    pages, prefix_len = None, int(prefix_len)
    if prefix_len > 0:
        if prefix_pages is None or prefix_pages.dtype is not _I32 or prefix_pages.dim() != 1 or not prefix_pages.is_contiguous():
            raise _vector_refused("prefix_pages")
        if prefix_pages.numel() * page < prefix_len:
            raise ValueError("prefix_pages must cover prefix_len tokens")
        if prefix_pages.get_device() != device:
            raise _devices_refused(k_cache, prefix_pages)
        pages = prefix_pages.data_ptr()
    if lse is False:
        lse = None
    if out is None or lse is True or ws is None:
        with _on(stream):
            out = out if out is not None else torch.empty(B, hq, d, dtype=_BF16, device=q.device)
            lse = torch.empty(B, hq, dtype=_F32, device=q.device) if lse is True else lse
            ws = ws if ws is not None else _ws(
                kv8_prefix_attention_workspace_size(B, hq, h, d, prefix_len, most, page), q.device)
    if out.dtype is not _BF16 or out.shape != q_shape or not out.is_contiguous():
        raise ValueError("out must be contiguous bf16 [B, query heads, D]")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    if out.get_device() != device or ws.get_device() != device:
        raise _devices_refused(k_cache, out, ws)
    to = None
    if lse is not None:
        if lse.dtype is not _F32 or lse.shape != (B, hq) or not lse.is_contiguous():
            raise ValueError("lse must be contiguous float32 [B, query heads]")
        if lse.get_device() != device:
            raise _devices_refused(k_cache, lse)
        to = lse.data_ptr()
    status = (_lib or _load()).kv8_prefix_attention(
        q.data_ptr(), q_stride, B, hq, h, d, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), n, page, len(scales) == 3, pages, prefix_len, table, row if B > 1 else most,
        most, lens, d ** -0.5 if sm_scale is None else float(sm_scale), float(logit_cap), out.data_ptr(), to,
        ws.data_ptr(), ws.nbytes, to_stream)
    if status:
        _check(status)
    return out, lse


# ---- rotation of queries and keys
_ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "yarn": 3, "wave": 4}
_ROPE_HIGH = {"yarn": 32.0, "wave": 4.0}


def rope_table(rotary_dim: int, base: float = 10000.0, scaling=None, factor: float = 1.0, original_len: float = 0.0,
               low: float = 1.0, high=None, inv_freq=None, device="cuda") -> RopeTable:
    """The frequencies of a rotary embedding as qk_norm_rope and kv8_norm_rope_write take them: base^(-2i / rotary_dim),
    stretched for long contexts by `scaling` (None, "linear", "base", "yarn" or "wave"; see rope_table in
    include/w4a8_moe.h), or the model's own inv_freq (radians per position, rotary_dim / 2 numbers). high defaults to 32
    for "yarn" and 4 for "wave"."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(_ROPE_SCALINGS)}")
    own = None
    if inv_freq is not None:
        if scaling is not None:
            raise ValueError("inv_freq are the frequencies as they are: scaling must be None")
        own = [float(f) for f in inv_freq]
        if 2 * len(own) != rotary_dim:
            raise ValueError("inv_freq must hold rotary_dim / 2 numbers")
        own = (ctypes.c_double * len(own))(*own)
    n = max(int(rotary_dim) // 2, 1)
    turns, magnitude = (ctypes.c_uint64 * n)(), ctypes.c_float(0.0)
    _check(_load().rope_table(rotary_dim, own, base, _ROPE_SCALINGS[scaling], factor, original_len, low,
                              _ROPE_HIGH.get(scaling, 2.0 * low) if high is None else high, turns,
                              ctypes.byref(magnitude)))
    bits = torch.frombuffer(bytearray(turns), dtype=torch.int64)   # the same 64 bits; torch computes with signed ones
    return RopeTable(bits.to(device), magnitude.value)


def _rope_refused():
    return ValueError("rope must be a RopeTable: contiguous int64 turns, a number")


def _weight(w, d, device, what):
    """The address of a norm's weights (None: no norm)."""
    if w is None:
        return None
    if w.dtype is not _BF16 or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{what} must be contiguous bf16 [D]")
    if w.get_device() != device:
        raise _devices_refused(w)
    return w.data_ptr()


def qk_norm_rope(q, k, positions, rope: RopeTable, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Norms (where weights are given) and rotates bf16 queries [T, query heads, D] and keys [T, kv heads, D] (None: no
    keys) by positions [T] (int32); rows may lie apart, as in a fused projection's output, and q_out / k_out may be q / k
    themselves. Returns (q_out, k_out)."""
    q_shape = q.shape
    if len(q_shape) != 3 or positions.dtype is not _I32 or positions.shape != q_shape[:1] or not positions.is_contiguous():
        raise ValueError("q must be bf16 [T, query heads, D], positions a contiguous int32 vector [T]")
    T, hq, d = q_shape
    turns, magnitude = rope
    if turns.dtype is not _I64 or turns.dim() != 1 or not turns.is_contiguous():
        raise _rope_refused()
    hkv = 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must be bf16 [T, kv heads, D]")
        hkv = k.shape[1]
    if q_out is None or (k is not None and k_out is None):
        with _on(stream):
            q_out = q_out if q_out is not None else torch.empty(T, hq, d, dtype=_BF16, device=q.device)
            if k is not None and k_out is None:
                k_out = torch.empty(T, hkv, d, dtype=_BF16, device=q.device)
    q_stride, q_to = _row_stride(q, T, hq, d, "q"), _row_stride(q_out, T, hq, d, "q_out")
    device = q.get_device()
    same = device == positions.get_device() == turns.get_device() == q_out.get_device()
    k_at = k_to_at = None
    k_stride = k_to = 0
    if k is not None:
        k_stride, k_to = _row_stride(k, T, hkv, d, "k"), _row_stride(k_out, T, hkv, d, "k_out")
        same = same and device == k.get_device() == k_out.get_device()
        k_at, k_to_at = k.data_ptr(), k_out.data_ptr()
    if device < 0 or not same or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(q, positions, turns, q_out, *(() if k is None else (k, k_out)))
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).qk_norm_rope(
        q.data_ptr(), q_stride, hq, k_at, k_stride, hkv, T, d, positions.data_ptr(), turns.data_ptr(), 2 * turns.numel(),
        magnitude, 1 if interleaved else 0, _weight(q_weight, d, device, "q_weight"),
        _weight(k_weight, d, device, "k_weight"), float(eps), q_out.data_ptr(), q_to, k_to_at, k_to, to_stream)
    if status:
        _check(status)
    return q_out, (None if k is None else k_out)


def kv8_norm_rope_write(q, k, v, positions, slots, rope: RopeTable, k_cache, v_cache, k_scale, v_scale, q_weight=None,
                        k_weight=None, eps: float = 1e-6, interleaved: bool = False, min_scale: float = 0.0, q_out=None,
                        stream=None):
    """qk_norm_rope and kv8_write in one pass: the queries [T, query heads, D] are normed, rotated and returned (q_out may
    be q), the keys and values [T, kv heads, D] go into slots [T] of the cache, the keys normed and rotated before."""
    shape, scales = k_cache.shape, k_scale.shape
    if k_cache.dtype not in _CODES or v_cache.dtype not in _CODES or len(shape) != 4 or v_cache.shape != shape \
            or k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or v_scale.shape != scales \
            or (scales != shape[1:2] and scales != shape[:3]) or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous() or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        raise _cache_refused(k_cache, v_cache, k_scale, v_scale)
    n, h, page, d = shape
    q_shape = q.shape
    if len(q_shape) != 3:
        raise ValueError("q must be bf16 [T, query heads, D of the cache]")
    T, hq, _ = q_shape
    if positions.dtype is not _I32 or positions.shape != (T,) or not positions.is_contiguous():
        raise _vector_refused("positions [T]")
    if slots.dtype is not _I32 or slots.shape != (T,) or not slots.is_contiguous():
        raise _vector_refused("slots [T]")
    turns, magnitude = rope
    if turns.dtype is not _I64 or turns.dim() != 1 or not turns.is_contiguous():
        raise _rope_refused()
    if q_out is None:
        with _on(stream):
            q_out = torch.empty(T, hq, d, dtype=_BF16, device=q.device)
    q_stride, q_to = _row_stride(q, T, hq, d, "q"), _row_stride(q_out, T, hq, d, "q_out")
    k_stride, v_stride = _row_stride(k, T, h, d, "k"), _row_stride(v, T, h, d, "v")
    device = k_cache.get_device()
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == q.get_device() == k.get_device() == v.get_device() == q_out.get_device()
                          == positions.get_device() == slots.get_device() == turns.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, q, k, v, q_out, positions, slots, turns)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv8_norm_rope_write(
        q.data_ptr(), q_stride, hq, k.data_ptr(), k_stride, v.data_ptr(), v_stride, h, T, d, positions.data_ptr(),
        slots.data_ptr(), turns.data_ptr(), 2 * turns.numel(), magnitude, 1 if interleaved else 0,
        _weight(q_weight, d, device, "q_weight"), _weight(k_weight, d, device, "k_weight"), float(eps), n, page,
        len(scales) == 3, float(min_scale), q_out.data_ptr(), q_to, k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), to_stream)
    if status:
        _check(status)
    return q_out


# ---- page tables
def _table(page_table):
    """(rows, pages of a row, row stride) of an int32 [sequences, max pages] table whose rows may lie apart."""
    if page_table.dtype is not _I32 or page_table.dim() != 2:
        raise ValueError("page_table must be int32 [sequences, max pages]")
    have, most = page_table.shape
    row, one = page_table.stride()
    if one != 1 and most > 1:
        raise ValueError("page_table must be int32 [sequences, max pages], each sequence's pages contiguous")
    return have, most, (row if have > 1 else most)


def _vectors(n, **vectors):
    for what, t in vectors.items():
        if t.dtype is not _I32 or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous int32 vector [{n}]")


def _pool_refused(B, lens, other, what, have, free_pages, free_count, ws):
    if lens.dtype is not _I32 or lens.dim() != 1 or not lens.is_contiguous():
        return _vector_refused("lens")
    if free_pages.dtype is not _I32 or free_pages.dim() != 1 or not free_pages.is_contiguous():
        return _vector_refused("free_pages")
    if have != B:
        return ValueError("page_table must have a row for each sequence")
    if not ws.is_contiguous():
        return ValueError("ws must be contiguous")
    try:
        _vectors(B, **{what: other})
        _vectors(1, free_count=free_count)
    except ValueError as e:
        return e
    return None


def kv_pages_extend(lens, new_lens, page_table, free_pages, free_count, page_size: int, capacity: int, out: PageStep = None,
                    ws=None, stream=None) -> PageStep:
    """Gives each sequence's new tokens (new_lens [B], behind lens [B]) pages off the stack free_pages [num pages], of
    which free_count [1] are there, and enters them in page_table [B, max pages]; all int32, on the GPU. Returns
    PageStep(starts [B + 1], and for up to `capacity` tokens seqs, positions, seen and slots, lens [B]); padding tokens
    have the slot -1. A sequence that cannot have all of its pages gets none (see kv_pages_extend in
    include/w4a8_moe.h). out.lens may be lens."""
    B, capacity = lens.numel(), int(capacity)
    n = (B,)
    have, most, row = _table(page_table)
    if ws is None:
        with _on(stream):
            ws = _ws(256, lens.device)
    if lens.dtype is not _I32 or lens.shape != n or not lens.is_contiguous() or new_lens.dtype is not _I32 \
            or new_lens.shape != n or not new_lens.is_contiguous() or have != B or free_pages.dtype is not _I32 \
            or free_pages.dim() != 1 or not free_pages.is_contiguous() or free_count.dtype is not _I32 \
            or free_count.shape != (1,) or not ws.is_contiguous():
        raise _pool_refused(B, lens, new_lens, "new_lens", have, free_pages, free_count, ws)
    device = lens.get_device()
    if device < 0 or not (device == new_lens.get_device() == page_table.get_device() == free_pages.get_device()
                          == free_count.get_device() == ws.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(lens, new_lens, page_table, free_pages, free_count, ws)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    if out is None:
        if capacity < 0:
            raise ValueError("capacity must be positive")
        with _on(stream):
            buf = torch.empty(2 * B + 1 + 4 * capacity, dtype=_I32, device=lens.device)
        # (whole numbers: no views that a gradient would have to know of, which take longer to make and to free)
        out = PageStep(*buf.unsafe_split_with_sizes((B + 1, capacity, capacity, capacity, capacity, B)))
        at, step = buf.data_ptr(), 4 * capacity
        tokens = at + 4 * (B + 1)
        to = at, tokens, tokens + step, tokens + 2 * step, tokens + 3 * step, tokens + 4 * step
    else:
        starts, seqs, positions, seen, slots, lens_out = out
        _vectors(B + 1, starts=starts)
        _vectors(capacity, seqs=seqs, positions=positions, seen=seen, slots=slots)
        _vectors(B, lens_out=lens_out)
        if not all(t.get_device() == device for t in out):
            raise _devices_refused(lens, *out)
        to = [t.data_ptr() for t in out]
    status = (_lib or _load()).kv_pages_extend(
        lens.data_ptr(), new_lens.data_ptr(), B, page_table.data_ptr(), row, most, int(page_size), free_pages.data_ptr(),
        free_count.data_ptr(), free_pages.numel(), capacity, *to, ws.data_ptr(), ws.nbytes, to_stream)
    if status:
        _check(status)
    return out


def kv_pages_truncate(lens, keep_lens, page_table, free_pages, free_count, page_size: int, out=None, ws=None, stream=None):
    """Gives the pages behind each sequence's first keep_lens [B] of lens [B] tokens back to the stack (0: the sequence is
    finished). Returns the lengths now, [B] (out, which may be lens or keep_lens)."""
    B = lens.numel()
    n = (B,)
    have, most, row = _table(page_table)
    if out is None or ws is None:
        with _on(stream):
            out = out if out is not None else torch.empty(B, dtype=_I32, device=lens.device)
            ws = ws if ws is not None else _ws(256, lens.device)
    if lens.dtype is not _I32 or lens.shape != n or not lens.is_contiguous() or keep_lens.dtype is not _I32 \
            or keep_lens.shape != n or not keep_lens.is_contiguous() or have != B or free_pages.dtype is not _I32 \
            or free_pages.dim() != 1 or not free_pages.is_contiguous() or free_count.dtype is not _I32 \
            or free_count.shape != (1,) or not ws.is_contiguous():
        raise _pool_refused(B, lens, keep_lens, "keep_lens", have, free_pages, free_count, ws)
    if out.dtype is not _I32 or out.shape != n or not out.is_contiguous():
        raise _vector_refused("out")
    device = lens.get_device()
    if device < 0 or not (device == keep_lens.get_device() == page_table.get_device() == free_pages.get_device()
                          == free_count.get_device() == ws.get_device() == out.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(lens, keep_lens, page_table, free_pages, free_count, ws, out)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv_pages_truncate(
        lens.data_ptr(), keep_lens.data_ptr(), B, page_table.data_ptr(), row, most, int(page_size), free_pages.data_ptr(),
        free_count.data_ptr(), free_pages.numel(), out.data_ptr(), ws.data_ptr(), ws.nbytes, to_stream)
    if status:
        _check(status)
    return out


# ---- the cache of 4 bits
_U8 = torch.uint8


def _cache4(k_cache, v_cache, k_scale, v_scale):
    """The shape of a 4-bit cache, [pages, kv heads, page size, D]."""
    shape = k_cache.shape
    if k_cache.dtype is not _U8 or v_cache.dtype is not _U8 or len(shape) != 4 or v_cache.shape != shape \
            or not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous uint8 [pages, kv heads, page size, D / 2]")
    n, h, page, half = shape
    scales = (n, h, page, 2)
    if k_scale.dtype is not _BF16 or v_scale.dtype is not _BF16 or k_scale.shape != scales or v_scale.shape != scales \
            or not (k_scale.is_contiguous() and v_scale.is_contiguous()):
        raise ValueError("k_scale and v_scale must be contiguous bf16 [pages, kv heads, page size, 2]")
    return n, h, page, 2 * half


def kv4_write(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """Quantize bf16 keys and values [T, kv heads, D] (rows may lie apart) to 4 bits into slots [T] (int32; out of range:
    skipped) of the cache: codes uint8 [pages, kv heads, page size, D / 2], and with each row its step and least value,
    bf16 [pages, kv heads, page size, 2]."""
    n, h, page, d = _cache4(k_cache, v_cache, k_scale, v_scale)
    if slots.dtype is not _I32 or slots.dim() != 1 or not slots.is_contiguous():
        raise _vector_refused("slots")
    T = slots.shape[0]
    k_stride, v_stride = _row_stride(k, T, h, d, "k"), _row_stride(v, T, h, d, "v")
    device = k_cache.get_device()
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == k.get_device() == v.get_device() == slots.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, k, v, slots)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv4_write(
        k.data_ptr(), v.data_ptr(), T, k_stride, v_stride, slots.data_ptr(), h, d, n, page, k_cache.data_ptr(),
        v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), to_stream)
    if status:
        _check(status)


def kv4_read(k_cache, v_cache, k_scale, v_scale, slots, k_out=None, v_out=None, stream=None):
    """The 4-bit cache's slots [T] (int32; out of range: zeros) as bf16 keys and values, each [T, kv heads, D]."""
    n, h, page, d = _cache4(k_cache, v_cache, k_scale, v_scale)
    if slots.dtype is not _I32 or slots.dim() != 1 or not slots.is_contiguous():
        raise _vector_refused("slots")
    T = slots.shape[0]
    if k_out is None or v_out is None:
        with _on(stream):
            k_out = k_out if k_out is not None else torch.empty(T, h, d, dtype=_BF16, device=k_cache.device)
            v_out = v_out if v_out is not None else torch.empty(T, h, d, dtype=_BF16, device=k_cache.device)
    k_stride, v_stride = _row_stride(k_out, T, h, d, "k_out"), _row_stride(v_out, T, h, d, "v_out")
    device = k_cache.get_device()
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == slots.get_device() == k_out.get_device() == v_out.get_device()) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out)
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv4_read(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), slots.data_ptr(), T, h, d, n,
        page, k_out.data_ptr(), k_stride, v_out.data_ptr(), v_stride, to_stream)
    if status:
        _check(status)
    return k_out, v_out


def kv4_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, seqs=None, sm_scale=None,
                  logit_cap: float = 0.0, out=None, lse=None, ws=None, stream=None):
    """Decode attention of bf16 q [T, query heads, D] over the 4-bit cache: token t sees the first lens[t] keys of sequence
    seqs[t] (None: sequence t), whose pages are page_table [sequences, max pages]; int32. Returns (bf16 out
    [T, query heads, D], fp32 lse [T, query heads] or None). Pass `lse` (a tensor, or True to allocate one) to receive it.
    sm_scale defaults to D ** -0.5; logit_cap 0 is no cap."""
    n, h, page, d = _cache4(k_cache, v_cache, k_scale, v_scale)
    q_shape = q.shape
    if len(q_shape) != 3:
        raise ValueError("q must be bf16 [T, query heads, D of the cache]")
    T, hq, _ = q_shape
    q_stride = _row_stride(q, T, hq, d, "q")
    have, most, row = _table(page_table)
    if lens.dtype is not _I32 or lens.shape != (T,) or not lens.is_contiguous():
        raise _vector_refused("lens [T]")
    if seqs is None:
        if have != T:
            raise ValueError("page_table must have a row for each token where seqs is None")
    elif seqs.dtype is not _I32 or seqs.shape != (T,) or not seqs.is_contiguous():
        raise _vector_refused("seqs [T]")
    if lse is False:
        lse = None
    if out is None or lse is True or ws is None:
        with _on(stream):
            out = out if out is not None else torch.empty(T, hq, d, dtype=_BF16, device=q.device)
            lse = torch.empty(T, hq, dtype=_F32, device=q.device) if lse is True else lse
            ws = ws if ws is not None else _ws(kv4_attention_workspace_size(T, hq, h, d, most, page), q.device)
    if out.dtype is not _BF16 or out.shape != q_shape or not out.is_contiguous():
        raise ValueError("out must be contiguous bf16 [T, query heads, D]")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != (T, hq) or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [T, query heads]")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    device = k_cache.get_device()
    if device < 0 or not (device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                          == q.get_device() == page_table.get_device() == lens.get_device() == out.get_device()
                          == ws.get_device()) \
            or (seqs is not None and seqs.get_device() != device) or (lse is not None and lse.get_device() != device) \
            or ((_gpus or _count_gpus()) != 1 and device != _current_device()):
        raise _devices_refused(k_cache, v_cache, k_scale, v_scale, q, page_table, lens, out, ws,
                               *(t for t in (seqs, lse) if t is not None))
    to_stream = _raw_stream(device) if stream is None else _handle(stream, device)
    status = (_lib or _load()).kv4_attention(
        q.data_ptr(), q_stride, T, hq, h, d, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), n, page, page_table.data_ptr(), row, have, most, None if seqs is None else seqs.data_ptr(),
        lens.data_ptr(), d ** -0.5 if sm_scale is None else float(sm_scale), float(logit_cap), out.data_ptr(),
        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes, to_stream)
    if status:
        _check(status)
    return out, lse


def w4a8_set_profile_events(events) -> None:
    """Measurement hook: torch.cuda.Event objects (up to 4, enable_timing=True)
    that moe_w4a8_forward records before/after its GEMMs on this host thread;
    None or [] switches recording off."""
    events = list(events or [])
    for e in events:
        if e.cuda_event == 0:  # torch creates the CUDA event on first record
            e.record()
    arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(_load().w4a8_set_profile_events(arr, len(events)))


def w4a8_selftest_wait_timeout(ws, stream=None):
    """Record a wait timeout in ws from a kernel whose barrier never completes (test hook)."""
    _check(_load().w4a8_selftest_wait_timeout(_ptr(ws), _stream(stream)))


def w4a8_device_error(ws, stream=None) -> int:
    """Read and clear a workspace's device error word (synchronizes the stream)."""
    code = ctypes.c_int(0)
    _check(_load().w4a8_device_error(_ptr(ws), ctypes.byref(code), _stream(stream)))
    return code.value
