"""ctypes binding of libmoe.so: same names as the C ABI in include/moe.h.

Argument marshalling only. Tensors are torch tensors (device memory and streams come from
PyTorch); their data pointers and the current CUDA stream are passed straight to the
library. The binding raises MoeError on any non-zero return, and fails loudly at import
of the library if libmoe.so has not been built: there is no other implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_NOT_INIT = -1
MOE_ERR_BAD_ARG = -2
MOE_ERR_BAD_ALIGN = -3
MOE_ERR_CUDA = -4
MOE_ERR_DEVICE_TIMEOUT = -5
MOE_ERR_UNSUPPORTED_DEVICE = -6
MOE_PATH_AUTO = 0
MOE_PATH_GEMV = 1
MOE_PATH_GEMM = 2
MOE_PATH_GEMV_SPLIT = 3

# Every symbol include/moe.h declares.
EXPORTED = (
    "moe_init", "moe_layer_forward", "moe_rmsnorm_bf16", "moe_stack_forward", "moe_set_path",
    "moe_destroy", "moe_last_error", "moe_debug_get_routing", "moe_debug_get_hidden",
    "moe_debug_check", "moe_workspace_bytes", "moe_profile_begin", "moe_profile_end",
    "moe_layer_forward_static", "moe_profile_kernel_launches", "moe_layer_forward_static_check",
    "moe_debug_set_wait_ns", "moe_debug_inject", "moe_block_forward", "moe_route", "moe_experts_forward",
    "moe_gather_rows", "moe_combine_slots", "moe_qk_norm_rope", "moe_rope_frequencies", "moe_attention_decode",
    "moe_attention_decode_workspace_bytes", "moe_copy_pages", "moe_cache_check",
)
MOE_INJECT_NONE = 0
MOE_INJECT_SKIP_ROUTER_ARRIVAL = 1
MOE_DT_BF16 = 0
MOE_DT_F16 = 1
MOE_DT_E4M3 = 2
MOE_ROPE_PLAIN = 0
MOE_ROPE_LINEAR = 1
MOE_ROPE_NTK = 2
MOE_ROPE_YARN = 3
PROF_GROUPS = ("route", "gateup_gemv", "down_gemv", "gateup_gemm", "down_gemm", "combine", "rmsnorm",
               "fused_decode")


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmoe error {code}: {msg}")
        self.code = code


_lib = None
_p = ctypes.c_void_p
_i = ctypes.c_int
_ll = ctypes.c_longlong
_f = ctypes.c_float
_d = ctypes.c_double


# moe_kv_cache and moe_heads, packed as C lays them out
_KV_CACHE = struct.Struct("@PPiiiiiiqqqqff")
_HEADS = struct.Struct("@Pqq")


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m mixture_experts_gemv_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_init.argtypes = [_i, _i, _i, _i, _i, _i]
        L.moe_init.restype = _i
        L.moe_layer_forward.argtypes = [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p]
        L.moe_layer_forward.restype = _i
        L.moe_route.argtypes = [_p, _p, _p, _i, _i, _i, _i, _p, _p, _p]
        L.moe_route.restype = _i
        L.moe_experts_forward.argtypes = [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _p, _p]
        L.moe_experts_forward.restype = _i
        L.moe_gather_rows.argtypes = [_p, _p, _i, ctypes.c_size_t, _p, _p]
        L.moe_gather_rows.restype = _i
        L.moe_combine_slots.argtypes = [_p, _i, _i, _i, _p, _p]
        L.moe_combine_slots.restype = _i
        L.moe_block_forward.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p]
        L.moe_block_forward.restype = _i
        L.moe_rmsnorm_bf16.argtypes = [_p, _p, _i, _i, ctypes.c_float, _p]
        L.moe_rmsnorm_bf16.restype = _i
        L.moe_stack_forward.argtypes = [_p, _i, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i,
                                        ctypes.c_float, _p, _p, _p]
        L.moe_stack_forward.restype = _i
        L.moe_set_path.argtypes = [_i, _i]
        L.moe_set_path.restype = _i
        L.moe_destroy.argtypes = []
        L.moe_destroy.restype = None
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_debug_get_routing.argtypes = [_p, _p, _p, _p, _p, _p]
        L.moe_debug_get_routing.restype = _i
        L.moe_debug_get_hidden.argtypes = [_p, _p]
        L.moe_debug_get_hidden.restype = _i
        L.moe_debug_check.argtypes = [_p]
        L.moe_debug_check.restype = _i
        L.moe_profile_begin.argtypes = []
        L.moe_profile_begin.restype = _i
        L.moe_profile_end.argtypes = [_p, _p]
        L.moe_profile_end.restype = _i
        L.moe_layer_forward_static.argtypes = [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p]
        L.moe_layer_forward_static.restype = _i
        L.moe_layer_forward_static_check.argtypes = [_p]
        L.moe_layer_forward_static_check.restype = _i
        L.moe_debug_set_wait_ns.argtypes = [ctypes.c_ulonglong]
        L.moe_debug_set_wait_ns.restype = _i
        L.moe_debug_inject.argtypes = [_i]
        L.moe_debug_inject.restype = _i
        L.moe_profile_kernel_launches.argtypes = []
        L.moe_profile_kernel_launches.restype = ctypes.c_longlong
        L.moe_qk_norm_rope.argtypes = [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _i, _i, _f, _p, _p, _f, _p, _p, _p,
                                       _i, _p, _p]
        L.moe_qk_norm_rope.restype = _i
        L.moe_rope_frequencies.argtypes = [_i, _i, _d, _d, _d, _d, _d, _p, _p]
        L.moe_rope_frequencies.restype = _i
        L.moe_attention_decode.argtypes = [_p, _i, _p, _i, _p, _ll, _i, _p, _i, _i, _f, _i, _p, _p, _p,
                                           ctypes.c_size_t, _p]
        L.moe_attention_decode.restype = _i
        L.moe_attention_decode_workspace_bytes.argtypes = [_i, _i, _i]
        L.moe_attention_decode_workspace_bytes.restype = ctypes.c_size_t
        L.moe_copy_pages.argtypes = [_p, _p, _p, _i, _p, _ll, _i, _i, _p]
        L.moe_copy_pages.restype = _i
        L.moe_cache_check.argtypes = [_p]
        L.moe_cache_check.restype = _i
        L.moe_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        _lib = L
    return _lib


def _check(rc: int) -> int:
    if rc != MOE_OK:
        raise MoeError(rc, lib().moe_last_error().decode(errors="replace"))
    return rc


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_init(device: int, max_tokens: int, max_d: int, max_f: int, max_E: int, max_k: int) -> None:
    _check(lib().moe_init(device, max_tokens, max_d, max_f, max_E, max_k))


def moe_layer_forward(x, router_w, router_scale, gate_up_q4, down_q4, expert_scale,
                      T: int, d: int, f: int, E: int, k: int, out, stream=None) -> None:
    _check(lib().moe_layer_forward(_ptr(x), _ptr(router_w), _ptr(router_scale), _ptr(gate_up_q4),
                                   _ptr(down_q4), _ptr(expert_scale), T, d, f, E, k, _ptr(out),
                                   _stream(stream)))


def moe_block_forward(x, router_w, router_scale, gate_up_q4, down_q4, expert_scale, gate_up_dense_q4,
                      down_dense_q4, T: int, d: int, f: int, f_dense: int, E: int, k: int, out, stream=None) -> None:
    _check(lib().moe_block_forward(_ptr(x), _ptr(router_w), _ptr(router_scale), _ptr(gate_up_q4),
                                   _ptr(down_q4), _ptr(expert_scale), _ptr(gate_up_dense_q4),
                                   _ptr(down_dense_q4), T, d, f, f_dense, E, k, _ptr(out), _stream(stream)))


def moe_route(x, router_w, router_scale, T: int, d: int, E: int, k: int, ids, w, stream=None) -> None:
    _check(lib().moe_route(_ptr(x), _ptr(router_w), _ptr(router_scale), T, d, E, k, _ptr(ids), _ptr(w),
                           _stream(stream)))


def moe_experts_forward(x_rows, row_expert, row_weight, gate_up_q4, down_q4, expert_scale, R: int, d: int,
                        f: int, E: int, out_rows, stream=None) -> None:
    _check(lib().moe_experts_forward(_ptr(x_rows), _ptr(row_expert), _ptr(row_weight), _ptr(gate_up_q4),
                                     _ptr(down_q4), _ptr(expert_scale), R, d, f, E, _ptr(out_rows),
                                     _stream(stream)))


def moe_gather_rows(src, index, n: int, row_bytes: int, dst, stream=None) -> None:
    _check(lib().moe_gather_rows(_ptr(src), _ptr(index), n, row_bytes, _ptr(dst), _stream(stream)))


def moe_combine_slots(y_slots, T: int, d: int, k: int, out, stream=None) -> None:
    _check(lib().moe_combine_slots(_ptr(y_slots), T, d, k, _ptr(out), _stream(stream)))


def moe_rmsnorm_bf16(y, x_out, T: int, d: int, eps: float, stream=None) -> None:
    _check(lib().moe_rmsnorm_bf16(_ptr(y), _ptr(x_out), T, d, eps, _stream(stream)))


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])
    return arr


def moe_stack_forward(x_in, router_w, router_scale, gate_up_q4, down_q4, expert_scale,
                      T: int, d: int, f: int, E: int, k: int, eps: float, out, x_trace=None,
                      stream=None) -> None:
    """router_w ... expert_scale are sequences of per-layer tensors (length L)."""
    L = len(router_w)
    keep = [_ptr_array(v) for v in (router_w, router_scale, gate_up_q4, down_q4, expert_scale)]
    _check(lib().moe_stack_forward(_ptr(x_in), L, *[ctypes.cast(a, _p) for a in keep], T, d, f, E, k,
                                   eps, _ptr(out), _ptr(x_trace), _stream(stream)))


def moe_set_path(path: int, gemv_max_tokens: int = 16) -> None:
    _check(lib().moe_set_path(path, gemv_max_tokens))


def moe_destroy() -> None:
    lib().moe_destroy()


def moe_last_error() -> str:
    return lib().moe_last_error().decode(errors="replace")


def moe_debug_get_routing(ids=None, w=None, counts=None, offsets=None, perm=None, stream=None) -> None:
    _check(lib().moe_debug_get_routing(_ptr(ids), _ptr(w), _ptr(counts), _ptr(offsets), _ptr(perm),
                                       _stream(stream)))


def moe_debug_get_hidden(h, stream=None) -> None:
    _check(lib().moe_debug_get_hidden(_ptr(h), _stream(stream)))


def moe_debug_check(stream=None) -> None:
    _check(lib().moe_debug_check(_stream(stream)))


def moe_workspace_bytes(max_tokens: int, max_d: int, max_f: int, max_E: int, max_k: int) -> int:
    return int(lib().moe_workspace_bytes(max_tokens, max_d, max_f, max_E, max_k))


def moe_profile_begin() -> None:
    _check(lib().moe_profile_begin())


def moe_profile_end() -> dict:
    """{group name: (total ms, launches)} for the groups that ran."""
    ms = (ctypes.c_float * 8)()
    n = (ctypes.c_int * 8)()
    _check(lib().moe_profile_end(ms, n))
    return {PROF_GROUPS[i]: (float(ms[i]), int(n[i])) for i in range(8) if n[i] > 0}


def moe_profile_kernel_launches() -> int:
    """Kernels launched (or captured) since moe_profile_begin."""
    return int(lib().moe_profile_kernel_launches())


def moe_layer_forward_static(x, router_w, router_scale, gate_up_q4, down_q4, expert_scale,
                             T: int, d: int, f: int, E: int, k: int, out, stream=None) -> None:
    """Decode path with a fixed static device scratch: no workspace, no allocation."""
    _check(lib().moe_layer_forward_static(_ptr(x), _ptr(router_w), _ptr(router_scale),
                                          _ptr(gate_up_q4), _ptr(down_q4), _ptr(expert_scale),
                                          T, d, f, E, k, _ptr(out), _stream(stream)))


def moe_layer_forward_static_check(stream=None) -> None:
    """Raise MoeError(MOE_ERR_DEVICE_TIMEOUT) if a static-entry call timed out since the last check."""
    _check(lib().moe_layer_forward_static_check(_stream(stream)))


def moe_debug_set_wait_ns(ns: int) -> None:
    _check(lib().moe_debug_set_wait_ns(int(ns)))


def moe_debug_inject(fault: int) -> None:
    _check(lib().moe_debug_inject(int(fault)))


# ---------------------------------------------------------------- attention beside the layer
#
# These take torch tensors with their shapes and strides (the C entries take pointers and
# strides), run on the tensors' device whichever device is current, and check here what the
# library cannot see: types, devices and sizes. A call is a few microseconds of host time, so
# the descriptors are packed into bytes rather than built as ctypes structures.

_torch = None        # torch and the codes of its types, at the first call
_dtype_codes = None
_raw_stream = None   # device -> the handle of its current stream
_device = None       # () -> the current device


def _setup():
    global _torch, _dtype_codes, _raw_stream, _device
    import torch
    _dtype_codes = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16, torch.float8_e4m3fn: MOE_DT_E4M3}
    # the current stream's handle without a Stream object around it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _refuse(msg: str):
    raise MoeError(MOE_ERR_BAD_ARG, msg)


def _dtype_code(dtype) -> int:
    code = _dtype_codes.get(dtype)
    if code is None:
        _refuse(f"{dtype} is neither bf16, fp16 nor e4m3")
    return code


def _need(t, name, dtype, shape, index):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(f"{name}: need a contiguous {dtype} tensor of shape {tuple(shape)} on {_place(index)}, "
                f"got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _heads(t, name, shape, dtype, index):
    """moe_heads of a [T, heads, head_dim] tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(f"{name}: need {dtype} {tuple(shape)} on {_place(index)}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    token, head, one = t.stride()
    if one != 1:
        _refuse(f"{name}: the elements of a head must be contiguous")
    return _HEADS.pack(t.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0)


def _place(index):
    return "the CPU" if index < 0 else f"cuda:{index}"


def _call(fn, index, stream, *args):
    """fn(*args, stream) with the tensors' device current; stream None: its current stream."""
    if index < 0:
        _refuse("tensors must be on a CUDA device, not on the CPU")
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _device() == index:
        rc = fn(*args, stream)
    else:
        with _torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != MOE_OK:
        _check(rc)


class MoeKvCache:
    """A paged cache of keys and values over two tensors of the caller's (kept alive here):
    layout "NHD": [pages, page_size, n_kv, head_dim]; "HND": [pages, n_kv, page_size, head_dim]; with a
    leading dimension of layers where one tensor holds several. Any strides; bf16, fp16 or
    float8_e4m3fn (a stored value stands for value * scale)."""

    def __init__(self, k, v, layout: str = "NHD", k_scale: float = 1.0, v_scale: float = 1.0):
        if _torch is None:
            _setup()
        shape, st = k.shape, k.stride()
        if v.shape != shape or v.stride() != st or v.dtype != k.dtype or v.device != k.device or len(shape) not in (4, 5):
            _refuse("k and v need the same shape, [(layers,) pages, ...], strides, type and device")
        layers, layer_st = (1, 0) if len(shape) == 4 else (shape[0], st[0])
        pages, a, b, dim = shape[-4:]
        page_st, a_st, b_st, one = st[-4:]
        if layout == "NHD":
            tokens, heads, token_st, head_st = a, b, a_st, b_st
        elif layout == "HND":
            tokens, heads, token_st, head_st = b, a, b_st, a_st
        else:
            _refuse(f"unknown layout {layout!r}")
        if one != 1 and dim > 1:
            _refuse("the elements of a head must be contiguous")
        self.k, self.v, self.layout, self.index, self.dtype = k, v, layout, k.get_device(), k.dtype
        self.n_layers, self.num_pages, self.page_size, self.n_kv, self.head_dim = layers, pages, tokens, heads, dim
        self.k_scale, self.v_scale = k_scale, v_scale
        # the stride of a dimension of one is not used and may be anything
        self.packed = _KV_CACHE.pack(k.data_ptr(), v.data_ptr(), _dtype_code(k.dtype), layers, pages, tokens, heads, dim,
                                     layer_st if layers > 1 else 0, page_st if pages > 1 else 0,
                                     token_st if tokens > 1 else 0, head_st if heads > 1 else 0, k_scale, v_scale)


def moe_qk_norm_rope(q, k, v, positions, inv_freq, q_gain=None, k_gain=None, eps: float = 1e-6,
                     interleaved: bool = False, rope_scale: float = 1.0, q_out=None, k_out=None, cache=None,
                     layer: int = 0, slots=None, stream=None) -> None:
    """Norms of q [T, n_q, D] and k [T, n_kv, D] per head, rotation by positions (int32 [T]) and inv_freq
    (float64 [rotary_dim / 2], None: no rotation), into q_out and k_out and, with v, into `cache` at
    slots (int64 [T], negative: not stored). q or k may be None."""
    if _torch is None:
        _setup()
    some = k if q is None else q
    if some is None or some.dim() != 3 or (k is not None and k.dim() != 3):
        _refuse("q or k of shape [T, heads, head_dim] needed")
    T, _, D = some.shape
    dev, dt = some.get_device(), some.dtype
    n_q = n_kv = 0
    pq = pk = pv = pq_out = pk_out = None
    if q is not None:
        of_q = q.shape
        n_q = of_q[1]
        pq = _heads(q, "q", of_q, dt, dev)
        if q_out is not None:
            pq_out = _heads(q_out, "q_out", of_q, dt, dev)
    if k is not None:
        n_kv = k.shape[1]
        of_k = (T, n_kv, D)
        pk = _heads(k, "k", of_k, dt, dev)
        if k_out is not None:
            pk_out = _heads(k_out, "k_out", of_k, dt, dev)
        if cache is not None and v is not None:
            pv = _heads(v, "v", of_k, dt, dev)
    rot, p_pos, p_freq = 0, None, None
    if inv_freq is not None:
        half = inv_freq.numel()
        p_freq = _need(inv_freq, "inv_freq", _torch.float64, (half,), dev)
        if positions is None:
            _refuse("positions needed")
        p_pos = _need(positions, "positions", _torch.int32, (T,), dev)
        rot = 2 * half
    p_qg = None if q_gain is None else _need(q_gain, "q_gain", _torch.float32, (D,), dev)
    p_kg = None if k_gain is None else _need(k_gain, "k_gain", _torch.float32, (D,), dev)
    packed = p_slots = None
    if cache is not None:
        if cache.index != dev:
            _refuse(f"the cache is on {_place(cache.index)}, q and k on {_place(dev)}")
        if slots is None:
            _refuse("slots needed with a cache")
        p_slots = _need(slots, "slots", _torch.int64, (T,), dev)
        packed = cache.packed
    code = _dtype_code(dt)
    if T == 0:
        return
    _call(lib().moe_qk_norm_rope, dev, stream, pq, pk, pv, code, T, n_q, n_kv, D, p_pos, p_freq, rot,
          1 if interleaved else 0, rope_scale, p_qg, p_kg, eps, pq_out, pk_out, packed, layer, p_slots)


def moe_rope_frequencies(rotary_dim: int, base: float = 10000.0, kind: int = MOE_ROPE_PLAIN, factor: float = 1.0,
                         original_length: float = 4096.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                         device=None):
    """(inv_freq, rope_scale): float64 [rotary_dim / 2] on `device` and the factor on the rotated values."""
    import torch
    out = torch.empty(max(0, rotary_dim // 2), dtype=torch.float64)
    scale = _f()
    _check(lib().moe_rope_frequencies(kind, rotary_dim, base, factor, original_length, beta_fast, beta_slow,
                                      out.data_ptr(), ctypes.byref(scale)))
    return (out if device is None else out.to(device)), scale.value


@functools.lru_cache(maxsize=64)
def _workspace_bytes(n_q, n_kv, head_dim):
    return int(lib().moe_attention_decode_workspace_bytes(n_q, n_kv, head_dim))


def moe_attention_decode_workspace_bytes(n_q: int, n_kv: int, head_dim: int) -> int:
    return int(lib().moe_attention_decode_workspace_bytes(n_q, n_kv, head_dim))


def moe_attention_decode(q, cache: MoeKvCache, block_tables, seq_lens, out, scale: float, window: int = 0,
                         layer: int = 0, lse=None, workspace=None, stream=None) -> None:
    """Attention of one new token per sequence, q [B, n_q, D], over its seq_lens[b] cached keys (block_tables
    int32 [B, max_pages]) into out [B, n_q, D] and, where given, lse float32 [B, n_q]. workspace: a
    tensor of at least moe_attention_decode_workspace_bytes bytes; None allocates it for this call (from
    the stream's own memory pool, a captured graph's under capture)."""
    if q.dim() != 3:
        _refuse("q of shape [B, n_q, head_dim] needed")
    shape, dev, dt = q.shape, q.get_device(), q.dtype
    B, n_q, D = shape
    if D != cache.head_dim or cache.index != dev:
        _refuse(f"q of {D} on {_place(dev)} over a cache of {cache.head_dim} on {_place(cache.index)}")
    pq = _heads(q, "q", shape, dt, dev)
    pout = _heads(out, "out", shape, dt, dev)
    if block_tables.dim() != 2 or block_tables.dtype is not _torch.int32 or block_tables.get_device() != dev:
        _refuse(f"block_tables: need int32 [{B}, max_pages] on {_place(dev)}")
    rows, cols = block_tables.shape
    table_st, one = block_tables.stride()
    if rows != B or (one != 1 and cols > 1):
        _refuse(f"block_tables: need int32 [{B}, max_pages] with contiguous rows")
    p_lens = _need(seq_lens, "seq_lens", _torch.int32, (B,), dev)
    p_lse = None if lse is None else _need(lse, "lse", _torch.float32, (B, n_q), dev)
    code = _dtype_code(dt)
    if B == 0:
        return
    L = lib()
    if workspace is None:
        size = _workspace_bytes(n_q, cache.n_kv, D)
        if dev < 0:
            _refuse("tensors must be on a CUDA device, not on the CPU")
        if stream is None:
            workspace = _torch.empty(size, dtype=_torch.uint8, device=q.device)
        else:   # from the pool of the stream that will use it
            s = _torch.cuda.ExternalStream(stream, device=q.device) if isinstance(stream, int) else stream
            with _torch.cuda.stream(s):
                workspace = _torch.empty(size, dtype=_torch.uint8, device=q.device)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse(f"workspace: need a contiguous tensor on {_place(dev)}")
        size = workspace.numel() * workspace.element_size()
    _call(L.moe_attention_decode, dev, stream, pq, code, cache.packed, layer, block_tables.data_ptr(),
          table_st if B > 1 else cols, cols, p_lens, B, n_q, scale, window, pout, p_lse, workspace.data_ptr(), size)


def _host_pages(v, name):
    """A host list of pages as a contiguous int32 CPU tensor."""
    t = v if isinstance(v, _torch.Tensor) else _torch.as_tensor(v, dtype=_torch.int32)
    if t.device.type != "cpu" or t.dim() != 1 or t.dtype != _torch.int32:
        _refuse(f"{name}: a list or a one-dimensional int32 tensor on the host needed")
    return t.contiguous()


def moe_copy_pages(cache: MoeKvCache, src, dst, block_tables=None, stream=None) -> None:
    """Page dst[i] = page src[i] of K and V in every layer of the cache (src, dst: host lists or int32 CPU
    tensors). With block_tables (int32 [rows, cols] on the device) it is a move: entries equal to
    src[i] become dst[i]."""
    src, dst = _host_pages(src, "src"), _host_pages(dst, "dst")
    n = len(src)
    if n != len(dst):
        _refuse(f"{n} sources, {len(dst)} destinations")
    rows = cols = table_st = 0
    p_tables = None
    if block_tables is not None:
        if block_tables.dim() != 2 or block_tables.dtype is not _torch.int32 or block_tables.get_device() != cache.index:
            _refuse(f"block_tables: need int32 [rows, cols] on {_place(cache.index)}")
        rows, cols = block_tables.shape
        table_st, one = block_tables.stride()
        if one != 1 and cols > 1:
            _refuse("block_tables: rows must be contiguous")
        if rows <= 1:
            table_st = cols
        p_tables = block_tables.data_ptr()
    if n == 0:
        return
    _call(lib().moe_copy_pages, cache.index, stream, cache.packed, src.data_ptr(), dst.data_ptr(), n, p_tables,
          table_st, rows, cols)


def moe_cache_check(device=None, stream=None) -> None:
    """Synchronise the stream and raise MoeError if a call since the last check met a page, length or slot out of range."""
    if _torch is None:
        _setup()
    dev = _torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        _refuse(f"{dev} is not a CUDA device")
    _call(lib().moe_cache_check, _torch.cuda.current_device() if dev.index is None else dev.index, stream)
