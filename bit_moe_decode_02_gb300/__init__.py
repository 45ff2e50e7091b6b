"""Python binding of libmoe (the C ABI in include/moe.h), argument marshalling only.

Every step of the routed-expert block runs in the library's CUDA kernels; this
module turns torch tensors into pointers and streams and raises on a non-zero
status.  There is no CPU fallback: if libmoe.so is missing the import of the
library fails loudly (build it with ``python -m bit_moe_decode_02_gb300.build_ext``).

The function names are the C names: moe_create, moe_load_experts, moe_load_experts_ex,
moe_forward, moe_forward_host, moe_forward_stack, moe_forward_stack_steps, moe_forward_steps,
moe_load_router, moe_debug_router_logits, moe_set_batched_numerics, moe_set_swiglu, moe_get_status,
moe_debug_dequant, moe_debug_route, moe_debug_stack_trace, moe_debug_forward_f32,
moe_debug_set_wait, moe_last_bytes, moe_expert_bytes, moe_last_launches, moe_last_error,
moe_forward_noalloc, moe_debug_stream_weights, moe_destroy; and the operators around the expert
block: moe_ops_create, moe_ops_get_status, moe_ops_destroy, moe_kv_write, moe_kv_read,
moe_attention, moe_kv_plan, moe_rope_turns, moe_rope, moe_linear, moe_lora, moe_sample.  Those take
torch tensors and read sizes and strides from them; moe_kv_cache_of, moe_kv_batch_of, moe_kv_pool_of,
moe_rope_of, moe_linear_of and moe_lora_of make the descriptors that a program builds once and keeps
(with the tensors, which they keep alive).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_OOM = -3
MOE_ERR_CUDA = -4
MOE_ERR_NOT_LOADED = -5
MOE_ERR_DEVICE_TIMEOUT = -6
MOE_ERR_DEVICE_FAULT = -7
MOE_FMT_MXFP4 = 1
MOE_FMT_INT4 = 2
MOE_LOAD_GATE_UP_INTERLEAVED = 1
MOE_LOAD_TRANSPOSED = 2
MOE_BATCHED_MXFP4 = 0
MOE_BATCHED_BF16 = 1
MOE_KV_E4M3 = 1
MOE_KV_INT8 = 2
MOE_KV_MXFP4 = 4
MOE_DT_F32 = 0
MOE_DT_BF16 = 1
MOE_ROPE_HALF = 0
MOE_ROPE_INTERLEAVED = 1
MOE_ROPE_PLAIN = 0
MOE_ROPE_LINEAR = 1
MOE_ROPE_PARTS = 2
MOE_ROPE_WAVELENGTH = 3

# every symbol include/moe.h declares
EXPORTS = ("moe_create", "moe_load_experts", "moe_load_experts_ex", "moe_forward", "moe_forward_host",
           "moe_forward_stack", "moe_forward_stack_steps", "moe_forward_steps", "moe_load_router",
           "moe_debug_router_logits", "moe_set_batched_numerics", "moe_set_swiglu", "moe_get_status", "moe_debug_dequant",
           "moe_debug_route",
           "moe_debug_stack_trace", "moe_debug_mx_quantize", "moe_debug_batched_h",
           "moe_debug_forward_f32", "moe_debug_set_wait",
           "moe_last_bytes", "moe_expert_bytes", "moe_last_launches", "moe_last_error",
           "moe_forward_noalloc", "moe_debug_stream_weights", "moe_destroy",
           "moe_ops_create", "moe_ops_get_status", "moe_ops_destroy", "moe_kv_write", "moe_kv_read",
           "moe_attention", "moe_linear", "moe_sample", "moe_kv_plan", "moe_rope_turns", "moe_rope", "moe_lora")


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libmoe status {status}: {msg}")
        self.status = status


class moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("intermediate", ctypes.c_int),
                ("num_experts", ctypes.c_int), ("num_layers", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("max_top_k", ctypes.c_int),
                ("format", ctypes.c_int), ("group", ctypes.c_int), ("has_bias", ctypes.c_int)]


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num_blocks", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("block", ctypes.c_int),
                ("format", ctypes.c_int)]


class moe_kv_batch(ctypes.Structure):
    _fields_ = [("cu", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int), ("n_tokens", ctypes.c_int), ("table_stride", ctypes.c_int)]


class moe_linear_weights(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("format", ctypes.c_int),
                ("group", ctypes.c_int)]


class moe_kv_pool(ctypes.Structure):
    _fields_ = [("ring", ctypes.c_void_p), ("table", ctypes.c_void_p), ("ring_size", ctypes.c_int),
                ("n_seqs", ctypes.c_int), ("table_stride", ctypes.c_int), ("block", ctypes.c_int)]


class moe_rope_config(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("length", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


class moe_rope_table(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("mscale", ctypes.c_float)]


class moe_lora_weights(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n_adapters", ctypes.c_int), ("rank", ctypes.c_int), ("rows", ctypes.c_int),
                ("cols", ctypes.c_int)]


class moe_sample_params(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("u", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run python -m bit_moe_decode_02_gb300.build_ext")
        L = ctypes.CDLL(LIB_PATH)
        p, i, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        L.moe_create.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(p)]
        L.moe_create.restype = i
        L.moe_load_experts.argtypes = [p, i, p, p, p, p, p, p, p]
        L.moe_load_experts.restype = i
        L.moe_load_experts_ex.argtypes = [p, i, p, p, p, p, p, p, i, p]
        L.moe_load_experts_ex.restype = i
        L.moe_debug_stream_weights.argtypes = [p, i, i, ll, p]
        L.moe_debug_stream_weights.restype = i
        L.moe_set_batched_numerics.argtypes = [p, i]
        L.moe_set_batched_numerics.restype = i
        L.moe_set_swiglu.argtypes = [p, ctypes.c_float, ctypes.c_float, ctypes.c_float]
        L.moe_set_swiglu.restype = i
        L.moe_forward.argtypes = [p, i, p, p, i, i, p, p]
        L.moe_forward.restype = i
        L.moe_forward_host.argtypes = [p, i, p, p, i, i, p, p]
        L.moe_forward_host.restype = i
        L.moe_forward_stack.argtypes = [p, p, p, i, i, p]
        L.moe_forward_stack.restype = i
        L.moe_forward_stack_steps.argtypes = [p, i, p, p, i, i, p]
        L.moe_forward_stack_steps.restype = i
        L.moe_load_router.argtypes = [p, i, p, p]
        L.moe_load_router.restype = i
        L.moe_debug_router_logits.argtypes = [p, p, i, p]
        L.moe_debug_router_logits.restype = i
        L.moe_forward_steps.argtypes = [p, i, i, p, p, i, i, p, p]
        L.moe_forward_steps.restype = i
        L.moe_get_status.argtypes = [p, p]
        L.moe_get_status.restype = i
        L.moe_debug_dequant.argtypes = [p, i, i, i, p, p]
        L.moe_debug_dequant.restype = i
        L.moe_debug_route.argtypes = [p, p, i, i, p, p, p]
        L.moe_debug_route.restype = i
        L.moe_debug_stack_trace.argtypes = [p, p, p, i, i, p, p]
        L.moe_debug_stack_trace.restype = i
        L.moe_debug_mx_quantize.argtypes = [p, ll, p, p, p]
        L.moe_debug_mx_quantize.restype = i
        L.moe_debug_batched_h.argtypes = [p, p, p, p]
        L.moe_debug_batched_h.restype = i
        L.moe_debug_forward_f32.argtypes = [p, i, p, p, i, i, p, p, p]
        L.moe_debug_forward_f32.restype = i
        L.moe_debug_set_wait.argtypes = [p, i, i]
        L.moe_debug_set_wait.restype = i
        L.moe_last_bytes.argtypes = [p, p, ctypes.POINTER(ll)]
        L.moe_last_bytes.restype = i
        L.moe_expert_bytes.argtypes = [p]
        L.moe_expert_bytes.restype = ll
        L.moe_last_launches.argtypes = [p]
        L.moe_last_launches.restype = i
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_forward_noalloc.argtypes = [ctypes.POINTER(moe_config), p, p, p, p, p, p, p, p, i, i,
                                          p, p]
        L.moe_forward_noalloc.restype = i
        L.moe_destroy.argtypes = [p]
        L.moe_destroy.restype = None
        cache, batch = ctypes.POINTER(moe_kv_cache), ctypes.POINTER(moe_kv_batch)
        L.moe_ops_create.argtypes = [ctypes.POINTER(p)]
        L.moe_ops_create.restype = i
        L.moe_ops_get_status.argtypes = [p, p]
        L.moe_ops_get_status.restype = i
        L.moe_ops_destroy.argtypes = [p]
        L.moe_ops_destroy.restype = None
        L.moe_kv_write.argtypes = [p, cache, batch, p, ll, p, ll, p]
        L.moe_kv_write.restype = i
        L.moe_kv_read.argtypes = [p, cache, batch, p, ll, p, ll, p]
        L.moe_kv_read.restype = i
        L.moe_attention.argtypes = [p, cache, batch, p, ll, i, ctypes.c_float, i, p, p, p, p]
        L.moe_attention.restype = i
        L.moe_linear.argtypes = [p, ctypes.POINTER(moe_linear_weights), p, ll, i, p, ll, i, p]
        L.moe_linear.restype = i
        L.moe_sample.argtypes = [p, p, i, ll, i, i, ctypes.POINTER(moe_sample_params), p, p, p]
        L.moe_sample.restype = i
        L.moe_kv_plan.argtypes = [p, ctypes.POINTER(moe_kv_pool), p, p, p, i, p, p, p, p, p, p, p, p]
        L.moe_kv_plan.restype = i
        L.moe_rope_turns.argtypes = [ctypes.POINTER(moe_rope_config), p]
        L.moe_rope_turns.restype = i
        L.moe_rope.argtypes = [p, ctypes.POINTER(moe_rope_table), p, i, i, i, p, ll, i, p, ll, p, ll, i, p, ll, p]
        L.moe_rope.restype = i
        L.moe_lora.argtypes = [p, ctypes.POINTER(moe_lora_weights), p, p, ll, i, p, ll, p, ll, i, p]
        L.moe_lora.restype = i
        # the same calls with their arguments as 64-bit words (moe_ops.cu): one conversion instead of many
        for name in ("kv_write", "kv_read", "rope", "kv_plan", "lora"):
            f = getattr(L, "moe_words_" + name)
            f.argtypes = [ctypes.c_char_p]
            f.restype = i
        _lib = L
    return _lib


_WORDS_KV = struct.Struct("=8q").pack
_WORDS_ROPE, _WORDS_PLAN, _WORDS_LORA = struct.Struct("=17q").pack, struct.Struct("=14q").pack, struct.Struct("=12q").pack


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def _check(rc: int) -> int:
    if rc != MOE_OK:
        raise MoeError(rc, moe_last_error())
    return rc


def _ptr(t):
    """device or host address of a torch tensor / numpy array / int / None"""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_create(hidden, intermediate, num_experts, num_layers=1, max_tokens=1, max_top_k=4,
               format=MOE_FMT_MXFP4, group=32, has_bias=1) -> int:
    cfg = moe_config(hidden, intermediate, num_experts, num_layers, max_tokens, max_top_k,
                     format, group, int(has_bias))
    h = ctypes.c_void_p()
    _check(lib().moe_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h.value


def moe_load_experts(h, layer, gu_codes, gu_scales, gu_bias, dn_codes, dn_scales, dn_bias,
                     stream=None):
    return _check(lib().moe_load_experts(h, layer, _ptr(gu_codes), _ptr(gu_scales), _ptr(gu_bias),
                                         _ptr(dn_codes), _ptr(dn_scales), _ptr(dn_bias),
                                         _stream(stream)))


def moe_load_experts_ex(h, layer, gu_codes, gu_scales, gu_bias, dn_codes, dn_scales, dn_bias, flags,
                        stream=None):
    return _check(lib().moe_load_experts_ex(h, layer, _ptr(gu_codes), _ptr(gu_scales), _ptr(gu_bias),
                                            _ptr(dn_codes), _ptr(dn_scales), _ptr(dn_bias), flags,
                                            _stream(stream)))


def moe_forward(h, layer, x, logits, M, top_k, out, stream=None):
    return _check(lib().moe_forward(h, layer, _ptr(x), _ptr(logits), M, top_k, _ptr(out),
                                    _stream(stream)))


def moe_forward_host(h, layer, x, logits, M, top_k, out, stream=None):
    return _check(lib().moe_forward_host(h, layer, _ptr(x), _ptr(logits), M, top_k, _ptr(out),
                                         _stream(stream)))


def moe_forward_stack(h, resid, logits, M, top_k, stream=None):
    return _check(lib().moe_forward_stack(h, _ptr(resid), _ptr(logits), M, top_k, _stream(stream)))


def moe_forward_stack_steps(h, n, resid, logits, M, top_k, stream=None):
    return _check(lib().moe_forward_stack_steps(h, n, _ptr(resid), _ptr(logits), M, top_k, _stream(stream)))


def moe_load_router(h, layer, w, bias=None):
    """Router weights w bf16 bits [E][H] and bias [E] (numpy uint16 arrays or tensors)."""
    return _check(lib().moe_load_router(h, layer, _ptr(w), _ptr(bias)))


def moe_debug_stream_weights(h, layer0, n, nbytes, stream=None):
    return _check(lib().moe_debug_stream_weights(h, layer0, n, nbytes, _stream(stream)))


def moe_set_swiglu(h, alpha, limit, beta):
    return _check(lib().moe_set_swiglu(h, alpha, limit, beta))


def moe_set_batched_numerics(h, numerics):
    return _check(lib().moe_set_batched_numerics(h, numerics))


def moe_debug_router_logits(h, out, M, stream=None):
    return _check(lib().moe_debug_router_logits(h, _ptr(out), M, _stream(stream)))


def moe_forward_steps(h, n, layer0, x, logits, M, top_k, out, stream=None):
    return _check(lib().moe_forward_steps(h, n, layer0, _ptr(x), _ptr(logits), M, top_k, _ptr(out),
                                          _stream(stream)))


def moe_get_status(h, stream=None) -> int:
    return lib().moe_get_status(h, _stream(stream))


def moe_debug_dequant(h, layer, expert, proj, out, stream=None):
    return _check(lib().moe_debug_dequant(h, layer, expert, proj, _ptr(out), _stream(stream)))


def moe_debug_route(h, logits, M, top_k, idx, w, stream=None):
    return _check(lib().moe_debug_route(h, _ptr(logits), M, top_k, _ptr(idx), _ptr(w),
                                        _stream(stream)))


def moe_debug_stack_trace(h, resid, logits, M, top_k, trace, stream=None):
    return _check(lib().moe_debug_stack_trace(h, _ptr(resid), _ptr(logits), M, top_k, _ptr(trace),
                                              _stream(stream)))


def moe_debug_mx_quantize(x, n, codes, scales, stream=None):
    return _check(lib().moe_debug_mx_quantize(_ptr(x), n, _ptr(codes), _ptr(scales), _stream(stream)))


def moe_debug_batched_h(h, codes, scales, stream=None):
    return _check(lib().moe_debug_batched_h(h, _ptr(codes), _ptr(scales), _stream(stream)))


def moe_debug_forward_f32(h, layer, x, logits, M, top_k, out, out_f32, stream=None):
    return _check(lib().moe_debug_forward_f32(h, layer, _ptr(x), _ptr(logits), M, top_k, _ptr(out),
                                              _ptr(out_f32), _stream(stream)))


def moe_debug_set_wait(h, spin_limit, skip_cta=-1):
    return _check(lib().moe_debug_set_wait(h, spin_limit, skip_cta))


def moe_last_bytes(h, stream=None) -> int:
    b = ctypes.c_longlong()
    _check(lib().moe_last_bytes(h, _stream(stream), ctypes.byref(b)))
    return b.value


def moe_expert_bytes(h) -> int:
    return lib().moe_expert_bytes(h)


def moe_last_launches(h) -> int:
    return lib().moe_last_launches(h)


def moe_forward_noalloc(cfg: moe_config, gu_codes, gu_scales, gu_bias, dn_codes, dn_scales, dn_bias,
                        x, logits, M, top_k, out, stream=None):
    """The allocation-free layer forward (see include/moe.h): caller-layout
    weights, inputs and outputs are all caller memory; scratch is the
    library's fixed device array."""
    return _check(lib().moe_forward_noalloc(ctypes.byref(cfg), _ptr(gu_codes), _ptr(gu_scales),
                                            _ptr(gu_bias), _ptr(dn_codes), _ptr(dn_scales),
                                            _ptr(dn_bias), _ptr(x), _ptr(logits), M, top_k,
                                            _ptr(out), _stream(stream)))


def moe_destroy(h) -> None:
    lib().moe_destroy(h)


# ------------------------------------------- operators around the expert block

def _need(t, name, dtype, dims):
    """A CUDA tensor of that type and number of dimensions, its last dimension
    contiguous: what the C call, which sees only an address, takes it for."""
    if not t.is_cuda or t.dim() != dims or t.dtype is not dtype or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name}: a CUDA tensor of {dtype} with {dims} dimensions, the last one contiguous, is needed "
                         f"(got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device})")
    return t


def _dense(t, name, dtype, dims):
    if not _need(t, name, dtype, dims).is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is needed (shape {tuple(t.shape)}, strides {t.stride()})")
    return t


def moe_ops_create() -> int:
    h = ctypes.c_void_p()
    _check(lib().moe_ops_create(ctypes.byref(h)))
    return h.value


def moe_ops_get_status(o, stream=None) -> int:
    return lib().moe_ops_get_status(o, _stream(stream))


def moe_ops_destroy(o) -> None:
    lib().moe_ops_destroy(o)


def moe_kv_cache_of(codes, scales, block, head_dim, format) -> moe_kv_cache:
    """The cache in codes uint8 [num_blocks][kv_heads][2][block * head_dim] and scales fp32
    [num_blocks][kv_heads][2]; MOE_KV_MXFP4: codes [num_blocks][kv_heads][2][block * head_dim * 17 / 32], scales None."""
    import torch
    mx = format == MOE_KV_MXFP4
    _dense(codes, "codes", torch.uint8, 4)
    nb, heads = codes.shape[:2]
    if mx:
        if scales is not None:
            raise ValueError("moe_kv_cache_of: an MXFP4 cache holds its scales with its codes: scales must be None")
    elif tuple(_dense(scales, "scales", torch.float32, 3).shape) != (nb, heads, 2):
        raise ValueError(f"moe_kv_cache_of: scales {tuple(scales.shape)} are not [{nb}][{heads}][2]")
    if tuple(codes.shape[2:]) != (2, block * head_dim * 17 // 32 if mx else block * head_dim):
        raise ValueError(f"moe_kv_cache_of: codes {tuple(codes.shape)} are not a cache of blocks of {block} tokens with head_dim "
                         f"{head_dim}")
    c = moe_kv_cache(codes.data_ptr(), None if mx else scales.data_ptr(), nb, heads, head_dim, block, format)
    c.tensors = (codes, scales)
    return c


def moe_kv_batch_of(cu, kv_len, table, n_tokens) -> moe_kv_batch:
    """The batch in int32 cu [n_seqs + 1], kv_len [n_seqs] and table [n_seqs][table_stride]."""
    import torch
    _dense(cu, "cu", torch.int32, 1)
    _dense(kv_len, "kv_len", torch.int32, 1)
    _dense(table, "table", torch.int32, 2)
    n = kv_len.shape[0]
    if cu.shape[0] != n + 1 or table.shape[0] != n:
        raise ValueError(f"moe_kv_batch_of: cu {tuple(cu.shape)}, kv_len {tuple(kv_len.shape)} and table {tuple(table.shape)} "
                         "do not describe the same sequences")
    b = moe_kv_batch(cu.data_ptr(), kv_len.data_ptr(), table.data_ptr(), n, n_tokens, table.shape[1])
    b.tensors = (cu, kv_len, table)
    return b


def _word(handle) -> int:
    """A handle as a 64-bit word: an address, None or what ctypes takes for a pointer (None: 0, which the library refuses)."""
    return handle if type(handle) is int else ctypes.cast(handle, ctypes.c_void_p).value or 0


_current = None


def _raw_stream(stream, t):
    """The stream's handle; None: the current stream of the tensor's device (asked for by its handle alone: building a
    torch.cuda.Stream takes as long as a launch)."""
    global _current
    if stream is None:
        if _current is None:
            import torch
            _current = torch._C._cuda_getCurrentRawStream
        return _current(t.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _heads(t, name, T, H, D):
    """Address and row stride of bf16 rows [T][H][D] with contiguous heads."""
    import torch
    st = t.stride()
    if t.dtype is not torch.bfloat16 or not t.is_cuda or t.shape != (T, H, D) or st[2] != 1 or (st[1] != D and H > 1):
        raise ValueError(f"{name}: CUDA bf16 rows [{T}][{H}][{D}] with contiguous heads are needed (got {t.dtype} "
                         f"{tuple(t.shape)}, strides {st}, on {t.device})")
    return t.data_ptr(), st[0] if T > 1 else H * D


def moe_kv_write(o, cache, batch, k, v, stream=None):
    T, H, D = batch.n_tokens, cache.kv_heads, cache.head_dim
    kp, ks = _heads(k, "k", T, H, D)
    vp, vs = _heads(v, "v", T, H, D)
    rc = lib().moe_words_kv_write(_WORDS_KV(_word(o), ctypes.addressof(cache), ctypes.addressof(batch), kp, ks, vp, vs, _raw_stream(stream, k)))
    return rc if rc == MOE_OK else _check(rc)


def moe_kv_read(o, cache, batch, k, v, stream=None):
    T, H, D = batch.n_tokens, cache.kv_heads, cache.head_dim
    kp, ks = _heads(k, "k", T, H, D)
    vp, vs = _heads(v, "v", T, H, D)
    rc = lib().moe_words_kv_read(_WORDS_KV(_word(o), ctypes.addressof(cache), ctypes.addressof(batch), kp, ks, vp, vs, _raw_stream(stream, k)))
    return rc if rc == MOE_OK else _check(rc)


def moe_attention(o, cache, batch, q, out, lse=None, sinks=None, window=0, scale=None, stream=None):
    """q bf16 [n_tokens][q_heads][head_dim] (rows may be strided), out like it and contiguous, lse fp32
    [n_tokens][q_heads], sinks fp32 [q_heads]; scale defaults to head_dim ** -0.5."""
    import torch
    T, heads, D = batch.n_tokens, q.shape[1] if q.dim() == 3 else 0, cache.head_dim
    qp, qs = _heads(q, "q", T, heads, D)
    op, _ = _heads(out, "out", T, heads, D)
    if not out.is_contiguous():
        raise ValueError(f"moe_attention: out must be contiguous (strides {out.stride()})")
    if lse is not None and (lse.shape != (T, heads) or lse.dtype is not torch.float32 or not lse.is_cuda or not lse.is_contiguous()):
        raise ValueError(f"moe_attention: lse must be a contiguous CUDA fp32 tensor [{T}][{heads}]")
    if sinks is not None and (sinks.shape != (heads,) or sinks.dtype is not torch.float32 or not sinks.is_cuda or
                              not sinks.is_contiguous()):
        raise ValueError(f"moe_attention: sinks must be a contiguous CUDA fp32 tensor [{heads}]")
    return _check(lib().moe_attention(o, cache, batch, qp, qs, heads, D ** -0.5 if scale is None else scale, window,
                                      None if sinks is None else sinks.data_ptr(), op, None if lse is None else lse.data_ptr(),
                                      _raw_stream(stream, q)))


def moe_kv_pool_of(ring, table, block) -> moe_kv_pool:
    """The pool of free blocks in ring int32 [number of blocks], with the block tables int32 [n_seqs][table_stride]."""
    import torch
    _dense(ring, "ring", torch.int32, 1)
    _dense(table, "table", torch.int32, 2)
    c = moe_kv_pool(ring.data_ptr(), table.data_ptr(), ring.shape[0], table.shape[0], table.shape[1], block)
    c.tensors = (ring, table)
    return c


_kinds = None


def _types():
    """torch.bfloat16, float32, int32, int64, looked up once."""
    global _kinds
    if _kinds is None:
        import torch
        _kinds = torch.bfloat16, torch.float32, torch.int32, torch.int64
    return _kinds


def _array(t, name, dtype, n):
    """Address of a contiguous CUDA tensor [n] of that type."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous CUDA tensor of {dtype} [{n}] is needed (got {t.dtype} {tuple(t.shape)} on {t.device})")
    return t.data_ptr()


def moe_kv_plan(o, pool, n_new, kv_len, state, cu, kv_len_out, state_out, admitted=None, seq=None, position=None, slot=None,
                n_tokens=None, stream=None):
    """n_new, kv_len, kv_len_out int32 [n_seqs], state, state_out int32 [2], cu int32 [n_seqs + 1], admitted int32 [1], seq and
    position int32 and slot int64 [n_tokens]; n_tokens (their length) has to be given where all three are None."""
    i, n = _types()[2], pool.n_seqs
    if n_tokens is None:
        t = slot if slot is not None else position if position is not None else seq
        if t is None:
            raise ValueError("moe_kv_plan: n_tokens is needed where seq, position and slot are None")
        n_tokens = t.shape[0]
    rc = lib().moe_words_kv_plan(_WORDS_PLAN(
        _word(o), ctypes.addressof(pool), _array(n_new, "n_new", i, n), _array(kv_len, "kv_len", i, n), _array(state, "state", i, 2), n_tokens,
        _array(cu, "cu", i, n + 1), _array(kv_len_out, "kv_len_out", i, n), _array(state_out, "state_out", i, 2),
        0 if admitted is None else _array(admitted, "admitted", i, 1), 0 if seq is None else _array(seq, "seq", i, n_tokens),
        0 if position is None else _array(position, "position", i, n_tokens),
        0 if slot is None else _array(slot, "slot", _types()[3], n_tokens), _raw_stream(stream, n_new)))
    return rc if rc == MOE_OK else _check(rc)


def moe_rope_turns(rot_dim, base, scaling=MOE_ROPE_PLAIN, factor=1.0, length=0.0, low=0.0, high=0.0):
    """Each pair's turns a position, as 64-bit fractions: a numpy array of uint64 [rot_dim / 2]."""
    import numpy as np
    out = np.empty(max(int(rot_dim) // 2, 1), np.uint64)
    c = moe_rope_config(rot_dim, scaling, base, factor, length, low, high)
    _check(lib().moe_rope_turns(ctypes.byref(c), out.ctypes.data))
    return out


def moe_rope_of(rot_dim, base, layout=MOE_ROPE_HALF, scaling=MOE_ROPE_PLAIN, factor=1.0, length=0.0, low=0.0, high=0.0, mscale=1.0,
                device="cuda") -> moe_rope_table:
    """The table of a configuration, on the device (see include/moe.h)."""
    import numpy as np
    import torch
    t = torch.from_numpy(moe_rope_turns(rot_dim, base, scaling, factor, length, low, high).view(np.int64)).to(device)
    r = moe_rope_table(t.data_ptr(), rot_dim, layout, mscale)
    r.tensors = (t,)
    return r


def _head_rows(t, name, kind, T, heads, D):
    """Address and row stride of rows [T][heads][D] of a type, with contiguous heads."""
    st = t.stride()
    if t.dtype is not kind or not t.is_cuda or t.shape != (T, heads, D) or st[2] != 1 or (st[1] != D and heads > 1):
        raise ValueError(f"{name}: CUDA rows [{T}][{heads}][{D}] of {kind} with contiguous heads are needed (got {t.dtype} {tuple(t.shape)}, "
                         f"strides {st}, on {t.device})")
    return t.data_ptr(), st[0] if T > 1 else heads * D


def moe_rope(o, rope, position, q, k=None, q_out=None, k_out=None, stream=None):
    """q [T][q_heads][head_dim], k [T][k_heads][head_dim] or None, of bf16 or fp32; q_out, k_out like them (None: in place);
    position int32 [T].  Rows may be strided, heads are contiguous."""
    bf16, fp32, i32, _ = _types()
    T, heads, D = q.shape if q.dim() == 3 else (0, 0, 0)
    kind = q.dtype
    if kind is bf16:
        code = MOE_DT_BF16
    elif kind is fp32:
        code = MOE_DT_F32
    else:
        raise ValueError(f"moe_rope: q must be bf16 or fp32 (got {kind})")
    pos = _array(position, "position", i32, T)
    qp, qs = _head_rows(q, "q", kind, T, heads, D)
    op, os_ = (qp, qs) if q_out is None else _head_rows(q_out, "q_out", kind, T, heads, D)
    if k is not None:
        kh = k.shape[1] if k.dim() == 3 else 0
        kp, ks = _head_rows(k, "k", kind, T, kh, D)
        lp, ls = (kp, ks) if k_out is None else _head_rows(k_out, "k_out", kind, T, kh, D)
    elif k_out is None:
        kp = lp = kh = ks = ls = 0
    else:
        raise ValueError("moe_rope: k_out without k")
    rc = lib().moe_words_rope(_WORDS_ROPE(_word(o), 0 if rope is None else ctypes.addressof(rope), pos, T, D, code, qp, qs, heads, op, os_,
                                          kp, ks, kh, lp, ls, _raw_stream(stream, q)))
    return rc if rc == MOE_OK else _check(rc)


def moe_lora_of(a, b, scale=None) -> moe_lora_weights:
    """Adapters in a bf16 [n_adapters][rank][cols], b bf16 [n_adapters][rows][rank], scale fp32 [n_adapters] or None."""
    import torch
    _dense(a, "a", torch.bfloat16, 3)
    _dense(b, "b", torch.bfloat16, 3)
    n, rank, cols = a.shape
    if b.shape[0] != n or b.shape[2] != rank:
        raise ValueError(f"moe_lora_of: a {tuple(a.shape)} and b {tuple(b.shape)} are not adapters of one rank")
    if scale is not None and _dense(scale, "scale", torch.float32, 1).shape[0] != n:
        raise ValueError(f"moe_lora_of: scale {tuple(scale.shape)} is not [{n}]")
    w = moe_lora_weights(a.data_ptr(), b.data_ptr(), _ptr(scale), n, rank, b.shape[1], cols)
    w.tensors = (a, b, scale)
    return w


def _out_rows(t, name, kind, M, rows):
    """Address and stride of rows [M][rows] of a type."""
    st = t.stride()
    if t.dtype is not kind or t.shape != (M, rows) or not t.is_cuda or (st[1] != 1 and rows > 1):
        raise ValueError(f"moe_lora: {name} must be CUDA {kind} rows [{M}][{rows}], y and out of one type (got {t.dtype} {tuple(t.shape)}, "
                         f"strides {st}, on {t.device})")
    return t.data_ptr(), st[0] if M > 1 else rows


def moe_lora(o, w, index, x, y, out=None, stream=None):
    """x bf16 [M][cols], y fp32 or bf16 [M][rows] or None (0), out like y (None: y, in place); rows may be strided; index int32
    [M], -1: no adapter."""
    bf16, fp32, i32, _ = _types()
    rows, cols = w.rows, w.cols
    if out is None:
        out = y
    if out is None:
        raise ValueError("moe_lora: out is needed where y is None")
    M, kind, sx = x.shape[0], out.dtype, x.stride()
    at = _array(index, "index", i32, M)
    if x.dtype is not bf16 or x.shape != (M, cols) or not x.is_cuda or sx[1] != 1:
        raise ValueError(f"moe_lora: x must be CUDA bf16 rows [M][{cols}] (got {x.dtype} {tuple(x.shape)}, strides {sx}, on {x.device})")
    if kind is bf16:
        code = MOE_DT_BF16
    elif kind is fp32:
        code = MOE_DT_F32
    else:
        raise ValueError(f"moe_lora: y and out must be bf16 or fp32 (got {kind})")
    op, so = _out_rows(out, "out", kind, M, rows)
    yp, sy = (0, 0) if y is None else (op, so) if y is out else _out_rows(y, "y", kind, M, rows)
    rc = lib().moe_words_lora(_WORDS_LORA(_word(o), ctypes.addressof(w), at, x.data_ptr(), sx[0] if M > 1 else cols, M, yp, sy, op, so, code,
                                          _raw_stream(stream, x)))
    return rc if rc == MOE_OK else _check(rc)


def moe_linear_of(codes, scales, bias, format, group) -> moe_linear_weights:
    """Weights in codes uint8 [rows][cols / 2], scales uint8 [rows][cols / 32] (MXFP4) or fp16 [rows][cols / group]
    (int4), bias bf16 [rows] or None."""
    import torch
    _dense(codes, "codes", torch.uint8, 2)
    _dense(scales, "scales", torch.uint8 if format == MOE_FMT_MXFP4 else torch.float16, 2)
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    if scales.shape[0] != rows or scales.shape[1] * group != cols:
        raise ValueError(f"moe_linear_of: scales {tuple(scales.shape)} are not one per {group} of [{rows}][{cols}]")
    if bias is not None and _dense(bias, "bias", torch.bfloat16, 1).shape[0] != rows:
        raise ValueError(f"moe_linear_of: bias {tuple(bias.shape)} is not [{rows}]")
    w = moe_linear_weights(codes.data_ptr(), scales.data_ptr(), _ptr(bias), rows, cols, format, group)
    w.tensors = (codes, scales, bias)
    return w


def moe_linear(o, w, x, out, stream=None):
    """x bf16 [M][cols], out fp32 or bf16 [M][rows]; the rows of both may be strided."""
    import torch
    rows, cols, kind = w.rows, w.cols, out.dtype
    sx, so = x.stride(), out.stride()
    M = x.shape[0]
    if (x.shape != (M, cols) or x.dtype is not torch.bfloat16 or not x.is_cuda or sx[1] != 1 or out.shape != (M, rows) or
            (kind is not torch.bfloat16 and kind is not torch.float32) or not out.is_cuda or (so[1] != 1 and rows > 1)):
        raise ValueError(f"moe_linear: x bf16 [M][{cols}] and out fp32 or bf16 [M][{rows}] on the GPU with contiguous rows are "
                         f"needed (got {x.dtype} {tuple(x.shape)} strides {sx}, {kind} {tuple(out.shape)} strides {so})")
    return _check(lib().moe_linear(o, w, x.data_ptr(), sx[0] if M > 1 else cols, M, out.data_ptr(), so[0] if M > 1 else rows,
                                   MOE_DT_BF16 if kind is torch.bfloat16 else MOE_DT_F32, _raw_stream(stream, x)))


def _per_row(t, name, dtype, M):
    if t is None:
        return None
    if t.shape != (M,) or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"moe_sample: {name} must be a contiguous CUDA tensor of {dtype} [{M}] (got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device})")
    return t.data_ptr()


def moe_sample(o, logits, temperature, top_k, top_p, min_p, u, token, logprob=None, stream=None):
    """logits fp32 or bf16 [M][V] (rows may be strided); temperature, top_p, min_p, u fp32 [M] and top_k int32 [M], each
    but u possibly None; token int32 [M], logprob fp32 [M] or None."""
    import torch
    bf = logits.dtype is torch.bfloat16
    _need(logits, "logits", torch.bfloat16 if bf else torch.float32, 2)
    M, V = logits.shape
    f = torch.float32
    par = moe_sample_params(_per_row(temperature, "temperature", f, M), _per_row(top_k, "top_k", torch.int32, M),
                            _per_row(top_p, "top_p", f, M), _per_row(min_p, "min_p", f, M), _per_row(u, "u", f, M))
    return _check(lib().moe_sample(o, logits.data_ptr(), MOE_DT_BF16 if bf else MOE_DT_F32, logits.stride(0) if M > 1 else V, M, V,
                                   par, _per_row(token, "token", torch.int32, M), _per_row(logprob, "logprob", f, M),
                                   _raw_stream(stream, logits)))
