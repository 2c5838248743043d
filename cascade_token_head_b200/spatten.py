"""Thin ctypes binding of libspatten.so (include/spatten.h).  Argument marshalling only: every step
of the computation runs in the library's CUDA kernels (and cuBLASLt for the FC projections).

Importing this module loads the library and raises ImportError if it has not been built
(``python -m cascade_token_head_b200.build``); there is no fallback implementation.
Functions take torch tensors (device memory) or raw integer pointers, and run on torch's current
CUDA stream unless a stream is given.  Each returns None and raises SpattenError on a non-OK
status.
"""
from __future__ import annotations

import ctypes as C
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspatten.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m cascade_token_head_b200.build`")
lib = C.CDLL(LIB_PATH)

# ---- enums (spatten.h) --------------------------------------------------------------------------
OK, E_ARG, E_SHAPE, E_ALIGN, E_WORKSPACE, E_NONFINITE, E_CUDA, E_TIMEOUT, E_UNSUPPORTED, E_INDEX, E_RANGE = range(11)
F32, BF16 = 0, 1
PREFILL, DECODE_STEP = 0, 1
ATTN_AUTO, ATTN_CUDA_CORE, ATTN_TENSOR_CORE, ATTN_DECODE, ATTN_DECODE_PREDICATED = 0, 1, 2, 3, 4
MAX_LAYERS = 64

vp, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t


class attn_args(C.Structure):
    _fields_ = [("B", i32), ("H", i32), ("n_q", i32), ("n_kv", i32), ("d_h", i32), ("H_kept", i32),
                ("head_idx", vp), ("head_idx_ld", i64),
                ("q", vp), ("q_dtype", i32), ("q_ld_tok", i64),
                ("quantized", i32), ("k_msb", vp), ("k_lsb", vp), ("k_scale", vp),
                ("v_msb", vp), ("v_lsb", vp), ("v_scale", vp), ("kv_cap", i32),
                ("k", vp), ("v", vp), ("kv_dtype", i32), ("kv_ld_tok", i64),
                ("kv_idx", vp), ("kv_idx_ld", i64),
                ("sm_scale", f32), ("refetch_threshold", f32),
                ("o", vp), ("o_ld_tok", i64), ("zero_pruned_heads", i32),
                ("tok_imp", vp), ("tok_imp_ld", i64), ("tok_imp_map", vp), ("tok_imp_map_ld", i64),
                ("head_imp", vp), ("refetch_flags", vp), ("refetch_flags_ld", i64), ("refetch_count", vp),
                ("dev_status", vp),
                ("kernel", i32), ("v_keep", i32)]


class cascade_cfg(C.Structure):
    _fields_ = [("mode", i32), ("B", i32), ("T", i32), ("D", i32), ("H", i32), ("d_h", i32), ("L", i32),
                ("dtype", i32), ("token_keep", i32 * MAX_LAYERS), ("head_keep", i32 * MAX_LAYERS),
                ("quant", i32), ("refetch_threshold", f32), ("sm_scale", f32)]


class layer_weights(C.Structure):
    _fields_ = [("w_qkv", vp), ("w_o", vp)]


class decode_cache(C.Structure):
    _fields_ = [("k_msb", vp), ("k_lsb", vp), ("k_scale", vp), ("v_msb", vp), ("v_lsb", vp), ("v_scale", vp)]


class cascade_io(C.Structure):
    _fields_ = [("x", vp), ("key_gain", vp), ("x_out", vp), ("kept_tok", vp), ("kept_head", vp),
                ("tok_imp", vp), ("head_imp", vp), ("refetch_count", vp), ("sat_count", vp), ("dev_status", vp),
                ("caches", C.POINTER(decode_cache)), ("cap", i32), ("n_old", i32), ("dec_tok_imp", vp),
                ("trace_x", vp), ("trace_qkv", vp), ("trace_o", vp), ("trace_tok_imp", vp),
                ("trace_head_imp", vp), ("trace_flags", vp), ("attn_events", C.POINTER(vp))]


class prompt_args(C.Structure):
    _fields_ = [("B", i32), ("H", i32), ("H_kv", i32), ("d_h", i32), ("total_q", i32), ("total_kv", i32),
                ("cu_q", vp), ("cu_kv", vp), ("dtype", i32), ("q", vp), ("q_ld_tok", i64),
                ("k", vp), ("v", vp), ("kv_ld_tok", i64), ("o", vp), ("o_ld_tok", i64), ("sm_scale", f32),
                ("weight", vp), ("weight_ld_seq", i64), ("weight_ld_head", i64), ("weight_cap", i32),
                ("dev_status", vp), ("kernel", i32), ("weight_len", vp)]


class kv4_cache(C.Structure):
    _fields_ = [("B", i32), ("H_kv", i32), ("d_h", i32), ("cap", i32),
                ("k_codes", vp), ("k_scale", vp), ("v_codes", vp), ("v_scale", vp), ("weight", vp), ("pos", vp)]


class kv4_attn_args(C.Structure):
    _fields_ = [("cache", kv4_cache), ("H", i32), ("q", vp), ("dtype", i32), ("q_ld", i64), ("o", vp), ("o_ld", i64),
                ("len", vp), ("n_max", i32), ("sm_scale", f32), ("update_weight", i32), ("dev_status", vp)]


lib.spatten_abi_version.restype = i32
lib.spatten_status_string.restype = C.c_char_p
lib.spatten_status_string.argtypes = [i32]
lib.spatten_last_cuda_error.restype = C.c_char_p
lib.spatten_kernel_launch_count.restype = C.c_uint64
lib.spatten_set_wait_limit.restype = None
lib.spatten_set_wait_limit.argtypes = [C.c_uint32]
lib.spatten_quantize_kv.restype = i32
lib.spatten_quantize_kv.argtypes = [vp, i32, i32, i32, i32, i32, i64, vp, i64, vp, vp, vp, i32, i32, vp, vp, vp]
lib.spatten_attention_workspace_size.restype = sz
lib.spatten_attention_workspace_size.argtypes = [C.POINTER(attn_args)]
lib.spatten_attention_layer.restype = i32
lib.spatten_attention_layer.argtypes = [C.POINTER(attn_args), vp, sz, vp]
lib.spatten_attention_layer_noalloc.restype = i32
lib.spatten_attention_layer_noalloc.argtypes = [C.POINTER(attn_args), vp]
lib.spatten_selftest_exp2_poly.restype = i32
lib.spatten_selftest_exp2_poly.argtypes = [vp, vp, i64, vp]
lib.spatten_topk_workspace_size.restype = sz
lib.spatten_topk_workspace_size.argtypes = [i32, i32, i32]
lib.spatten_topk_select.restype = i32
lib.spatten_topk_select.argtypes = [vp, i32, i32, i64, i32, vp, i64, vp, i64, vp, vp, sz, vp, vp]
lib.spatten_gather_kept.restype = i32
lib.spatten_gather_kept.argtypes = [vp, i64, i64, i32, i64, i32, vp, i64, i32, vp, i64, i64, vp, i64, vp, i32, vp, vp]
lib.spatten_cascade_workspace_size.restype = sz
lib.spatten_cascade_workspace_size.argtypes = [C.POINTER(cascade_cfg)]
lib.spatten_cascade_forward.restype = i32
lib.spatten_cascade_forward.argtypes = [C.POINTER(cascade_cfg), C.POINTER(layer_weights), C.POINTER(cascade_io), vp, sz, vp]
lib.spatten_prompt_workspace_size.restype = sz
lib.spatten_prompt_workspace_size.argtypes = [C.POINTER(prompt_args)]
lib.spatten_prompt_attention.restype = i32
lib.spatten_prompt_attention.argtypes = [C.POINTER(prompt_args), vp, sz, vp]
lib.spatten_kv4_append.restype = i32
lib.spatten_kv4_append.argtypes = [C.POINTER(kv4_cache), vp, vp, i32, i64, i32, vp, vp, vp, vp, vp, vp, vp]
lib.spatten_kv4_read.restype = i32
lib.spatten_kv4_read.argtypes = [C.POINTER(kv4_cache), vp, vp, i32, vp, vp, i32, i64, vp, vp]
lib.spatten_kv4_attention_workspace_size.restype = sz
lib.spatten_kv4_attention_workspace_size.argtypes = [C.POINTER(kv4_attn_args)]
lib.spatten_kv4_attention.restype = i32
lib.spatten_kv4_attention.argtypes = [C.POINTER(kv4_attn_args), vp, sz, vp]
lib.spatten_kv4_evict_workspace_size.restype = sz
lib.spatten_kv4_evict_workspace_size.argtypes = [C.POINTER(kv4_cache), i32, i32]
lib.spatten_kv4_evict.restype = i32
lib.spatten_kv4_evict.argtypes = [C.POINTER(kv4_cache), C.POINTER(kv4_cache), vp, vp, vp, i32, i32, i32, vp, sz, vp, vp]

# every extern "C" symbol of include/spatten.h
EXPORTS = ["spatten_abi_version", "spatten_status_string", "spatten_last_cuda_error",
           "spatten_kernel_launch_count", "spatten_quantize_kv",
           "spatten_attention_workspace_size", "spatten_attention_layer", "spatten_attention_layer_noalloc",
           "spatten_topk_workspace_size",
           "spatten_topk_select", "spatten_gather_kept", "spatten_cascade_workspace_size",
           "spatten_cascade_forward", "spatten_selftest_exp2_poly", "spatten_set_wait_limit",
           "spatten_prompt_workspace_size", "spatten_prompt_attention", "spatten_kv4_append", "spatten_kv4_read",
           "spatten_kv4_attention_workspace_size", "spatten_kv4_attention", "spatten_kv4_evict_workspace_size",
           "spatten_kv4_evict"]


class SpattenError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib.spatten_status_string(status).decode()
        if status == E_CUDA:
            msg += f" ({lib.spatten_last_cuda_error().decode()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


def check(status: int, where: str) -> None:
    if status != OK:
        raise SpattenError(status, where)


def ptr(t) -> int | None:
    """Device address of a torch tensor (None passes through; ints are taken as addresses)."""
    if t is None:
        return None
    try:
        return t.data_ptr()
    except AttributeError:
        return t


_current_stream = None


def _stream(stream) -> int | None:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    global _current_stream
    if _current_stream is None:
        import torch
        torch.cuda.current_stream()   # initialises CUDA; its Stream object costs 3 us a call, the handle alone 0.2
        device, raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _current_stream = lambda: raw(device())
    return _current_stream()


_dtype_codes: dict = {}   # torch dtype -> code, filled as dtypes are met (a lookup in `torch` costs 0.1 us a call)


def dtype_code(t) -> int:
    code = _dtype_codes.get(t.dtype)
    if code is None:
        import torch
        code = {torch.float32: F32, torch.bfloat16: BF16}.get(t.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
        _dtype_codes[t.dtype] = code
    return code


# ---- calls --------------------------------------------------------------------------------------
def quantize_kv(x, B, H, n, d_h, ld_tok, msb, lsb, cap, row0=0, scale_out=None, scale_in=None,
                row_gain=None, ld_gain=0, sat_count=None, dtype=None, stream=None):
    dt = dtype_code(x) if dtype is None and not isinstance(x, int) else dtype
    check(lib.spatten_quantize_kv(ptr(x), dt, B, H, n, d_h, ld_tok, ptr(row_gain), ld_gain, ptr(scale_in),
                                  ptr(msb), ptr(lsb), cap, row0, ptr(scale_out), ptr(sat_count), _stream(stream)),
          "spatten_quantize_kv")


def attention_workspace_size(args: attn_args) -> int:
    return lib.spatten_attention_workspace_size(C.byref(args))


def attention_layer(args: attn_args, ws, ws_bytes: int, stream=None):
    check(lib.spatten_attention_layer(C.byref(args), ptr(ws), ws_bytes, _stream(stream)), "spatten_attention_layer")


NOALLOC_SCRATCH_BYTES = 8 << 20   # SPATTEN_NOALLOC_SCRATCH_BYTES


def attention_layer_noalloc(args: attn_args, stream=None):
    """The attention layer without a caller workspace (library-owned scratch; see spatten.h)."""
    check(lib.spatten_attention_layer_noalloc(C.byref(args), _stream(stream)), "spatten_attention_layer_noalloc")


def topk_workspace_size(R: int, n: int, k: int) -> int:
    return lib.spatten_topk_workspace_size(R, n, k)


def topk_select(scores, R, n, ld, k, idx_out, ld_out, map=None, ld_map=0, comp_out=None, ws=None, ws_bytes=0,
                dev_status=None, stream=None):
    check(lib.spatten_topk_select(ptr(scores), R, n, ld, k, ptr(map), ld_map, ptr(idx_out), ld_out, ptr(comp_out),
                                  ptr(ws), ws_bytes, ptr(dev_status), _stream(stream)), "spatten_topk_select")


def gather_kept(src, src_batch, src_row, n_src, row_bytes, R, idx, ld_idx, k, dst, dst_batch, dst_row,
                compose_in=None, ld_compose=0, compose_out=None, check_index=0, dev_status=None, stream=None):
    check(lib.spatten_gather_kept(ptr(src), src_batch, src_row, n_src, row_bytes, R, ptr(idx), ld_idx, k, ptr(dst),
                                  dst_batch, dst_row, ptr(compose_in), ld_compose, ptr(compose_out), check_index,
                                  ptr(dev_status), _stream(stream)), "spatten_gather_kept")


def selftest_exp2_poly(x, y, n, stream=None):
    """y = 2^x by the attention kernels' FMA-pipe polynomial (diagnostic)."""
    check(lib.spatten_selftest_exp2_poly(ptr(x), ptr(y), n, _stream(stream)), "spatten_selftest_exp2_poly")


def kernel_launch_count() -> int:
    return int(lib.spatten_kernel_launch_count())


def set_wait_limit(polls: int) -> None:
    """Polls of one pipeline wait of the tensor-core kernels before they give up (0: default)."""
    lib.spatten_set_wait_limit(polls)


def cascade_workspace_size(cfg: cascade_cfg) -> int:
    return lib.spatten_cascade_workspace_size(C.byref(cfg))


def cascade_forward(cfg: cascade_cfg, weights, io: cascade_io, ws, ws_bytes: int, stream=None):
    """weights: sequence of (w_qkv, w_o) device tensors/pointers, one pair per layer."""
    arr = (layer_weights * cfg.L)(*[layer_weights(ptr(a), ptr(b)) for a, b in weights])
    check(lib.spatten_cascade_forward(C.byref(cfg), arr, C.byref(io), ptr(ws), ws_bytes, _stream(stream)),
          "spatten_cascade_forward")


def make_cfg(mode, B, T, D, H, d_h, L, dtype, token_keep, head_keep, quant, theta, sm_scale=0.0) -> cascade_cfg:
    c = cascade_cfg()
    c.mode, c.B, c.T, c.D, c.H, c.d_h, c.L, c.dtype = mode, B, T, D, H, d_h, L, dtype
    for l in range(L):
        c.token_keep[l] = token_keep[l]
        c.head_keep[l] = head_keep[l] if head_keep is not None else H
    c.quant, c.refetch_threshold, c.sm_scale = int(quant), float(theta), float(sm_scale)
    return c


# ---- prompts and the 4-bit cache --------------------------------------------------------------------
def _one_device(*tensors) -> int:
    """The GPU (-1: host memory) that all of a call's tensors are on."""
    on = {t.get_device() for t in tensors if t is not None}
    if len(on) > 1:
        raise ValueError("the tensors of a call are on one device")
    return on.pop() if on else -1


def _check_device(device, *tensors):
    """What a call is given besides its cache (tensors, or addresses, which are not looked at)."""
    for t in tensors:
        if t is not None and type(t) is not int and t.get_device() != device:
            raise ValueError("the tensors of a call are on one device")


def _rows_dtype(device, dtype, *tensors) -> int:
    """The dtype code of a call's row blocks, all on `device` (addresses are not looked at): the one they have, or
    the one given, of whose size their elements are."""
    code = dtype
    for t in tensors:
        if t is None or type(t) is int:
            continue
        if t.get_device() != device:
            raise ValueError("the tensors of a call are on one device")
        if dtype is not None:
            same = t.element_size() == (2 if dtype == BF16 else 4)
        else:
            same = code is None or code == dtype_code(t)
            code = dtype_code(t)
        if not same:
            raise TypeError("the rows of a call have one dtype")
    return code


_int32 = None   # torch.int32, set with the first cache (a lookup in `torch` costs 0.1 us a call)


def _vector(t, n, device):
    """Address of a vector of at least n counts, positions or offsets on `device` (None and addresses pass through)."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not _int32 or not t.is_contiguous():
        raise TypeError("counts, positions, offsets and status words are contiguous int32 vectors")
    if t.numel() < n:
        raise ValueError(f"a vector has {t.numel()} entries where the call reads {n}")
    if t.get_device() != device:
        raise ValueError("the tensors of a call are on one device")
    return t.data_ptr()


_get_device = None


def _run(fn, name, device, stream, *args):
    """One call on `device`, which becomes the current one meanwhile if it is not."""
    global _get_device
    if device < 0:
        raise ValueError(f"{name}: the tensors are not on a GPU")
    if _get_device is None:
        import torch
        torch.cuda.init()
        _get_device = torch._C._cuda_getDevice
    if device == _get_device():
        status = fn(*args, _stream(stream))
    else:
        import torch
        with torch.cuda.device(device):
            status = fn(*args, _stream(stream))
    if status != OK:
        raise SpattenError(status, name)


def make_prompt_args(q, k, v, o, cu_q, cu_kv=None, weight=None, sm_scale=0.0, dev_status=None,
                     kernel=ATTN_AUTO, weight_len=None) -> prompt_args:
    """Arguments of ``prompt_attention`` from torch tensors: q, o [rows, H, d_h] and k, v [rows, H_kv, d_h]
    (the heads of a row contiguous, the rows at any stride), cu_q, cu_kv int32 [B + 1], weight
    float32 [B, H_kv, n], weight_len int32 [B].  The tensors are kept alive by the result."""
    for t in (q, k, v, o):
        if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError("q, k, v and o are [rows, heads, d_h] with the heads of a row contiguous")
    if q.shape != o.shape or k.shape != v.shape or k.shape[2] != q.shape[2] or k.stride(0) != v.stride(0):
        raise ValueError("q and o, and k and v, have the same shapes, and k and v the same row stride")
    if not (q.dtype == k.dtype == v.dtype == o.dtype):
        raise TypeError("q, k, v and o have one dtype")
    a = prompt_args()
    a._device = _one_device(q, k, v, o, cu_q, cu_kv, weight, dev_status, weight_len)
    a.B, a.H, a.H_kv, a.d_h = _i32_vector(cu_q, "cu_q") - 1, q.shape[1], k.shape[1], q.shape[2]
    if cu_kv is not None and _i32_vector(cu_kv, "cu_kv") != a.B + 1:
        raise ValueError("cu_kv and cu_q have the same length")
    if weight_len is not None and _i32_vector(weight_len, "weight_len") != a.B:
        raise ValueError("weight_len has one entry per sequence")
    a.total_q, a.total_kv, a.cu_q, a.cu_kv, a.dtype = q.shape[0], k.shape[0], ptr(cu_q), ptr(cu_kv), dtype_code(q)
    a.q, a.q_ld_tok, a.k, a.v, a.kv_ld_tok = ptr(q), _row_stride(q), ptr(k), ptr(v), _row_stride(k)
    a.o, a.o_ld_tok, a.sm_scale, a.dev_status, a.kernel = ptr(o), _row_stride(o), sm_scale, ptr(dev_status), kernel
    a.weight_len = ptr(weight_len)
    if weight is not None:
        _dense_f32(weight, (a.B, a.H_kv), "weight")
        a.weight, a.weight_ld_seq, a.weight_ld_head, a.weight_cap = (
            ptr(weight), weight.stride(0), weight.stride(1), weight.shape[2])
    a._keep = (q, k, v, o, cu_q, cu_kv, weight, dev_status, weight_len)
    return a


def _row_stride(t) -> int:
    """Elements between rows; a block of at most one row has none of its own."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] * t.shape[2])


def _i32_vector(t, name) -> int:
    import torch
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} is a contiguous int32 vector")
    return t.shape[0]


def _dense_f32(t, lead, name):
    import torch
    if t.dtype != torch.float32 or t.dim() != 3 or tuple(t.shape[:2]) != tuple(lead) or t.stride(2) != 1:
        raise TypeError(f"{name} is float32 [{lead[0]}, {lead[1]}, n] with contiguous rows")


def prompt_workspace_size(args: prompt_args) -> int:
    return lib.spatten_prompt_workspace_size(C.byref(args))


def prompt_attention(args: prompt_args, ws=None, ws_bytes: int = 0, stream=None):
    _check_device(args._device, ws)
    _run(lib.spatten_prompt_attention, "spatten_prompt_attention", args._device, stream, C.byref(args), ptr(ws), ws_bytes)


def make_kv4_cache(k_codes, k_scale, v_codes, v_scale, weight=None, pos=None) -> kv4_cache:
    """The description of a 4-bit cache from its tensors: codes uint8 [B, H_kv, cap, d_h / 2], scales
    bfloat16 [B, H_kv, cap, d_h / 32], weight float32 and pos int32 [B, H_kv, cap] (all contiguous)."""
    global _int32
    import torch
    _int32 = torch.int32
    B, H, cap, half = k_codes.shape
    want = [(k_codes, torch.uint8, (half,)), (v_codes, torch.uint8, (half,)), (k_scale, torch.bfloat16, (half // 16,)),
            (v_scale, torch.bfloat16, (half // 16,)), (weight, torch.float32, ()), (pos, torch.int32, ())]
    for t, dt, tail in want:
        if t is not None and (t.dtype != dt or tuple(t.shape) != (B, H, cap) + tail or not t.is_contiguous()):
            raise TypeError(f"a cache tensor is not a contiguous {dt} {(B, H, cap) + tail}")
    c = kv4_cache(B, H, 2 * half, cap, ptr(k_codes), ptr(k_scale), ptr(v_codes), ptr(v_scale), ptr(weight), ptr(pos))
    c._keep = (k_codes, k_scale, v_codes, v_scale, weight, pos)
    c._device, c._ref = _one_device(*c._keep), C.byref(c)
    return c


_append_fn, _read_fn = lib.spatten_kv4_append, lib.spatten_kv4_read


def kv4_append(cache: kv4_cache, k, v, ld_tok, total, len, len_out, seen=None, seen_out=None, cu=None, dtype=None,
               dev_status=None, stream=None):
    device, B = cache._device, cache.B
    dt = _rows_dtype(device, dtype, k, v)
    _run(_append_fn, "spatten_kv4_append", device, stream, cache._ref, ptr(k), ptr(v), dt, ld_tok, total, _vector(cu, B + 1, device),
         _vector(len, B, device), _vector(len_out, B, device), _vector(seen, B, device), _vector(seen_out, B, device),
         _vector(dev_status, 1, device))


def kv4_read(cache: kv4_cache, cu, total, k_out, v_out, ld_tok, row0=None, dtype=None, dev_status=None, stream=None):
    device, B = cache._device, cache.B
    dt = _rows_dtype(device, dtype, k_out, v_out)
    _run(_read_fn, "spatten_kv4_read", device, stream, cache._ref, _vector(cu, B + 1, device), _vector(row0, B, device), total,
         ptr(k_out), ptr(v_out), dt, ld_tok, _vector(dev_status, 1, device))


def make_kv4_attn_args(cache: kv4_cache, q, o, len, n_max, update_weight=True, sm_scale=0.0,
                       dev_status=None) -> kv4_attn_args:
    """Arguments of ``kv4_attention``: q, o [B, H, d_h] (the heads of a row contiguous), len int32 [B]."""
    for t in (q, o):
        if t.dim() != 3 or tuple(t.shape) != (cache.B, q.shape[1], cache.d_h) or t.stride(2) != 1 or (
                t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError("q and o are [B, H, d_h] with the heads of a row contiguous")
    if q.dtype != o.dtype:
        raise TypeError("q and o have one dtype")
    if _i32_vector(len, "len") != cache.B:
        raise ValueError("len has one entry per sequence")
    a = kv4_attn_args()
    a.cache, a.H, a.q, a.dtype, a.q_ld = cache, q.shape[1], ptr(q), dtype_code(q), _row_stride(q)
    a.o, a.o_ld, a.len, a.n_max, a.sm_scale = ptr(o), _row_stride(o), ptr(len), n_max, sm_scale
    a.update_weight, a.dev_status = int(update_weight), ptr(dev_status)
    a._keep = (cache, q, o, len, dev_status)
    a._device = _one_device(cache._keep[0], q, o, len, dev_status)
    return a


def kv4_attention_workspace_size(args: kv4_attn_args) -> int:
    return lib.spatten_kv4_attention_workspace_size(C.byref(args))


def kv4_attention(args: kv4_attn_args, ws, ws_bytes: int, stream=None):
    _check_device(args._device, ws)
    _run(lib.spatten_kv4_attention, "spatten_kv4_attention", args._device, stream, C.byref(args), ptr(ws), ws_bytes)


def kv4_evict_workspace_size(cache: kv4_cache, n_max: int, keep: int) -> int:
    return lib.spatten_kv4_evict_workspace_size(C.byref(cache), n_max, keep)


def kv4_evict(src: kv4_cache, dst: kv4_cache, len, len_out, seen, n_max, keep, recent, ws, ws_bytes: int,
              dev_status=None, stream=None):
    device, B = src._device, src.B
    if dst._device != device:
        raise ValueError("the tensors of a call are on one device")
    _check_device(device, ws)
    _run(lib.spatten_kv4_evict, "spatten_kv4_evict", device, stream, src._ref, dst._ref, _vector(len, B, device),
         _vector(len_out, B, device), _vector(seen, B, device), n_max, keep, recent, ptr(ws), ws_bytes, _vector(dev_status, 1, device))
