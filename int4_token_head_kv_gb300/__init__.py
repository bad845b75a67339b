"""INT4 per-(token, head) KV cache for NVIDIA GB300: Python binding of the C ABI in include/kv_int4.h.

The functions below have the C entry points' names.  They only marshal arguments: check that the
torch tensors are CUDA, contiguous and of the right dtype and shape, then pass raw device pointers
and the current CUDA stream to ``libkv_int4.so``.  Every step of the write and of the attention
runs in that library's kernels; there is no fallback: the first call (or ``load()``) raises
ImportError when the library has not been built (``python int4_token_head_kv_gb300/_build.py``).
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libkv_int4.so")

KV_INT4_F16, KV_INT4_BF16, KV_INT4_F32 = 0, 1, 2
STAT_NAMES = ["slot_out_of_range", "block_out_of_range", "bad_sequence", "wait_timeout", "bad_sign",
              "position_out_of_range"]
_STAT_COUNT = 8
_DTYPES = {torch.float16: KV_INT4_F16, torch.bfloat16: KV_INT4_BF16, torch.float32: KV_INT4_F32}


class AttnOptions(ctypes.Structure):
    """kv_int4_attn_options: window_left (< 0: none), softcap (0: none), alibi_slopes (device
    pointer to fp32 [num_q_heads], or None), qq_bias (device pointer to fp32 rows of
    qq_bias_stride elements, or None)."""
    _fields_ = [("window_left", ctypes.c_int32), ("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("qq_bias", ctypes.c_void_p), ("qq_bias_stride", ctypes.c_int32)]


class KVInt4Error(RuntimeError):
    """A non-OK status returned by the C library."""

    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {message} (status {status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m int4_token_head_kv_gb300._build` "
                          "(the CUDA library is required; there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, szt = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.kv_int4_row_bytes.argtypes = [i32]
    lib.kv_int4_row_bytes.restype = i32
    lib.kv_int4_status_string.argtypes = [ctypes.c_int]
    lib.kv_int4_status_string.restype = ctypes.c_char_p
    lib.kv_int4_write.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, vp, vp, vp, i64, i32, vp]
    lib.kv_int4_write.restype = ctypes.c_int
    lib.kv_int8_row_bytes.argtypes = [i32]
    lib.kv_int8_row_bytes.restype = i32
    lib.kv_int8_write.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, vp, vp, i64, i32, vp]
    lib.kv_int8_write.restype = ctypes.c_int
    lib.kv_int2_row_bytes.argtypes = [i32]
    lib.kv_int2_row_bytes.restype = i32
    lib.kv_int2_write.argtypes = lib.kv_int4_write.argtypes
    lib.kv_int2_write.restype = ctypes.c_int
    lib.kv_int4_rope_write.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, vp, i64, i32, i32,
                                       vp, vp, vp, i64, vp, i64, i32, vp]
    lib.kv_int4_rope_write.restype = ctypes.c_int
    lib.kv_int8_rope_write.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, vp, i64, i32, i32,
                                       vp, vp, i64, vp, i64, i32, vp]
    lib.kv_int8_rope_write.restype = ctypes.c_int
    lib.kv_int2_rope_write.argtypes = lib.kv_int4_rope_write.argtypes
    lib.kv_int2_rope_write.restype = ctypes.c_int
    for name, signs in (("kv_int4_mrope_write", [vp]), ("kv_int8_mrope_write", []), ("kv_int2_mrope_write", [vp])):
        f = getattr(lib, name)
        f.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, i32, ctypes.c_char_p, vp, i64, i32,
                      i32, vp] + signs + [vp, i64, vp, i64, i32, vp]
        f.restype = ctypes.c_int
    lib.kv_int4_read.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, vp, vp, ctypes.c_int, vp]
    lib.kv_int4_read.restype = ctypes.c_int
    lib.kv_int8_read.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, vp, ctypes.c_int, vp]
    lib.kv_int8_read.restype = ctypes.c_int
    lib.kv_int2_read.argtypes = lib.kv_int4_read.argtypes
    lib.kv_int2_read.restype = ctypes.c_int
    lib.kv_int4_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.kv_int4_attention_workspace_bytes.restype = szt
    lib.kv_int4_attention_segment_len.argtypes = [i32, i32, i32]
    lib.kv_int4_attention_segment_len.restype = i32
    lib.kv_int4_paged_attention.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, vp,
                                            i32, i32, i32, f32, vp, i32, vp, ctypes.c_int, vp, szt, vp]
    lib.kv_int4_paged_attention.restype = ctypes.c_int
    lib.kv_int4_paged_attention_noalloc.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp,
                                                    vp, i32, i32, i32, f32, vp, i32, vp, ctypes.c_int, vp]
    lib.kv_int4_paged_attention_noalloc.restype = ctypes.c_int
    lib.kv_int4_paged_attention_noalloc_ex.argtypes = lib.kv_int4_paged_attention_noalloc.argtypes + [
        ctypes.POINTER(AttnOptions)]
    lib.kv_int4_paged_attention_noalloc_ex.restype = ctypes.c_int
    lib.kv_int4_paged_attention_ex.argtypes = lib.kv_int4_paged_attention.argtypes + [ctypes.POINTER(AttnOptions)]
    lib.kv_int4_paged_attention_ex.restype = ctypes.c_int
    lib.kv_int8_paged_attention.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, vp,
                                            i32, i32, i32, f32, i32, vp, ctypes.c_int, vp, szt, vp]
    lib.kv_int8_paged_attention.restype = ctypes.c_int
    lib.kv_int2_paged_attention.argtypes = lib.kv_int4_paged_attention.argtypes
    lib.kv_int2_paged_attention.restype = ctypes.c_int
    lib.kv_int4_shared_prefix_attention.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, i32,
                                                    vp, vp, i32, i32, i32, f32, vp, i32, vp, ctypes.c_int, vp, szt, vp,
                                                    ctypes.POINTER(AttnOptions)]
    lib.kv_int4_shared_prefix_attention.restype = ctypes.c_int
    lib.kv_int4_shared_prefix_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    lib.kv_int4_shared_prefix_workspace_bytes.restype = szt
    for name, signs in (("kv_int4_span_attention", [vp]), ("kv_int8_span_attention", []), ("kv_int2_span_attention", [vp])):
        f = getattr(lib, name)
        f.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, vp, i32, i32, i32, f32] + signs + [
            vp, vp, f32, vp, vp, ctypes.c_int, vp, szt, vp]
        f.restype = ctypes.c_int
    lib.kv_int4_span_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32, i32]
    lib.kv_int4_span_workspace_bytes.restype = szt
    lib.kv_int4_read_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
    lib.kv_int4_read_device_status.restype = ctypes.c_int
    lib.kv_int4_clear_device_status.argtypes = [vp]
    lib.kv_int4_clear_device_status.restype = ctypes.c_int
    lib.kv_int4_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.kv_int4_selftest_wait_timeout.restype = ctypes.c_int
    return lib


_lib = None


def load():
    """Load libkv_int4.so (once); raises ImportError when it has not been built."""
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise KVInt4Error(fn, status, load().kv_int4_status_string(status).decode())


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _one_device(*tensors) -> torch.device:
    """The device all the given CUDA tensors (None entries skipped) are on; the library launches on the
    current device, so the calls below make it this one."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"all tensors must be on one CUDA device, got {sorted(map(str, devs))}")
    return devs.pop()


def _cuda(t: torch.Tensor, name: str, dtypes=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t


def kv_int4_row_bytes(head_size: int) -> int:
    return int(load().kv_int4_row_bytes(head_size))


def kv_int4_cache_shape(num_blocks: int, block_size: int, num_kv_heads: int, head_size: int):
    """Shape of the packed cache: (num_blocks, 2, block_size, num_kv_heads, head_size/2 + 4) uint8."""
    return (num_blocks, 2, block_size, num_kv_heads, kv_int4_row_bytes(head_size))


def kv_int4_write(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor, rht_signs: torch.Tensor,
                  kv_cache: torch.Tensor, stream=None) -> None:
    """Rotate, quantise and pack ``key``/``value`` [T, H, d] into ``kv_cache`` at ``slot_mapping``."""
    _rotated_write("kv_int4_write", kv_int4_row_bytes, key, value, slot_mapping, rht_signs, kv_cache, stream)


def _rotated_write(fn, row_bytes, key, value, slot_mapping, rht_signs, kv_cache, stream):
    _cuda(key, "key", (torch.float16, torch.bfloat16))
    _cuda(value, "value", (key.dtype,))
    _cuda(slot_mapping, "slot_mapping", (torch.int64,))
    _cuda(rht_signs, "rht_signs", (torch.float32,))
    _cuda(kv_cache, "kv_cache", (torch.uint8,))
    if key.dim() != 3 or value.shape != key.shape:
        raise ValueError("key and value must both be [num_tokens, num_kv_heads, head_size]")
    T, H, d = key.shape
    if slot_mapping.shape != (T,) or rht_signs.shape != (d,):
        raise ValueError("slot_mapping must be [num_tokens] and rht_signs [head_size]")
    if kv_cache.dim() != 5 or kv_cache.shape[1] != 2 or kv_cache.shape[3] != H or \
            kv_cache.shape[4] != row_bytes(d):
        raise ValueError(f"kv_cache must be (NB, 2, bs, {H}, {row_bytes(d)})")
    with torch.cuda.device(_one_device(key, value, slot_mapping, rht_signs, kv_cache)):
        st = getattr(load(), fn)(key.data_ptr(), value.data_ptr(), _DTYPES[key.dtype], T, H, d,
                                 slot_mapping.data_ptr(), rht_signs.data_ptr(), kv_cache.data_ptr(), kv_cache.shape[0],
                                 kv_cache.shape[2], _stream(stream))
    _check(fn, st)


def kv_int8_row_bytes(head_size: int) -> int:
    return int(load().kv_int8_row_bytes(head_size))


def kv_int8_cache_shape(num_blocks: int, block_size: int, num_kv_heads: int, head_size: int):
    """INT8 per-(token, head) comparator cache: (num_blocks, 2, block_size, H, head_size + 4) uint8."""
    return (num_blocks, 2, block_size, num_kv_heads, kv_int8_row_bytes(head_size))


def kv_int8_write(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor, kv_cache: torch.Tensor,
                  stream=None) -> None:
    """Quantise ``key``/``value`` [T, H, d] to INT8 per-(token, head) rows of ``kv_cache`` at ``slot_mapping``."""
    _cuda(key, "key", (torch.float16, torch.bfloat16))
    _cuda(value, "value", (key.dtype,))
    _cuda(slot_mapping, "slot_mapping", (torch.int64,))
    _cuda(kv_cache, "kv_cache", (torch.uint8,))
    if key.dim() != 3 or value.shape != key.shape:
        raise ValueError("key and value must both be [num_tokens, num_kv_heads, head_size]")
    T, H, d = key.shape
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    if kv_cache.dim() != 5 or kv_cache.shape[1] != 2 or kv_cache.shape[3] != H or \
            kv_cache.shape[4] != kv_int8_row_bytes(d):
        raise ValueError(f"kv_cache must be {kv_int8_cache_shape('NB', 'bs', H, d)}")
    with torch.cuda.device(_one_device(key, value, slot_mapping, kv_cache)):
        st = load().kv_int8_write(key.data_ptr(), value.data_ptr(), _DTYPES[key.dtype], T, H, d,
                                  slot_mapping.data_ptr(), kv_cache.data_ptr(), kv_cache.shape[0], kv_cache.shape[2],
                                  _stream(stream))
    _check("kv_int8_write", st)


def kv_int2_row_bytes(head_size: int) -> int:
    return int(load().kv_int2_row_bytes(head_size))


def kv_int2_cache_shape(num_blocks: int, block_size: int, num_kv_heads: int, head_size: int):
    """INT2 Lloyd-Max cache: (num_blocks, 2, block_size, H, head_size/4 + 4) uint8."""
    return (num_blocks, 2, block_size, num_kv_heads, kv_int2_row_bytes(head_size))


def kv_int2_write(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor, rht_signs: torch.Tensor,
                  kv_cache: torch.Tensor, stream=None) -> None:
    """Rotate ``key``/``value`` [T, H, d] as kv_int4_write does, quantise them to INT2 Lloyd-Max codes
    and pack them into ``kv_cache`` at ``slot_mapping``."""
    _rotated_write("kv_int2_write", kv_int2_row_bytes, key, value, slot_mapping, rht_signs, kv_cache, stream)


# The serving calls below run once per layer and step, where a Python call of 25 us would be most of a small
# step: they ask for the stream by its raw handle, enter a device only when it is not the current one, and
# size rows without a call into the library (the framework's own calls above cost what they did).
try:
    _raw_stream = torch._C._cuda_getCurrentRawStream   # what torch.cuda.current_stream(device).cuda_stream holds
except AttributeError:
    def _raw_stream(device: int) -> int:
        return torch.cuda.current_stream(device).cuda_stream


def _current(stream, tensor: torch.Tensor):
    """A context with ``stream`` (a torch stream, or a raw handle on the tensor's device) as the current one.
    The serving calls run whole inside it, so that what they allocate belongs to the stream that uses it:
    memory from another stream's pool could be in use there, or be handed out again while this one runs."""
    if not isinstance(tensor, torch.Tensor) or not tensor.is_cuda:
        raise ValueError("the call's tensors must be CUDA tensors")
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = (torch.cuda.ExternalStream(handle, device=tensor.device) if handle else
                  torch.cuda.default_stream(tensor.device))
    elif stream.device != tensor.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {tensor.device}")
    return torch.cuda.stream(stream)


def _checked(t, name: str, dtypes):
    """_cuda for the serving calls: the tests alone while nothing is wrong."""
    if type(t) is torch.Tensor and t.dtype in dtypes and t.is_cuda and t.is_contiguous():
        return t
    return _cuda(t, name, dtypes)


def _call(fn: str, tensors, tail, *args) -> None:
    """Call the library's ``fn`` with ``args``, the current stream and ``tail`` (a tuple) on the device that
    all ``tensors`` (None entries skipped) are on."""
    dev = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if dev >= 0:
                    _one_device(*tensors)   # raises
                dev = i
    stream = _raw_stream(dev)
    f = getattr(_lib or load(), fn)
    if dev == torch.cuda.current_device():
        st = f(*args, stream, *tail)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream, *tail)
    if st != 0:
        _check(fn, st)


def _token_rows(t: torch.Tensor, name: str, dtypes):
    """Shape and token stride of a CUDA tensor [tokens, heads, head_size] whose tokens' rows are contiguous,
    with any stride between them."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or stride[2] != 1 or (stride[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must be [num_tokens, num_heads, head_size] with each token's heads contiguous")
    return shape, stride[0]


_HALF_TYPES = (torch.float16, torch.bfloat16)
_I64, _F32, _U8, _I32 = (torch.int64,), (torch.float32,), (torch.uint8,), (torch.int32,)


@functools.lru_cache(maxsize=256)
def _axes_of(counts: tuple, mixed: bool) -> bytes:
    """_pair_axes for a tuple of plain integers."""
    if not mixed:
        return bytes(a for a, n in enumerate(counts) for _ in range(n))
    turns = range(max(counts))
    return bytes(a for i in turns for a, n in enumerate(counts) if i < n)


def _pair_axes(sections, mixed: bool) -> bytes:
    """The axis of every rotated pair, one byte each: the sections one after another, or dealt out in turn while
    they last when ``mixed``.  Integers of any type; what is refused does not depend on what was asked before."""
    try:
        counts = tuple(operator.index(n) for n in sections)
    except TypeError:
        counts = ()
    if not 1 <= len(counts) <= 4 or min(counts) < 0 or sum(counts) > 1024:
        raise ValueError("sections must be one to four counts of pairs, one for each axis")
    return _axes_of(counts, mixed)


def _rope_write(fn, bits, query, key, value, positions, cos_sin, slot_mapping, rht_signs, kv_cache, query_out,
                interleaved, stream, sections=None, mixed=False):
    if stream is not None:
        with _current(stream, key):
            return _rope_write(fn, bits, query, key, value, positions, cos_sin, slot_mapping, rht_signs, kv_cache,
                               query_out, interleaved, None, sections, mixed)
    kshape, kst = _token_rows(key, "key", _HALF_TYPES)
    dtype = key.dtype
    vshape, vst = _token_rows(value, "value", (dtype,))
    _checked(positions, "positions", _I64)
    _checked(cos_sin, "cos_sin", _F32)
    _checked(slot_mapping, "slot_mapping", _I64)
    _checked(kv_cache, "kv_cache", _U8)
    if vshape != kshape:
        raise ValueError("key and value must both be [num_tokens, num_kv_heads, head_size]")
    T, H, d = kshape
    signs = ()
    if bits != 8:
        _checked(rht_signs, "rht_signs", _F32)
        if rht_signs.shape != (d,):
            raise ValueError("rht_signs must be [head_size]")
        signs = (rht_signs.data_ptr(),)
    table = cos_sin.shape
    if len(table) != 2:
        raise ValueError("cos_sin must be [max_position, rot_dim]")
    axes = ()
    if sections is None:
        if slot_mapping.shape != (T,) or positions.shape != (T,):
            raise ValueError("positions and slot_mapping must be [num_tokens]")
    else:
        pairs = _pair_axes(sections, bool(mixed))
        if 2 * len(pairs) != table[1]:
            raise ValueError("the sections must sum to rot_dim / 2 pairs")
        if slot_mapping.shape != (T,) or positions.shape != (len(sections), T):
            raise ValueError("positions must be [num_axes, num_tokens], one row for each section, and slot_mapping [num_tokens]")
        axes = (len(sections), pairs)
    cshape, rb = kv_cache.shape, d * bits // 8 + 4
    if len(cshape) != 5 or cshape[1] != 2 or cshape[3] != H or cshape[4] != rb:
        raise ValueError(f"kv_cache must be (NB, 2, bs, {H}, {rb})")
    Hq = qst = qost = 0
    qptr = qoptr = None
    if query is not None:
        qshape, qst = _token_rows(query, "query", (dtype,))
        if qshape[0] != T or qshape[2] != d:
            raise ValueError("query must be [num_tokens, num_q_heads, head_size]")
        Hq = qshape[1]
        if query_out is None:
            query_out = torch.empty(qshape, dtype=dtype, device=query.device)
            qost = Hq * d
        else:
            oshape, qost = _token_rows(query_out, "query_out", (dtype,))
            if oshape != qshape:
                raise ValueError("query_out must have the query's shape")
        qptr, qoptr = query.data_ptr(), query_out.data_ptr()
    elif query_out is not None:
        raise ValueError("query_out needs a query")
    _call(fn, (query, key, value, positions, cos_sin, slot_mapping, rht_signs, kv_cache, query_out), (),
          qptr, qst, Hq, key.data_ptr(), kst, value.data_ptr(), vst, _DTYPES[dtype], T, H, d, positions.data_ptr(),
          *axes, cos_sin.data_ptr(), table[0], table[1], 1 if interleaved else 0, slot_mapping.data_ptr(), *signs, qoptr, qost,
          kv_cache.data_ptr(), cshape[0], cshape[2])
    return query_out


def kv_int4_rope_write(query, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                       slot_mapping: torch.Tensor, rht_signs: torch.Tensor, kv_cache: torch.Tensor, query_out=None,
                       interleaved: bool = False, stream=None):
    """kv_int4_write with the rotary position embedding applied on the way: ``query`` [T, Hq, d] (or None)
    and ``key`` [T, H, d] are rotated by the rows ``cos_sin[positions]`` (fp32 [max_position, rot_dim]:
    rot_dim / 2 cosines, then as many sines; halves paired, or neighbours when ``interleaved``), the keys
    and values go into ``kv_cache`` at ``slot_mapping``, and the rotated queries are returned
    (``query_out``, which may be ``query`` itself).  Query, key, value and query_out may have any stride
    between tokens, as the slices of a fused projection do.  A token whose position is outside the table
    is skipped: its ``query_out`` row is left as it was."""
    return _rope_write("kv_int4_rope_write", 4, query, key, value, positions, cos_sin, slot_mapping,
                       rht_signs, kv_cache, query_out, interleaved, stream)


def kv_int8_rope_write(query, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                       slot_mapping: torch.Tensor, kv_cache: torch.Tensor, query_out=None, interleaved: bool = False,
                       stream=None):
    """kv_int4_rope_write into the INT8 comparator's cache (no signs)."""
    return _rope_write("kv_int8_rope_write", 8, query, key, value, positions, cos_sin, slot_mapping,
                       None, kv_cache, query_out, interleaved, stream)


def kv_int2_rope_write(query, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                       slot_mapping: torch.Tensor, rht_signs: torch.Tensor, kv_cache: torch.Tensor, query_out=None,
                       interleaved: bool = False, stream=None):
    """kv_int4_rope_write into the INT2 Lloyd-Max cache."""
    return _rope_write("kv_int2_rope_write", 2, query, key, value, positions, cos_sin, slot_mapping,
                       rht_signs, kv_cache, query_out, interleaved, stream)


def kv_int4_mrope_write(query, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                        sections, slot_mapping: torch.Tensor, rht_signs: torch.Tensor, kv_cache: torch.Tensor,
                        query_out=None, interleaved: bool = False, mixed_sections: bool = False, stream=None):
    """kv_int4_rope_write with positions on several axes (time, height, width): ``positions`` is int64 [axes, T] and
    ``sections`` the number of rotated pairs of each axis (one to four axes, summing to rot_dim / 2).  The axes'
    pairs follow one another, or are dealt out in turn while they last when ``mixed_sections`` (sections (3, 2, 2):
    axes 0 1 2 0 1 2 0).  Pair i takes column i of its own axis's row ``cos_sin[positions[axis]]``."""
    return _rope_write("kv_int4_mrope_write", 4, query, key, value, positions, cos_sin, slot_mapping, rht_signs, kv_cache,
                       query_out, interleaved, stream, sections, mixed_sections)


def kv_int8_mrope_write(query, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                        sections, slot_mapping: torch.Tensor, kv_cache: torch.Tensor, query_out=None,
                        interleaved: bool = False, mixed_sections: bool = False, stream=None):
    """kv_int4_mrope_write into the INT8 comparator's cache (no signs)."""
    return _rope_write("kv_int8_mrope_write", 8, query, key, value, positions, cos_sin, slot_mapping, None, kv_cache,
                       query_out, interleaved, stream, sections, mixed_sections)


def kv_int2_mrope_write(query, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                        sections, slot_mapping: torch.Tensor, rht_signs: torch.Tensor, kv_cache: torch.Tensor,
                        query_out=None, interleaved: bool = False, mixed_sections: bool = False, stream=None):
    """kv_int4_mrope_write into the INT2 Lloyd-Max cache."""
    return _rope_write("kv_int2_mrope_write", 2, query, key, value, positions, cos_sin, slot_mapping, rht_signs, kv_cache,
                       query_out, interleaved, stream, sections, mixed_sections)


def _read(fn, bits, kv_cache, slot_mapping, rht_signs, dtype, key_out, value_out, stream):
    if stream is not None:
        with _current(stream, kv_cache):
            return _read(fn, bits, kv_cache, slot_mapping, rht_signs, dtype, key_out, value_out, None)
    _checked(kv_cache, "kv_cache", _U8)
    _checked(slot_mapping, "slot_mapping", _I64)
    sshape, cshape = slot_mapping.shape, kv_cache.shape
    if len(sshape) != 1:
        raise ValueError("slot_mapping must be [num_tokens]")
    d = (cshape[-1] - 4) * 8 // bits if len(cshape) == 5 and cshape[1] == 2 else 0
    if d not in (64, 128) or d * bits // 8 + 4 != cshape[4]:
        raise ValueError(f"kv_cache must be (NB, 2, bs, H, row bytes) with rows of {8 * bits + 4} or {16 * bits + 4} bytes")
    T, H = sshape[0], cshape[3]
    signs = ()
    if bits != 8:
        _checked(rht_signs, "rht_signs", _F32)
        if rht_signs.shape != (d,):
            raise ValueError("rht_signs must be [head_size]")
        signs = (rht_signs.data_ptr(),)
    shape = (T, H, d)
    if key_out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype}, expected one of {tuple(_DTYPES)}")
        key_out = torch.empty(shape, dtype=dtype, device=kv_cache.device)
    else:
        _checked(key_out, "key_out", tuple(_DTYPES))
    if value_out is None:
        value_out = torch.empty(shape, dtype=key_out.dtype, device=kv_cache.device)
    else:
        _checked(value_out, "value_out", (key_out.dtype,))
    if key_out.shape != shape or value_out.shape != shape:
        raise ValueError(f"key_out and value_out must be [num_tokens, {H}, {d}]")
    _call(fn, (kv_cache, slot_mapping, rht_signs, key_out, value_out), (), kv_cache.data_ptr(), cshape[0],
          cshape[2], H, d, slot_mapping.data_ptr(), T, *signs, key_out.data_ptr(), value_out.data_ptr(), _DTYPES[key_out.dtype])
    return key_out, value_out


def kv_int4_read(kv_cache: torch.Tensor, slot_mapping: torch.Tensor, rht_signs: torch.Tensor, dtype=torch.bfloat16,
                 key_out=None, value_out=None, stream=None):
    """The keys and values [T, H, d] (``dtype``: fp16, bf16 or fp32, or that of ``key_out``) that the cached
    rows at ``slot_mapping`` stand for; negative slots give rows of zeros."""
    return _read("kv_int4_read", 4, kv_cache, slot_mapping, rht_signs, dtype, key_out, value_out, stream)


def kv_int8_read(kv_cache: torch.Tensor, slot_mapping: torch.Tensor, dtype=torch.bfloat16, key_out=None, value_out=None,
                 stream=None):
    """kv_int4_read for the INT8 comparator's cache (no signs)."""
    return _read("kv_int8_read", 8, kv_cache, slot_mapping, None, dtype, key_out, value_out, stream)


def kv_int2_read(kv_cache: torch.Tensor, slot_mapping: torch.Tensor, rht_signs: torch.Tensor, dtype=torch.bfloat16,
                 key_out=None, value_out=None, stream=None):
    """kv_int4_read for the INT2 Lloyd-Max cache."""
    return _read("kv_int2_read", 2, kv_cache, slot_mapping, rht_signs, dtype, key_out, value_out, stream)


def kv_int4_attention_segment_len(num_seqs: int, max_seq_len: int, segment_len: int = 0) -> int:
    return int(load().kv_int4_attention_segment_len(num_seqs, max_seq_len, segment_len))


def kv_int4_attention_workspace_bytes(num_q_heads: int, num_kv_heads: int, head_size: int, num_seqs: int,
                                      max_seq_len: int, segment_len: int = 0) -> int:
    return int(load().kv_int4_attention_workspace_bytes(num_q_heads, num_kv_heads, head_size, num_seqs,
                                                      max_seq_len, segment_len))


def _options(Hq, max_query_len, window_left, softcap, alibi_slopes, qq_bias):
    """kv_int4_attn_options for the given keywords, or None when none is set."""
    if window_left < 0 and softcap == 0.0 and alibi_slopes is None and qq_bias is None:
        return None
    if alibi_slopes is not None:
        _cuda(alibi_slopes, "alibi_slopes", (torch.float32,))
        if alibi_slopes.shape != (Hq,):
            raise ValueError("alibi_slopes must be [num_q_heads]")
    if qq_bias is not None:
        _cuda(qq_bias, "qq_bias", (torch.float32,))
        if qq_bias.dim() != 2 or qq_bias.stride(1) != 1 or qq_bias.shape[0] < max_query_len:
            raise ValueError("qq_bias must be a row-contiguous [rows >= max_query_len, cols] matrix")
    return AttnOptions(int(window_left), float(softcap),
                       alibi_slopes.data_ptr() if alibi_slopes is not None else None,
                       qq_bias.data_ptr() if qq_bias is not None else None,
                       int(qq_bias.stride(0)) if qq_bias is not None else 0)


def kv_int4_paged_attention(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                            seq_lens: torch.Tensor, query_start_loc: torch.Tensor, softmax_scale: float,
                            rht_signs: torch.Tensor, max_query_len: int, max_seq_len: int, out=None,
                            out_dtype=None, segment_len: int = 0, workspace=None, stream=None,
                            window_left: int = -1, softcap: float = 0.0, alibi_slopes=None,
                            qq_bias=None) -> torch.Tensor:
    """Causal paged attention of ``query`` [Nq, Hq, d] over the INT4 cache; returns ``out``.  With
    ``window_left >= 0``, ``softcap > 0``, ``alibi_slopes`` (fp32 [Hq] on the device) or ``qq_bias``
    (fp32 [rows >= max_query_len, stride >= max_query_len] on the device, contiguous rows) the call
    goes through kv_int4_paged_attention_ex."""
    _cuda(query, "query", (torch.float16, torch.bfloat16))
    _cuda(kv_cache, "kv_cache", (torch.uint8,))
    _cuda(block_tables, "block_tables", (torch.int32,))
    _cuda(seq_lens, "seq_lens", (torch.int32,))
    _cuda(query_start_loc, "query_start_loc", (torch.int32,))
    _cuda(rht_signs, "rht_signs", (torch.float32,))
    Nq, Hq, d = query.shape
    NB, two, bs, H, rb = kv_cache.shape
    S = seq_lens.shape[0]
    if two != 2 or rb != kv_int4_row_bytes(d) or rht_signs.shape != (d,):
        raise ValueError("kv_cache / rht_signs do not match the query's head size")
    if query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    if out is None:
        out = torch.empty((Nq, Hq, d), dtype=out_dtype or query.dtype, device=query.device)
    _cuda(out, "out", tuple(_DTYPES))
    if out.shape != query.shape:
        raise ValueError("out must have the query's shape")
    need = kv_int4_attention_workspace_bytes(Hq, H, d, S, max_seq_len, segment_len)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    opts = _options(Hq, max_query_len, window_left, softcap, alibi_slopes, qq_bias)
    with torch.cuda.device(_one_device(query, kv_cache, block_tables, seq_lens, query_start_loc, rht_signs, out,
                                       workspace, alibi_slopes, qq_bias)):
        args = (query.data_ptr(), _DTYPES[query.dtype], Nq, Hq, kv_cache.data_ptr(), NB, H, d, bs,
                block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), S,
                max_query_len, max_seq_len, float(softmax_scale), rht_signs.data_ptr(), segment_len, out.data_ptr(),
                _DTYPES[out.dtype], ws_ptr, ws_bytes, _stream(stream))
        if opts is not None:
            st, fn = load().kv_int4_paged_attention_ex(*args, ctypes.byref(opts)), "kv_int4_paged_attention_ex"
        else:
            st, fn = load().kv_int4_paged_attention(*args), "kv_int4_paged_attention"
    _check(fn, st)
    return out


def kv_int4_paged_attention_noalloc(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                                    seq_lens: torch.Tensor, query_start_loc: torch.Tensor, softmax_scale: float,
                                    rht_signs: torch.Tensor, max_query_len: int, max_seq_len: int, out=None,
                                    out_dtype=None, segment_len: int = 0, stream=None, window_left: int = -1,
                                    softcap: float = 0.0, alibi_slopes=None, qq_bias=None) -> torch.Tensor:
    """kv_int4_paged_attention without a workspace: the split-KV partials live in the library's fixed
    device scratch array (calls that overlap on the GPU must be serialised).  ``out`` is allocated
    here when not given; pass it to keep the call free of allocations.  The options as for
    kv_int4_paged_attention (through kv_int4_paged_attention_noalloc_ex)."""
    _cuda(query, "query", (torch.float16, torch.bfloat16))
    _cuda(kv_cache, "kv_cache", (torch.uint8,))
    _cuda(block_tables, "block_tables", (torch.int32,))
    _cuda(seq_lens, "seq_lens", (torch.int32,))
    _cuda(query_start_loc, "query_start_loc", (torch.int32,))
    _cuda(rht_signs, "rht_signs", (torch.float32,))
    Nq, Hq, d = query.shape
    NB, two, bs, H, rb = kv_cache.shape
    S = seq_lens.shape[0]
    if two != 2 or rb != kv_int4_row_bytes(d) or rht_signs.shape != (d,):
        raise ValueError("kv_cache / rht_signs do not match the query's head size")
    if query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    if out is None:
        out = torch.empty((Nq, Hq, d), dtype=out_dtype or query.dtype, device=query.device)
    _cuda(out, "out", tuple(_DTYPES))
    if out.shape != query.shape:
        raise ValueError("out must have the query's shape")
    opts = _options(Hq, max_query_len, window_left, softcap, alibi_slopes, qq_bias)
    with torch.cuda.device(_one_device(query, kv_cache, block_tables, seq_lens, query_start_loc, rht_signs, out,
                                       alibi_slopes, qq_bias)):
        args = (query.data_ptr(), _DTYPES[query.dtype], Nq, Hq, kv_cache.data_ptr(), NB, H, d, bs,
                block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), S,
                max_query_len, max_seq_len, float(softmax_scale), rht_signs.data_ptr(), segment_len, out.data_ptr(),
                _DTYPES[out.dtype], _stream(stream))
        if opts is None:
            st, fn = load().kv_int4_paged_attention_noalloc(*args), "kv_int4_paged_attention_noalloc"
        else:
            st, fn = (load().kv_int4_paged_attention_noalloc_ex(*args, ctypes.byref(opts)),
                      "kv_int4_paged_attention_noalloc_ex")
    _check(fn, st)
    return out


def kv_int8_paged_attention(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                            seq_lens: torch.Tensor, query_start_loc: torch.Tensor, softmax_scale: float,
                            max_query_len: int, max_seq_len: int, out=None, out_dtype=None, segment_len: int = 0,
                            workspace=None, stream=None) -> torch.Tensor:
    """Decode attention of ``query`` [Nq, Hq, d] (one query token per sequence) over the INT8
    comparator's cache; returns ``out``.  The workspace size is the INT4 call's."""
    _cuda(query, "query", (torch.float16, torch.bfloat16))
    _cuda(kv_cache, "kv_cache", (torch.uint8,))
    _cuda(block_tables, "block_tables", (torch.int32,))
    _cuda(seq_lens, "seq_lens", (torch.int32,))
    _cuda(query_start_loc, "query_start_loc", (torch.int32,))
    Nq, Hq, d = query.shape
    NB, two, bs, H, rb = kv_cache.shape
    S = seq_lens.shape[0]
    if two != 2 or rb != kv_int8_row_bytes(d):
        raise ValueError("kv_cache does not match the query's head size")
    if query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    if out is None:
        out = torch.empty((Nq, Hq, d), dtype=out_dtype or query.dtype, device=query.device)
    _cuda(out, "out", tuple(_DTYPES))
    if out.shape != query.shape:
        raise ValueError("out must have the query's shape")
    need = kv_int4_attention_workspace_bytes(Hq, H, d, S, max_seq_len, segment_len)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with torch.cuda.device(_one_device(query, kv_cache, block_tables, seq_lens, query_start_loc, out, workspace)):
        st = load().kv_int8_paged_attention(query.data_ptr(), _DTYPES[query.dtype], Nq, Hq, kv_cache.data_ptr(), NB,
                                          H, d, bs, block_tables.data_ptr(), block_tables.shape[1],
                                          seq_lens.data_ptr(), query_start_loc.data_ptr(), S, max_query_len,
                                          max_seq_len, float(softmax_scale), segment_len, out.data_ptr(),
                                          _DTYPES[out.dtype], ws_ptr, ws_bytes, _stream(stream))
    _check("kv_int8_paged_attention", st)
    return out


def kv_int2_paged_attention(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                            seq_lens: torch.Tensor, query_start_loc: torch.Tensor, softmax_scale: float,
                            rht_signs: torch.Tensor, max_query_len: int, max_seq_len: int, out=None,
                            out_dtype=None, segment_len: int = 0, workspace=None, stream=None) -> torch.Tensor:
    """Decode attention of ``query`` [Nq, Hq, d] (one query token per sequence) over the INT2
    Lloyd-Max cache; returns ``out``.  The workspace size is the INT4 call's."""
    _cuda(query, "query", (torch.float16, torch.bfloat16))
    _cuda(kv_cache, "kv_cache", (torch.uint8,))
    _cuda(block_tables, "block_tables", (torch.int32,))
    _cuda(seq_lens, "seq_lens", (torch.int32,))
    _cuda(query_start_loc, "query_start_loc", (torch.int32,))
    _cuda(rht_signs, "rht_signs", (torch.float32,))
    Nq, Hq, d = query.shape
    NB, two, bs, H, rb = kv_cache.shape
    S = seq_lens.shape[0]
    if two != 2 or rb != kv_int2_row_bytes(d) or rht_signs.shape != (d,):
        raise ValueError("kv_cache / rht_signs do not match the query's head size")
    if query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    if out is None:
        out = torch.empty((Nq, Hq, d), dtype=out_dtype or query.dtype, device=query.device)
    _cuda(out, "out", tuple(_DTYPES))
    if out.shape != query.shape:
        raise ValueError("out must have the query's shape")
    need = kv_int4_attention_workspace_bytes(Hq, H, d, S, max_seq_len, segment_len)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with torch.cuda.device(_one_device(query, kv_cache, block_tables, seq_lens, query_start_loc, rht_signs, out,
                                       workspace)):
        st = load().kv_int2_paged_attention(query.data_ptr(), _DTYPES[query.dtype], Nq, Hq, kv_cache.data_ptr(), NB,
                                          H, d, bs, block_tables.data_ptr(), block_tables.shape[1],
                                          seq_lens.data_ptr(), query_start_loc.data_ptr(), S, max_query_len,
                                          max_seq_len, float(softmax_scale), rht_signs.data_ptr(), segment_len,
                                          out.data_ptr(), _DTYPES[out.dtype], ws_ptr, ws_bytes, _stream(stream))
    _check("kv_int2_paged_attention", st)
    return out


def kv_int4_shared_prefix_workspace_bytes(num_q_tokens: int, num_q_heads: int, num_kv_heads: int, head_size: int,
                                          num_seqs: int, prefix_len: int, max_seq_len: int, segment_len: int = 0) -> int:
    return int(load().kv_int4_shared_prefix_workspace_bytes(num_q_tokens, num_q_heads, num_kv_heads, head_size, num_seqs,
                                                          prefix_len, max_seq_len, segment_len))


def kv_int4_shared_prefix_attention(query: torch.Tensor, kv_cache: torch.Tensor, prefix_blocks: torch.Tensor,
                                    prefix_len: int, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                    query_start_loc: torch.Tensor, softmax_scale: float, rht_signs: torch.Tensor,
                                    max_seq_len: int, out=None, out_dtype=None, segment_len: int = 0, workspace=None,
                                    stream=None, window_left: int = -1, softcap: float = 0.0, alibi_slopes=None,
                                    qq_bias=None) -> torch.Tensor:
    """kv_int4_paged_attention of a decode batch (one query token per sequence) whose first ``prefix_len``
    cached tokens are the same: their whole blocks are ``prefix_blocks`` (int32 [prefix_len // 16]), read once
    for the batch; the other arguments and the options as there, ``block_tables`` and ``seq_lens`` counting
    the prefix."""
    if stream is not None:
        with _current(stream, query):
            return kv_int4_shared_prefix_attention(query, kv_cache, prefix_blocks, prefix_len, block_tables, seq_lens,
                                                   query_start_loc, softmax_scale, rht_signs, max_seq_len, out,
                                                   out_dtype, segment_len, workspace, None, window_left, softcap,
                                                   alibi_slopes, qq_bias)
    _cuda(query, "query", _HALF_TYPES)
    _cuda(kv_cache, "kv_cache", _U8)
    _cuda(prefix_blocks, "prefix_blocks", _I32)
    _cuda(block_tables, "block_tables", _I32)
    _cuda(seq_lens, "seq_lens", _I32)
    _cuda(query_start_loc, "query_start_loc", _I32)
    _cuda(rht_signs, "rht_signs", _F32)
    qshape, cshape, tshape = query.shape, kv_cache.shape, block_tables.shape
    if len(qshape) != 3 or len(cshape) != 5 or seq_lens.dim() != 1:
        raise ValueError("query must be [num_q_tokens, num_q_heads, head_size], kv_cache 5-D and seq_lens [num_seqs]")
    Nq, Hq, d = qshape
    NB, two, bs, H, rb = cshape
    S = seq_lens.shape[0]
    if two != 2 or rb != d // 2 + 4 or rht_signs.shape != (d,):
        raise ValueError("kv_cache / rht_signs do not match the query's head size")
    if query_start_loc.shape != (S + 1,) or len(tshape) != 2 or tshape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    if prefix_blocks.dim() != 1 or prefix_blocks.shape[0] < prefix_len // max(bs, 1):
        raise ValueError("prefix_blocks must hold the prefix's prefix_len // block_size block ids")
    if out is None:
        out = torch.empty(qshape, dtype=out_dtype or query.dtype, device=query.device)
    _cuda(out, "out", tuple(_DTYPES))
    if out.shape != qshape:
        raise ValueError("out must have the query's shape")
    if workspace is None:
        need = (_lib or load()).kv_int4_shared_prefix_workspace_bytes(Nq, Hq, H, d, S, prefix_len, max_seq_len, segment_len)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    opts = None
    if window_left >= 0 or softcap != 0.0 or alibi_slopes is not None or qq_bias is not None:
        opts = ctypes.byref(_options(Hq, 1, window_left, softcap, alibi_slopes, qq_bias))
    _call("kv_int4_shared_prefix_attention",
          (query, kv_cache, prefix_blocks, block_tables, seq_lens, query_start_loc, rht_signs, out, workspace,
           alibi_slopes, qq_bias), (opts,),
          query.data_ptr(), _DTYPES[query.dtype], Nq, Hq, kv_cache.data_ptr(), NB, H, d, bs, prefix_blocks.data_ptr(),
          prefix_len, block_tables.data_ptr(), tshape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), S, 1,
          max_seq_len, float(softmax_scale), rht_signs.data_ptr(), segment_len, out.data_ptr(), _DTYPES[out.dtype],
          ws_ptr, ws_bytes)
    return out


def kv_int4_span_workspace_bytes(num_q_tokens: int, num_q_heads: int, num_kv_heads: int, head_size: int, num_seqs: int,
                                 max_query_len: int, max_seq_len: int) -> int:
    return int(load().kv_int4_span_workspace_bytes(num_q_tokens, num_q_heads, num_kv_heads, head_size, num_seqs,
                                                   max_query_len, max_seq_len))


@functools.lru_cache(maxsize=4096)
def _span_workspace(device: int, *sizes) -> int:
    """The workspace size, which depends on the device's SMs; one step's layers ask for the same sizes."""
    with torch.cuda.device(device):
        return int(load().kv_int4_span_workspace_bytes(*sizes))


def _span_attention(fn, bits, query, kv_cache, block_tables, seq_lens, query_start_loc, softmax_scale, rht_signs,
                    max_query_len, max_seq_len, key_begin, key_end, softcap, alibi_slopes, out, out_dtype, workspace, stream):
    if stream is not None:
        with _current(stream, query):
            return _span_attention(fn, bits, query, kv_cache, block_tables, seq_lens, query_start_loc, softmax_scale,
                                   rht_signs, max_query_len, max_seq_len, key_begin, key_end, softcap, alibi_slopes, out,
                                   out_dtype, workspace, None)
    _checked(query, "query", _HALF_TYPES)
    _checked(kv_cache, "kv_cache", _U8)
    _checked(block_tables, "block_tables", _I32)
    _checked(seq_lens, "seq_lens", _I32)
    _checked(query_start_loc, "query_start_loc", _I32)
    qshape, cshape, tshape = query.shape, kv_cache.shape, block_tables.shape
    if len(qshape) != 3 or len(cshape) != 5 or seq_lens.dim() != 1:
        raise ValueError("query must be [num_q_tokens, num_q_heads, head_size], kv_cache 5-D and seq_lens [num_seqs]")
    Nq, Hq, d = qshape
    NB, two, bs, H, rb = cshape
    S = seq_lens.shape[0]
    signs = ()
    if bits != 8:
        _checked(rht_signs, "rht_signs", _F32)
        if rht_signs.shape != (d,):
            raise ValueError("rht_signs must be [head_size]")
        signs = (rht_signs.data_ptr(),)
    if two != 2 or rb != d * bits // 8 + 4:
        raise ValueError("kv_cache does not match the query's head size")
    if query_start_loc.shape != (S + 1,) or len(tshape) != 2 or tshape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    begin = end = slopes = None
    if key_begin is not None:
        if _checked(key_begin, "key_begin", _I32).shape != (Nq,):
            raise ValueError("key_begin must be [num_q_tokens]")
        begin = key_begin.data_ptr()
    if key_end is not None:
        if _checked(key_end, "key_end", _I32).shape != (Nq,):
            raise ValueError("key_end must be [num_q_tokens]")
        end = key_end.data_ptr()
    if alibi_slopes is not None:
        if _checked(alibi_slopes, "alibi_slopes", _F32).shape != (Hq,):
            raise ValueError("alibi_slopes must be [num_q_heads]")
        slopes = alibi_slopes.data_ptr()
    if out is None:
        out = torch.empty(qshape, dtype=out_dtype or query.dtype, device=query.device)
    _checked(out, "out", tuple(_DTYPES))
    if out.shape != qshape:
        raise ValueError("out must have the query's shape")
    if workspace is None:
        need = _span_workspace(query.get_device(), Nq, Hq, H, d, S, max_query_len, max_seq_len)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call(fn, (query, kv_cache, block_tables, seq_lens, query_start_loc, rht_signs, key_begin, key_end, alibi_slopes, out,
               workspace), (),
          query.data_ptr(), _DTYPES[query.dtype], Nq, Hq, kv_cache.data_ptr(), NB, H, d, bs, block_tables.data_ptr(),
          tshape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), S, max_query_len, max_seq_len, float(softmax_scale),
          *signs, begin, end, float(softcap), slopes, out.data_ptr(), _DTYPES[out.dtype], ws_ptr, ws_bytes)
    return out


def kv_int4_span_attention(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                           query_start_loc: torch.Tensor, softmax_scale: float, rht_signs: torch.Tensor, max_query_len: int,
                           max_seq_len: int, key_begin=None, key_end=None, softcap: float = 0.0, alibi_slopes=None, out=None,
                           out_dtype=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of ``query`` [Nq, Hq, d] over the INT4 cache in which query row r sees the cached keys
    ``key_begin[r] <= j < key_end[r]`` of its sequence (int32 [Nq]; by default from 0, and up to its own position):
    document masks of packed prompts, prefixes and images that see themselves whole, windows, or plain causal
    attention, for chunks of any length and single tokens.  ``softcap`` > 0 caps the scaled scores by a tanh,
    ``alibi_slopes`` (fp32 [Hq]) takes slope * |pos - j| off them.  A row whose span is empty gives zeros.  The other
    arguments as kv_int4_paged_attention's (1, 2, 4 or 8 kv heads with 1, 2, 4 or 8 query heads each, head size 64 or 128);
    the workspace is sized by kv_int4_span_workspace_bytes.  kv_int4_paged_attention takes plain causal single tokens
    in less time."""
    return _span_attention("kv_int4_span_attention", 4, query, kv_cache, block_tables, seq_lens, query_start_loc,
                           softmax_scale, rht_signs, max_query_len, max_seq_len, key_begin, key_end, softcap, alibi_slopes,
                           out, out_dtype, workspace, stream)


def kv_int8_span_attention(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                           query_start_loc: torch.Tensor, softmax_scale: float, max_query_len: int, max_seq_len: int,
                           key_begin=None, key_end=None, softcap: float = 0.0, alibi_slopes=None, out=None, out_dtype=None,
                           workspace=None, stream=None) -> torch.Tensor:
    """kv_int4_span_attention over the INT8 comparator's cache (no signs)."""
    return _span_attention("kv_int8_span_attention", 8, query, kv_cache, block_tables, seq_lens, query_start_loc,
                           softmax_scale, None, max_query_len, max_seq_len, key_begin, key_end, softcap, alibi_slopes, out,
                           out_dtype, workspace, stream)


def kv_int2_span_attention(query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                           query_start_loc: torch.Tensor, softmax_scale: float, rht_signs: torch.Tensor, max_query_len: int,
                           max_seq_len: int, key_begin=None, key_end=None, softcap: float = 0.0, alibi_slopes=None, out=None,
                           out_dtype=None, workspace=None, stream=None) -> torch.Tensor:
    """kv_int4_span_attention over the INT2 Lloyd-Max cache."""
    return _span_attention("kv_int2_span_attention", 2, query, kv_cache, block_tables, seq_lens, query_start_loc,
                           softmax_scale, rht_signs, max_query_len, max_seq_len, key_begin, key_end, softcap, alibi_slopes,
                           out, out_dtype, workspace, stream)


def kv_int4_read_device_status(stream=None) -> dict:
    """Synchronise the stream and return the device's status counters by name."""
    buf = (ctypes.c_uint32 * _STAT_COUNT)()
    _check("kv_int4_read_device_status", load().kv_int4_read_device_status(buf, _stream(stream)))
    return {name: int(buf[i]) for i, name in enumerate(STAT_NAMES)}


def kv_int4_clear_device_status(stream=None) -> None:
    _check("kv_int4_clear_device_status", load().kv_int4_clear_device_status(_stream(stream)))


def kv_int4_selftest_wait_timeout(timeout_ns: int = 5_000_000, stream=None) -> None:
    """Run the bounded-wait diagnostic (a wait nothing completes); it records one wait_timeout."""
    _check("kv_int4_selftest_wait_timeout", load().kv_int4_selftest_wait_timeout(int(timeout_ns), _stream(stream)))
