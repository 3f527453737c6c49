"""Python binding of libpa.so, the paged KV cache attention library for GB300.

Argument marshalling only: every function takes torch tensors, checks that they
are contiguous CUDA tensors of the expected shapes, and passes raw device
pointers, sizes and the current CUDA stream to the C ABI declared in
``include/pa.h``.  All computation happens in the library's CUDA kernels; there
is no fallback.  Importing this package raises ImportError when libpa.so has
not been built (``python paged_kv_cache_pagedattention_gb300/build.py``).

Cache tensors have shape ``[num_blocks][num_kv_heads][block_size][head_size]``;
FP8 e4m3 caches are uint8 tensors of codes with per-tensor fp32 scales passed as
one-element float32 CUDA tensors (one value per KV head selects per-head scales).
NVFP4 caches are 3-D uint8 tensors ``[num_blocks][num_kv_heads][tile_bytes]``,
``tile_bytes = 9 * block_size * head_size / 16`` (codes, then block scales; see
``include/pa.h``); their head size is taken from the query or key tensor.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libpa.so not found at {LIB_PATH}; build it with "
                      "`python paged_kv_cache_pagedattention_gb300/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_BOUNDS, \
    PA_ERR_TIMEOUT, PA_ERR_CUDA = range(7)
PA_F32, PA_F16, PA_BF16, PA_FP8_E4M3, PA_FP8_E5M2, PA_FP8_E4M3_PER_HEAD, PA_FP8_E5M2_PER_HEAD, PA_NVFP4, \
    PA_NVFP4_PER_HEAD = range(9)
PA_ERRFLAG_BLOCK_TABLE, PA_ERRFLAG_SLOT, PA_ERRFLAG_SEQ_LEN, PA_ERRFLAG_QUERY, PA_ERRFLAG_TIMEOUT = \
    0x1, 0x2, 0x4, 0x8, 0x10
# diagnostic only: a declared shared block differed for some member (the output is unaffected)
PA_ERRFLAG_SHARED_MISMATCH = 0x20
PA_ERRFLAG_PARENT, PA_ERRFLAG_POOL, PA_ERRFLAG_REF_COUNT, PA_ERRFLAG_MEDIA = 0x40, 0x80, 0x100, 0x200
PA_MAX_BEAM_CANDIDATES, PA_MAX_BEAMS, PA_MAX_VOCAB = 32, 1024, 1 << 30
PA_MAX_ROTARY_AXES, PA_MAX_ROTARY_AXES_DIM = 4, 512
ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}

# Names of the kernel kinds reported by pa_trace_read.
TRACE_KINDS = ("reshape_and_cache", "attention", "merge", "varlen_plan", "prefill_tiles", "shared_prefix",
               "shared_span", "copy_blocks", "varlen_span", "rotary_and_cache", "beam_select", "fork_blocks",
               "append_blocks", "release_blocks", "positions_and_slots", "diff_attention", "diff_merge",
               "diff_prefill_tiles")

# Every symbol include/pa.h declares, with its ctypes signature.
_P, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_D = ctypes.c_double
SIGNATURES = {
    "pa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pa_version": (_I32, []),
    "pa_reshape_and_cache": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32,
                                            ctypes.c_int, ctypes.c_int, _P, _P, _P]),
    "pa_copy_blocks": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _I32, ctypes.c_int, _P]),
    "pa_rotary_frequencies": (ctypes.c_int, [ctypes.POINTER(_F), ctypes.POINTER(_F), _I32, _D, ctypes.c_int, _D, _D,
                                             _D, _D]),
    "pa_rotary_and_cache": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32,
                                           _I32, _I32, _F, _I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int,
                                           _P, _P, _P]),
    "pa_rotary_pair_axes": (ctypes.c_int, [_P, _I32, ctypes.POINTER(_I32), _I32, _I32]),
    "pa_rotary_axes_and_cache": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_char_p, _I32, _I32, _I32,
                                                _I32, _I32, _I32, _I32, _I32, _I32, _F, _I64, _I64, _I64, _I64,
                                                ctypes.c_int, ctypes.c_int, _P, _P, _P]),
    "pa_positions_and_slots": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                              _P]),
    "pa_beam_select_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "pa_beam_select": (ctypes.c_int, [_P, _P, _P, _P, _I64, _P, _I32, _I32, _I32, _I32, ctypes.c_int, _P, _SZ, _P]),
    "pa_fork_blocks": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P]),
    "pa_append_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "pa_append_blocks": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P]),
    "pa_release_blocks": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, _I32, _I32, _P]),
    "pa_default_partition_size": (_I32, [_I32, _I32, _I32, _I32]),
    "pa_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "pa_decode": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32,
                                 _I32, _F, ctypes.c_int, ctypes.c_int, _P, _P, _I32, _P, _SZ, _P]),
    "pa_decode_windowed": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32,
                                          _I32, _F, _I32, ctypes.c_int, ctypes.c_int, _P, _P, _I32, _P, _SZ, _P]),
    "pa_decode_shared_prefix_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "pa_decode_shared_prefix": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32,
                                               _I32, _F, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P, _I32,
                                               _I32, _I32, _P, _SZ, _P]),
    "pa_decode_static_workspace": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32,
                                                  _I32, _I32, _F, ctypes.c_int, ctypes.c_int, _P, _P, _I32, _P]),
    "pa_varlen_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "pa_varlen_attn": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32,
                                      _I32, _I32, _I32, _I32, _F, _I32, ctypes.c_int, ctypes.c_int,
                                      _P, _P, _I32, _P, _SZ, _P]),
    "pa_varlen_attn_windowed": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32,
                                               _I32, _I32, _I32, _I32, _F, _I32, _I32, ctypes.c_int, ctypes.c_int,
                                               _P, _P, _I32, _P, _SZ, _P]),
    "pa_diff_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "pa_diff_decode": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F, _P,
                                      _I64, _I64, _P, _F, _I32, ctypes.c_int, ctypes.c_int, _P, _P, _I32, _P, _SZ, _P]),
    "pa_diff_varlen_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "pa_diff_varlen_attn": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32,
                                           _I32, _I32, _F, _P, _I64, _I64, _P, _F, _I32, _I32, ctypes.c_int,
                                           ctypes.c_int, _P, _P, _I32, _P, _SZ, _P]),
    "pa_get_error_flags": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _I32, _P]),
    "pa_trace_enable": (ctypes.c_int, [_I32]),
    "pa_trace_read": (ctypes.c_int, [_I32, ctypes.POINTER(_I64), ctypes.POINTER(ctypes.c_double), _I32]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class PAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.pa_status_string(status).decode()}")


def _check(status: int, where: str) -> None:
    if status != PA_OK:
        raise PAError(status, where)


# FP8 caches: uint8 codes are e4m3; torch's float8 dtypes name their format
_DT = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16, torch.uint8: PA_FP8_E4M3,
       torch.float8_e4m3fn: PA_FP8_E4M3, torch.float8_e5m2: PA_FP8_E5M2}


def dtype_code(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported tensor dtype {t.dtype}") from None


def is_nvfp4(cache: torch.Tensor) -> bool:
    """NVFP4 caches are the 3-D uint8 tensors [num_blocks][num_kv_heads][tile_bytes]."""
    return cache.dim() == 3 and cache.dtype == torch.uint8


def kv_code(cache: torch.Tensor, k_scale=None) -> int:
    """Cache dtype code; scales holding more than one value (one per KV head, the
    cache's dimension 1) select the per-head format."""
    code = PA_NVFP4 if is_nvfp4(cache) else dtype_code(cache)
    if k_scale is None:
        return code
    if code in (PA_FP8_E4M3, PA_FP8_E5M2, PA_NVFP4) and k_scale.numel() > 1:
        if k_scale.numel() != cache.shape[1]:
            raise ValueError("scales: one per tensor or one per KV head")
        return {PA_FP8_E4M3: PA_FP8_E4M3_PER_HEAD, PA_FP8_E5M2: PA_FP8_E5M2_PER_HEAD,
                PA_NVFP4: PA_NVFP4_PER_HEAD}[code]
    return code


def cache_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor, head_size: int):
    """(num_blocks, num_kv_heads, block_size, head_size) of a K/V cache pair; the
    head size of an NVFP4 cache comes from the caller's query or key tensor."""
    shape = k_cache.shape
    if v_cache.shape != shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must match")
    if len(shape) == 3 and k_cache.dtype == torch.uint8:
        nb, hkv, tile = shape
        if head_size < 1 or (16 * tile) % (9 * head_size):
            raise ValueError("NVFP4 cache: tile_bytes must be 9 * block_size * head_size / 16")
        return nb, hkv, 16 * tile // (9 * head_size), head_size
    if len(shape) != 4:
        raise ValueError("cache must be [num_blocks][num_kv_heads][block_size][head_size]")
    return tuple(shape)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def pa_status_string(status: int) -> str:
    return _lib.pa_status_string(status).decode()


def pa_version() -> int:
    return _lib.pa_version()


def pa_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, k_scale=None, v_scale=None,
                         stream=None) -> None:
    """Write key/value [T][Hkv][d] into the paged caches at slot_mapping (int64 [T])."""
    nb, hkv, bs, d = cache_geometry(k_cache, v_cache, key.shape[-1])
    if key.dim() != 3 or tuple(key.shape[1:]) != (hkv, d) or key.shape != value.shape:
        raise ValueError("key/value must be [num_tokens][num_kv_heads][head_size]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != key.shape[0]:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    _check(_lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(slot_mapping), key.shape[0], nb, hkv, d, bs,
                                     dtype_code(key), kv_code(k_cache, k_scale), _ptr(k_scale), _ptr(v_scale),
                                     _stream(stream)), "pa_reshape_and_cache")


def pa_copy_blocks(k_cache, v_cache, block_mapping, stream=None) -> None:
    """Copy whole physical blocks: block_mapping is int64 [num_pairs][2] of (src, dst)."""
    if is_nvfp4(k_cache):
        # only the tile size matters for a copy: any (block_size, head_size) with
        # 9 * block_size * head_size / 16 == tile_bytes names it
        nb, hkv, bs, d = cache_geometry(k_cache, v_cache, k_cache.shape[2] // 9)
    else:
        nb, hkv, bs, d = cache_geometry(k_cache, v_cache, 0)
    if block_mapping.dtype != torch.int64 or block_mapping.dim() != 2 or block_mapping.shape[1] != 2:
        raise ValueError("block_mapping must be int64 [num_pairs][2]")
    if not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be contiguous")
    n = block_mapping.shape[0]
    k_ptr, v_ptr = _ptr(k_cache), _ptr(v_cache)
    s = _raw_stream(_current_device()) if stream is None else stream.cuda_stream
    _check(_lib.pa_copy_blocks(k_ptr, v_ptr, _ptr(block_mapping) if n else None, n, nb, hkv, d, bs,
                               kv_code(k_cache), s), "pa_copy_blocks")


# A device's current stream and the current device as torch keeps them.  Their public forms
# (torch.cuda.current_stream, torch.cuda.current_device) take 1.1 and 0.2 us on the host, these
# 0.1; the calls below take 6 to 10.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_int32, _int64, _float32 = torch.int32, torch.int64, torch.float32


def _on_device(index, call, *args, **kwargs):
    """``call`` again with the tensors' device current; refuses tensors that are not CUDA's."""
    if index < 0:
        raise ValueError(f"{call.__name__}: expected CUDA tensors")
    with torch.cuda.device(index):
        return call(*args, **kwargs)


def _stream_on(stream, index, where):
    """The raw handle of the caller's stream, which has to be on device ``index``."""
    if stream.device.index != index:
        raise ValueError(f"{where}: the stream belongs to another device than the tensors")
    return stream.cuda_stream


def _bad(t, shape, what):
    """Refuse a tensor that is not contiguous int32 of ``shape``, or is on another device."""
    if t.dtype is not _int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {list(shape)}")
    raise ValueError(f"{what}: all tensors must be on one CUDA device")


def _check_heads(t, what):
    """Refuse a [tokens][heads][head_size] tensor whose heads are not contiguous."""
    _, head, elem = t.stride()
    if (elem != 1 and t.shape[2] > 1) or (head != t.shape[2] and t.shape[1] > 1):
        raise ValueError(f"{what}: every token's [heads][head_size] must be contiguous")


def pa_rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_max_position=0.0,
                          low_turns=1.0, high_turns=32.0, device=None):
    """(inv_freq, attn_factor) for pa_rotary_and_cache: a float32 tensor [rotary_dim/2] on
    ``device`` (default: the current CUDA device) and the factor on the rotated values.
    scaling: "none", "linear", "ntk" or "by_parts" (see pa.h)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}")
    host = (ctypes.c_float * max(1, int(rotary_dim) // 2))()
    attn = ctypes.c_float(1.0)
    _check(_lib.pa_rotary_frequencies(host, ctypes.byref(attn), int(rotary_dim), float(base),
                                      ROTARY_SCALINGS[scaling], float(factor), float(original_max_position),
                                      float(low_turns), float(high_turns)), "pa_rotary_frequencies")
    freq = torch.tensor(list(host), dtype=torch.float32, device="cuda" if device is None else device)
    return freq, float(attn.value)


def pa_rotary_and_cache(q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq,
                        interleaved=False, attn_factor=1.0, k_scale=None, v_scale=None, stream=None,
                        pair_axis=None) -> None:
    """Rotate q [T][Hq][d] into q_out (which may be q) and key [T][Hkv][d] by positions (int32
    [T]), and write key and value into the paged caches at slot_mapping (int64 [T]; a negative
    slot skips the token).  inv_freq float32 [rotary_dim/2].  q, key and value may be slices of
    one projection (any distance between tokens).  q and q_out None: keys only.  pair_axis: see
    pa_rotary_axes_and_cache."""
    shape, dtype, dev = key.shape, key.dtype, key.get_device()
    if len(shape) != 3 or value.shape != shape or value.dtype is not dtype:
        raise ValueError("key/value must be [num_tokens][num_kv_heads][head_size] of one dtype")
    t, hkv, d = shape
    nb, heads, bs, head = cache_geometry(k_cache, v_cache, d)
    if heads != hkv or head != d or not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous and match key's heads")
    # rows: heads are contiguous, tokens any distance apart
    k_stride, k_head, k_elem = key.stride()
    v_stride, v_head, v_elem = value.stride()
    if k_elem != 1 or v_elem != 1 or k_head != d or v_head != d:
        _check_heads(key, "key")
        _check_heads(value, "value")
    hq = q_ptr = q_out_ptr = q_stride = q_out_stride = 0
    if q is not None or q_out is not None:
        q_shape = None if q is None else q.shape
        if q_out is None or q_shape is None or q_out.shape != q_shape or len(q_shape) != 3 or \
                q.dtype is not dtype or q_out.dtype is not dtype or q_shape[0] != t or q_shape[2] != d:
            raise ValueError("q/q_out must be [num_tokens][num_q_heads][head_size] of key's dtype")
        if q.get_device() != dev or q_out.get_device() != dev:
            raise ValueError("q/q_out: all tensors must be on one CUDA device")
        hq, q_ptr, q_out_ptr = q_shape[1], q.data_ptr(), q_out.data_ptr()
        q_stride, q_head, q_elem = q.stride()
        q_out_stride, q_out_head, q_out_elem = q_out.stride()
        if q_elem != 1 or q_out_elem != 1 or q_head != d or q_out_head != d:
            _check_heads(q, "q")
            _check_heads(q_out, "q_out")
    axes = 0
    if pair_axis is not None:
        if positions.dim() != 2:
            raise ValueError("positions must be int32 [num_axes][num_tokens]")
        axes = positions.shape[0]
        if type(pair_axis) is not bytes or len(pair_axis) != inv_freq.numel():
            raise ValueError("pair_axis must be bytes, one for each pair of inv_freq")
    places = (t,) if pair_axis is None else (axes, t)
    if positions.dtype is not _int32 or positions.shape != places or not positions.is_contiguous():
        _bad(positions, places, "positions")
    if slot_mapping.dtype is not _int64 or slot_mapping.shape != (t,) or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 tensor [num_tokens]")
    if inv_freq.dtype is not _float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float32 tensor [rotary_dim/2]")
    code = kv_code(k_cache, k_scale)
    k_scale_ptr = v_scale_ptr = None
    if code >= PA_FP8_E4M3 and k_scale is not None and v_scale is not None:
        n = k_scale.numel()
        if (n != 1 and n != hkv) or v_scale.numel() != n or k_scale.dtype is not _float32 or \
                v_scale.dtype is not _float32 or not (k_scale.is_contiguous() and v_scale.is_contiguous()) or \
                not k_scale.get_device() == v_scale.get_device() == dev:
            raise ValueError("scales: float32, both one per tensor or both one per KV head, on the caches' device")
        k_scale_ptr, v_scale_ptr = k_scale.data_ptr(), v_scale.data_ptr()
    if not (value.get_device() == k_cache.get_device() == v_cache.get_device() == positions.get_device() ==
            slot_mapping.get_device() == inv_freq.get_device() == dev):
        raise ValueError("pa_rotary_and_cache: all tensors must be on one CUDA device")
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_rotary_and_cache, q_out, q, key, value, k_cache, v_cache, positions, slot_mapping,
                          inv_freq, interleaved, attn_factor, k_scale, v_scale, stream, pair_axis)
    if pair_axis is not None:
        st = _lib.pa_rotary_axes_and_cache(
            q_out_ptr, q_ptr, key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            positions.data_ptr(), slot_mapping.data_ptr(), inv_freq.data_ptr(), pair_axis, axes, t, nb, hq, hkv, d,
            2 * inv_freq.numel(), bs, 1 if interleaved else 0, attn_factor, q_out_stride, q_stride, k_stride, v_stride,
            dtype_code(key), code, k_scale_ptr, v_scale_ptr,
            _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_rotary_axes_and_cache"))
        if st != PA_OK:
            raise PAError(st, "pa_rotary_axes_and_cache")
        return
    st = _lib.pa_rotary_and_cache(
        q_out_ptr, q_ptr, key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        positions.data_ptr(), slot_mapping.data_ptr(), inv_freq.data_ptr(), t, nb, hq, hkv, d, 2 * inv_freq.numel(),
        bs, 1 if interleaved else 0, attn_factor, q_out_stride, q_stride, k_stride, v_stride, dtype_code(key), code,
        k_scale_ptr, v_scale_ptr, _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_rotary_and_cache"))
    if st != PA_OK:
        raise PAError(st, "pa_rotary_and_cache")


def pa_rotary_pair_axes(sections, cycled=False) -> bytes:
    """The axis of every pair for pa_rotary_axes_and_cache: sections[a] pairs turn on axis a,
    the axes one after the other, or dealt round (see pa.h)."""
    sections = [int(n) for n in sections]
    pairs = sum(sections)
    if not 1 <= pairs <= PA_MAX_ROTARY_AXES_DIM // 2:
        raise ValueError("sections must sum to the rotated pairs, at most 256")
    out = (ctypes.c_uint8 * pairs)()
    _check(_lib.pa_rotary_pair_axes(out, 2 * pairs, (_I32 * len(sections))(*sections), len(sections),
                                    1 if cycled else 0), "pa_rotary_pair_axes")
    return bytes(out)


def pa_rotary_axes_and_cache(q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq, pair_axis,
                             interleaved=False, attn_factor=1.0, k_scale=None, v_scale=None, stream=None) -> None:
    """pa_rotary_and_cache with positions on several axes (int32 [num_axes][T]): pair i turns by
    the token's position on axis pair_axis[i] (bytes [rotary_dim/2]; pa_rotary_pair_axes)."""
    if pair_axis is None:
        raise ValueError("pair_axis must be bytes, one for each pair of inv_freq")
    pa_rotary_and_cache(q_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq, interleaved,
                        attn_factor, k_scale, v_scale, stream, pair_axis)


def pa_beam_select_workspace_size(num_seqs, num_beams, vocab_size, num_candidates) -> int:
    return _lib.pa_beam_select_workspace_size(num_seqs, num_beams, vocab_size, num_candidates)


def pa_beam_select(out_scores, out_tokens, out_parents, logits, beam_scores, workspace, stream=None) -> None:
    """The best candidates of each sequence's beams: out_scores float32, out_tokens and
    out_parents int32, all [num_seqs][num_candidates]; logits [num_seqs*num_beams][vocab]
    (rows may be padded), beam_scores float32 [num_seqs][num_beams]."""
    beams, rows, shape, dev = beam_scores.shape, logits.shape, out_scores.shape, logits.get_device()
    if beam_scores.dtype is not _float32 or len(beams) != 2 or not beam_scores.is_contiguous():
        raise ValueError("beam_scores must be a contiguous float32 tensor [num_seqs][num_beams]")
    b, w = beams
    stride = logits.stride()
    if len(rows) != 2 or rows[0] != b * w or (stride[1] != 1 and rows[1] > 1):
        raise ValueError("logits must be [num_seqs*num_beams][vocab_size] with contiguous rows")
    if len(shape) != 2 or shape[0] != b or out_scores.dtype is not _float32 or not out_scores.is_contiguous():
        raise ValueError("out_scores must be a contiguous float32 tensor [num_seqs][num_candidates]")
    if out_tokens.dtype is not _int32 or out_tokens.shape != shape or not out_tokens.is_contiguous():
        _bad(out_tokens, shape, "out_tokens")
    if out_parents.dtype is not _int32 or out_parents.shape != shape or not out_parents.is_contiguous():
        _bad(out_parents, shape, "out_parents")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not (beam_scores.get_device() == out_scores.get_device() == out_tokens.get_device() ==
            out_parents.get_device() == workspace.get_device() == dev):
        raise ValueError("pa_beam_select: all tensors must be on one CUDA device")
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_beam_select, out_scores, out_tokens, out_parents, logits, beam_scores, workspace,
                          stream)
    st = _lib.pa_beam_select(
        out_scores.data_ptr(), out_tokens.data_ptr(), out_parents.data_ptr(), logits.data_ptr(), stride[0],
        beam_scores.data_ptr(), b, w, rows[1], shape[1], dtype_code(logits), workspace.data_ptr(),
        workspace.nbytes, _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_beam_select"))
    if st != PA_OK:
        raise PAError(st, "pa_beam_select")


def _pages(block_tables, seq_lens, ref_counts):
    """(rows, max_blocks_per_seq, num_blocks, device) of a pool's arrays."""
    shape, blocks, dev = block_tables.shape, ref_counts.shape, block_tables.get_device()
    if len(shape) != 2 or len(blocks) != 1:
        raise ValueError("block_tables must be [rows][max_blocks_per_seq] and ref_counts [num_blocks]")
    n, width = shape
    if block_tables.dtype is not _int32 or not block_tables.is_contiguous():
        _bad(block_tables, shape, "block_tables")
    if seq_lens.dtype is not _int32 or seq_lens.shape != (n,) or not seq_lens.is_contiguous() or \
            seq_lens.get_device() != dev:
        _bad(seq_lens, (n,), "seq_lens")
    if ref_counts.dtype is not _int32 or not ref_counts.is_contiguous() or ref_counts.get_device() != dev:
        _bad(ref_counts, blocks, "ref_counts")
    return n, width, blocks[0], dev


def pa_fork_blocks(block_tables_out, seq_lens_out, block_tables, seq_lens, parents, ref_counts, block_size,
                   stream=None) -> None:
    """Children rows take the blocks and lengths of rows ``parents`` (int32 [children];
    negative: an empty row) of block_tables/seq_lens; ref_counts int32 [num_blocks] counts
    the holders of every block.  See pa.h."""
    m, width, blocks, dev = _pages(block_tables, seq_lens, ref_counts)
    n = parents.numel()
    if parents.dtype is not _int32 or parents.dim() != 1 or not parents.is_contiguous() or parents.get_device() != dev:
        _bad(parents, (n,), "parents")
    if block_tables_out.dtype is not _int32 or block_tables_out.shape != (n, width) or \
            not block_tables_out.is_contiguous() or block_tables_out.get_device() != dev:
        _bad(block_tables_out, (n, width), "block_tables_out")
    if seq_lens_out.dtype is not _int32 or seq_lens_out.shape != (n,) or not seq_lens_out.is_contiguous() or \
            seq_lens_out.get_device() != dev:
        _bad(seq_lens_out, (n,), "seq_lens_out")
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_fork_blocks, block_tables_out, seq_lens_out, block_tables, seq_lens, parents,
                          ref_counts, block_size, stream)
    st = _lib.pa_fork_blocks(
        block_tables_out.data_ptr(), seq_lens_out.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
        parents.data_ptr(), ref_counts.data_ptr(), n, m, width, blocks, block_size,
        _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_fork_blocks"))
    if st != PA_OK:
        raise PAError(st, "pa_fork_blocks")


def pa_append_workspace_size(num_seqs, total_q_tokens, block_size) -> int:
    return _lib.pa_append_workspace_size(num_seqs, total_q_tokens, block_size)


def pa_append_blocks(block_tables, seq_lens, query_start_loc, slot_mapping, block_mapping, ref_counts, block_size,
                     workspace, stream=None) -> None:
    """Room for the next tokens of every row (query_start_loc int32 [rows+1]): blocks from the
    pool, slots (int64 [new tokens]) and copy-on-write pairs (block_mapping int64 [rows][2],
    for pa_copy_blocks).  All or nothing; see pa.h."""
    n, width, blocks, dev = _pages(block_tables, seq_lens, ref_counts)
    if query_start_loc.dtype is not _int32 or query_start_loc.shape != (n + 1,) or \
            not query_start_loc.is_contiguous() or query_start_loc.get_device() != dev:
        _bad(query_start_loc, (n + 1,), "query_start_loc")
    if slot_mapping.dtype is not _int64 or slot_mapping.dim() != 1 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 tensor [total_q_tokens]")
    if block_mapping.dtype is not _int64 or block_mapping.shape != (n, 2) or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous int64 tensor [rows][2]")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not (slot_mapping.get_device() == block_mapping.get_device() == workspace.get_device() == dev):
        raise ValueError("pa_append_blocks: all tensors must be on one CUDA device")
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_append_blocks, block_tables, seq_lens, query_start_loc, slot_mapping, block_mapping,
                          ref_counts, block_size, workspace, stream)
    st = _lib.pa_append_blocks(
        block_tables.data_ptr(), seq_lens.data_ptr(), query_start_loc.data_ptr(), slot_mapping.data_ptr(),
        block_mapping.data_ptr(), ref_counts.data_ptr(), n, slot_mapping.numel(), width, blocks, block_size,
        workspace.data_ptr(), workspace.nbytes,
        _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_append_blocks"))
    if st != PA_OK:
        raise PAError(st, "pa_append_blocks")


def pa_release_blocks(block_tables, seq_lens, ref_counts, block_size, keep_lens=None, stream=None) -> None:
    """Give up what lies behind the first keep_lens (int32 [rows]; None: 0) tokens of every row:
    the blocks lose a holder and seq_lens is cut.  See pa.h."""
    n, width, blocks, dev = _pages(block_tables, seq_lens, ref_counts)
    keep_ptr = None
    if keep_lens is not None:
        if keep_lens.dtype is not _int32 or keep_lens.shape != (n,) or not keep_lens.is_contiguous() or \
                keep_lens.get_device() != dev:
            _bad(keep_lens, (n,), "keep_lens")
        keep_ptr = keep_lens.data_ptr()
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_release_blocks, block_tables, seq_lens, ref_counts, block_size, keep_lens, stream)
    st = _lib.pa_release_blocks(
        block_tables.data_ptr(), seq_lens.data_ptr(), keep_ptr, ref_counts.data_ptr(), n, width, blocks, block_size,
        _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_release_blocks"))
    if st != PA_OK:
        raise PAError(st, "pa_release_blocks")


def pa_positions_and_slots(positions, slot_mapping, query_start_loc, seq_lens, block_tables, num_blocks, block_size,
                           media_start=None, media=None, stream=None) -> None:
    """Positions (int32 [T], or [3][T] for time, height and width; None: not wanted) and cache slots
    (int64 [T]; None: not wanted, and block_tables may be None) of a step's tokens: query_start_loc
    int32 [rows+1], seq_lens int32 [rows] with the new tokens, block_tables int32 [rows][width].
    media int32 [M][5] (first token, frames, rows, columns, step) of the sequences, media_start
    int32 [rows+1].  See pa.h."""
    n, dev = seq_lens.numel(), seq_lens.get_device()
    if seq_lens.dtype is not _int32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        _bad(seq_lens, (n,), "seq_lens")
    if query_start_loc.dtype is not _int32 or query_start_loc.shape != (n + 1,) or \
            not query_start_loc.is_contiguous() or query_start_loc.get_device() != dev:
        _bad(query_start_loc, (n + 1,), "query_start_loc")
    total, axes, width, records = 0, 1, 0, 0
    positions_ptr = slots_ptr = tables_ptr = start_ptr = media_ptr = None
    if slot_mapping is not None:
        if slot_mapping.dtype is not _int64 or slot_mapping.dim() != 1 or not slot_mapping.is_contiguous() or \
                slot_mapping.get_device() != dev:
            raise ValueError("slot_mapping must be a contiguous int64 tensor [total_q_tokens] on seq_lens' device")
        if block_tables is None or block_tables.dim() != 2:
            raise ValueError("slot_mapping needs block_tables [rows][max_blocks_per_seq]")
        total, width = slot_mapping.numel(), block_tables.shape[1]
        if block_tables.dtype is not _int32 or block_tables.shape[0] != n or not block_tables.is_contiguous() or \
                block_tables.get_device() != dev:
            _bad(block_tables, (n, width), "block_tables")
        slots_ptr, tables_ptr = slot_mapping.data_ptr(), block_tables.data_ptr()
    if positions is not None:
        shape = positions.shape
        if len(shape) not in (1, 2):
            raise ValueError("positions must be int32 [total_q_tokens] or [3][total_q_tokens]")
        axes = shape[0] if len(shape) == 2 else 1
        if positions.dtype is not _int32 or not positions.is_contiguous() or positions.get_device() != dev or \
                (slot_mapping is not None and shape[-1] != total):
            _bad(positions, shape[:-1] + (total or shape[-1],), "positions")
        total, positions_ptr = shape[-1], positions.data_ptr()
    elif media is not None or media_start is not None:
        axes = 3
    if media is not None or media_start is not None:
        if media is None or media_start is None or media.dim() != 2:
            raise ValueError("media [M][5] and media_start [rows+1] go together")
        records = media.shape[0]
        if media.dtype is not _int32 or media.shape[1] != 5 or not media.is_contiguous() or media.get_device() != dev:
            _bad(media, (records, 5), "media")
        if media_start.dtype is not _int32 or media_start.shape != (n + 1,) or not media_start.is_contiguous() or \
                media_start.get_device() != dev:
            _bad(media_start, (n + 1,), "media_start")
        start_ptr, media_ptr = media_start.data_ptr(), media.data_ptr()
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_positions_and_slots, positions, slot_mapping, query_start_loc, seq_lens,
                          block_tables, num_blocks, block_size, media_start, media, stream)
    st = _lib.pa_positions_and_slots(
        positions_ptr, slots_ptr, query_start_loc.data_ptr(), seq_lens.data_ptr(), tables_ptr, start_ptr, media_ptr,
        n, total, axes, records, width, num_blocks, block_size,
        _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_positions_and_slots"))
    if st != PA_OK:
        raise PAError(st, "pa_positions_and_slots")


def pa_default_partition_size(num_seqs, num_kv_heads, max_seq_len, block_size) -> int:
    return _lib.pa_default_partition_size(num_seqs, num_kv_heads, max_seq_len, block_size)


def pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len, block_size,
                             partition_size=0) -> int:
    return _lib.pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len,
                                         block_size, partition_size)


def pa_decode(out, q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, scale, workspace,
              k_scale=None, v_scale=None, partition_size=0, stream=None, window=0) -> None:
    """PagedAttention decode; out/q [B][Hq][d], block_tables int32 [B][max_blocks], seq_lens int32 [B].
    window > 0: sliding-window attention (pa_decode_windowed)."""
    nb, hkv, bs, d = cache_geometry(k_cache, v_cache, q.shape[-1])
    b, hq = q.shape[0], q.shape[1]
    if q.dim() != 3 or q.shape[2] != d or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q/out must be [num_seqs][num_q_heads][head_size] of one dtype")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b:
        raise ValueError("block_tables must be int32 [num_seqs][max_blocks_per_seq]")
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != b:
        raise ValueError("seq_lens must be int32 [num_seqs]")
    _check(_lib.pa_decode_windowed(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), nb, _ptr(block_tables),
                                   block_tables.shape[1], _ptr(seq_lens), b, int(max_seq_len), hq, hkv, d, bs,
                                   float(scale), int(window), dtype_code(q), kv_code(k_cache, k_scale), _ptr(k_scale),
                                   _ptr(v_scale), int(partition_size), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)), "pa_decode")


def pa_decode_shared_prefix_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads, head_size,
                                           max_seq_len, block_size, partition_size=0) -> int:
    return _lib.pa_decode_shared_prefix_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads,
                                                       head_size, max_seq_len, block_size, partition_size)


def pa_decode_shared_prefix(out, q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, scale, workspace,
                            group_start, group_shared_blocks, max_group_size, k_scale=None, v_scale=None,
                            partition_size=0, stream=None) -> None:
    """pa_decode where groups of consecutive sequences share leading blocks.

    group_start int32 [G+1] (device), group_shared_blocks int32 [G] (device)."""
    nb, hkv, bs, d = cache_geometry(k_cache, v_cache, q.shape[-1])
    b, hq = q.shape[0], q.shape[1]
    if q.dim() != 3 or q.shape[2] != d or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q/out must be [num_seqs][num_q_heads][head_size] of one dtype")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b:
        raise ValueError("block_tables must be int32 [num_seqs][max_blocks_per_seq]")
    if group_start.dtype != torch.int32 or group_shared_blocks.dtype != torch.int32 or \
            group_start.numel() != group_shared_blocks.numel() + 1:
        raise ValueError("group_start int32 [G+1], group_shared_blocks int32 [G]")
    _check(_lib.pa_decode_shared_prefix(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), nb, _ptr(block_tables),
                                        block_tables.shape[1], _ptr(seq_lens), b, int(max_seq_len), hq, hkv, d,
                                        bs, float(scale), dtype_code(q), kv_code(k_cache, k_scale), _ptr(k_scale),
                                        _ptr(v_scale), _ptr(group_start), _ptr(group_shared_blocks),
                                        group_shared_blocks.numel(), int(max_group_size), int(partition_size),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "pa_decode_shared_prefix")


def pa_decode_static_workspace(out, q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, scale,
                               k_scale=None, v_scale=None, partition_size=0, stream=None) -> None:
    """pa_decode with the library's fixed scratch array instead of a workspace: for
    callers that cannot allocate device memory where attention runs.  See pa.h."""
    nb, hkv, bs, d = cache_geometry(k_cache, v_cache, q.shape[-1])
    b, hq = q.shape[0], q.shape[1]
    if q.dim() != 3 or q.shape[2] != d or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q/out must be [num_seqs][num_q_heads][head_size] of one dtype")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b:
        raise ValueError("block_tables must be int32 [num_seqs][max_blocks_per_seq]")
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != b:
        raise ValueError("seq_lens must be int32 [num_seqs]")
    _check(_lib.pa_decode_static_workspace(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), nb,
                                           _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), b,
                                           int(max_seq_len), hq, hkv, d, bs, float(scale), dtype_code(q),
                                           kv_code(k_cache, k_scale), _ptr(k_scale), _ptr(v_scale),
                                           int(partition_size), _stream(stream)),
           "pa_decode_static_workspace")


def pa_varlen_workspace_size(num_seqs, total_q_tokens, max_query_len, num_q_heads, num_kv_heads,
                             head_size, max_seq_len, block_size, partition_size=0) -> int:
    return _lib.pa_varlen_workspace_size(num_seqs, total_q_tokens, max_query_len, num_q_heads,
                                         num_kv_heads, head_size, max_seq_len, block_size, partition_size)


def pa_varlen_attn(out, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens, max_query_len,
                   max_seq_len, scale, workspace, causal=True, k_scale=None, v_scale=None,
                   partition_size=0, stream=None, window=0) -> None:
    """Attention of a flattened varlen batch; out/q [T][Hq][d], query_start_loc int32 [B+1].
    window > 0: sliding-window attention (pa_varlen_attn_windowed)."""
    nb, hkv, bs, d = cache_geometry(k_cache, v_cache, q.shape[-1])
    t, hq = q.shape[0], q.shape[1]
    b = seq_lens.numel()
    if q.dim() != 3 or q.shape[2] != d or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q/out must be [total_q_tokens][num_q_heads][head_size] of one dtype")
    if query_start_loc.dtype != torch.int32 or query_start_loc.numel() != b + 1:
        raise ValueError("query_start_loc must be int32 [num_seqs+1]")
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != b:
        raise ValueError("block_tables must be int32 [num_seqs][max_blocks_per_seq]")
    _check(_lib.pa_varlen_attn_windowed(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), nb, _ptr(block_tables),
                               block_tables.shape[1], _ptr(query_start_loc), _ptr(seq_lens), b, t,
                               int(max_query_len), int(max_seq_len), hq, hkv, d, bs, float(scale), int(window),
                               1 if causal else 0, dtype_code(q), kv_code(k_cache, k_scale), _ptr(k_scale),
                               _ptr(v_scale), int(partition_size), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "pa_varlen_attn")


def pa_diff_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len, block_size,
                                  partition_size=0) -> int:
    return _lib.pa_diff_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size, max_seq_len,
                                              block_size, partition_size)


def pa_diff_varlen_workspace_size(num_seqs, total_q_tokens, max_query_len, num_q_heads, num_kv_heads, head_size,
                                  max_seq_len, block_size, partition_size=0) -> int:
    return _lib.pa_diff_varlen_workspace_size(num_seqs, total_q_tokens, max_query_len, num_q_heads, num_kv_heads,
                                              head_size, max_seq_len, block_size, partition_size)


def _diff_bad(where, out, q, block_tables, seq_lens, lambda_, norm_weight, k_scale, v_scale, hkv):
    """Refuse a differential call: what _diff_args found wrong, named."""
    t, hq, d = q.shape
    if hq % 2 or hkv % 2 or out.shape != (t, hq // 2, 2 * d) or out.dtype is not q.dtype:
        raise ValueError(f"{where}: q must be [rows][num_q_heads][head_size] and out [rows][num_q_heads/2]"
                         "[2*head_size] of one dtype, with even numbers of heads and the caches' head size")
    if seq_lens.dtype is not _int32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        _bad(seq_lens, (seq_lens.numel(),), "seq_lens")
    if block_tables.dtype is not _int32 or block_tables.dim() != 2 or \
            block_tables.shape[0] != seq_lens.numel() or not block_tables.is_contiguous():
        raise ValueError(f"{where}: block_tables must be a contiguous int32 tensor [num_seqs][max_blocks_per_seq]")
    if lambda_.dtype is not _float32:
        raise ValueError(f"{where}: lambda must be float32: a number, [heads] or [rows][heads]")
    if norm_weight is not None and (norm_weight.dtype is not _float32 or norm_weight.shape != (2 * d,) or
                                    not norm_weight.is_contiguous()):
        raise ValueError(f"{where}: norm_weight must be a contiguous float32 tensor [2*head_size]")
    raise ValueError(f"{where}: q, out, the caches and the workspace must be contiguous, and all tensors on one "
                     "CUDA device")


def _diff_args(where, out, q, k_cache, v_cache, block_tables, seq_lens, lambda_, workspace, norm_weight, k_scale,
               v_scale):
    """Checks of a differential call's tensors; (rows, num_q_heads, sequences, geometry, lambda's
    strides, device)."""
    shape, dev = q.shape, q.get_device()
    if len(shape) != 3:
        raise ValueError(f"{where}: q must be [rows][num_q_heads][head_size]")
    t, hq, d = shape
    nb, hkv, bs, head = cache_geometry(k_cache, v_cache, d)
    lens, tables, lam = seq_lens.shape, block_tables.shape, lambda_.shape
    if head != d or hq % 2 or hkv % 2 or out.shape != (t, hq // 2, 2 * d) or out.dtype is not q.dtype or \
            len(lens) != 1 or len(tables) != 2 or tables[0] != lens[0] or seq_lens.dtype is not _int32 or \
            block_tables.dtype is not _int32 or lambda_.dtype is not _float32 or \
            not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and
                 seq_lens.is_contiguous() and block_tables.is_contiguous() and workspace.is_contiguous()) or \
            not (out.get_device() == k_cache.get_device() == v_cache.get_device() == block_tables.get_device() ==
                 seq_lens.get_device() == lambda_.get_device() == workspace.get_device() == dev) or \
            (norm_weight is not None and (norm_weight.dtype is not _float32 or norm_weight.shape != (2 * d,) or
                                          not norm_weight.is_contiguous() or norm_weight.get_device() != dev)):
        _diff_bad(where, out, q, block_tables, seq_lens, lambda_, norm_weight, k_scale, v_scale, hkv)
    row_stride = head_stride = 0
    n = len(lam)
    if n == 1 or n == 2:
        heads = lam[n - 1]
        if heads != 1:
            head_stride = lambda_.stride(n - 1)
        if n == 2 and lam[0] != 1:
            row_stride = lambda_.stride(0)
        if (heads != 1 and heads != hq // 2) or (n == 2 and lam[0] != 1 and lam[0] != t):
            raise ValueError(f"{where}: lambda must be a number, [heads] or [rows][heads]")
    elif n:
        raise ValueError(f"{where}: lambda must be a number, [heads] or [rows][heads]")
    code = kv_code(k_cache, k_scale)
    k_ptr = v_ptr = None
    if code >= PA_FP8_E4M3 and (k_scale is not None or v_scale is not None):
        if k_scale is None or v_scale is None or k_scale.dtype is not _float32 or v_scale.dtype is not _float32 or \
                v_scale.numel() != k_scale.numel() or k_scale.numel() not in (1, hkv) or \
                not (k_scale.is_contiguous() and v_scale.is_contiguous()) or \
                not k_scale.get_device() == v_scale.get_device() == dev:
            raise ValueError(f"{where}: scales: float32, both one per tensor or both one per KV head, on the caches' "
                             "device")
        k_ptr, v_ptr = k_scale.data_ptr(), v_scale.data_ptr()
    return t, hq, lens[0], nb, hkv, bs, d, row_stride, head_stride, dev, code, k_ptr, v_ptr


def pa_diff_decode(out, q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, scale, lambda_, workspace,
                   norm_weight=None, norm_eps=1e-5, k_scale=None, v_scale=None, partition_size=0, stream=None,
                   window=0) -> None:
    """Differential attention, one query a sequence: out [B][Hq/2][2d] = softmax(q[2h] K_1) V -
    lambda softmax(q[2h+1] K_2) V of q [B][Hq][d] on caches whose KV heads 2g, 2g+1 hold group g's
    two keys and its value's halves.  lambda_ float32: a number, [Hq/2] or [B][Hq/2] (any strides);
    norm_weight float32 [2d]: root-mean-square norm of every head.  See pa.h."""
    t, hq, b, nb, hkv, bs, d, row_stride, head_stride, dev, code, k_ptr, v_ptr = _diff_args(
        "pa_diff_decode", out, q, k_cache, v_cache, block_tables, seq_lens, lambda_, workspace, norm_weight, k_scale,
        v_scale)
    if t != b:
        raise ValueError("pa_diff_decode: one row of q a sequence")
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_diff_decode, out, q, k_cache, v_cache, block_tables, seq_lens, max_seq_len, scale,
                          lambda_, workspace, norm_weight, norm_eps, k_scale, v_scale, partition_size, stream, window)
    st = _lib.pa_diff_decode(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), b, max_seq_len, hq, hkv, d, bs, scale, lambda_.data_ptr(),
        row_stride, head_stride, None if norm_weight is None else norm_weight.data_ptr(), norm_eps, window,
        dtype_code(q), code, k_ptr, v_ptr, partition_size, workspace.data_ptr(), workspace.nbytes,
        _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_diff_decode"))
    if st != PA_OK:
        raise PAError(st, "pa_diff_decode")


def pa_diff_varlen_attn(out, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens, max_query_len, max_seq_len,
                        scale, lambda_, workspace, norm_weight=None, norm_eps=1e-5, causal=True, k_scale=None,
                        v_scale=None, partition_size=0, stream=None, window=0) -> None:
    """Differential attention of a flattened varlen batch (pa_diff_decode's heads, lambda and norm;
    q [T][Hq][d], query_start_loc int32 [B+1]).  See pa.h."""
    t, hq, b, nb, hkv, bs, d, row_stride, head_stride, dev, code, k_ptr, v_ptr = _diff_args(
        "pa_diff_varlen_attn", out, q, k_cache, v_cache, block_tables, seq_lens, lambda_, workspace, norm_weight,
        k_scale, v_scale)
    if query_start_loc.dtype is not _int32 or query_start_loc.shape != (b + 1,) or \
            not query_start_loc.is_contiguous() or query_start_loc.get_device() != dev:
        _bad(query_start_loc, (b + 1,), "query_start_loc")
    if dev < 0 or dev != _current_device():
        return _on_device(dev, pa_diff_varlen_attn, out, q, k_cache, v_cache, block_tables, query_start_loc, seq_lens,
                          max_query_len, max_seq_len, scale, lambda_, workspace, norm_weight, norm_eps, causal,
                          k_scale, v_scale, partition_size, stream, window)
    st = _lib.pa_diff_varlen_attn(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), nb, block_tables.data_ptr(),
        block_tables.shape[1], query_start_loc.data_ptr(), seq_lens.data_ptr(), b, t, max_query_len, max_seq_len, hq,
        hkv, d, bs, scale, lambda_.data_ptr(), row_stride, head_stride,
        None if norm_weight is None else norm_weight.data_ptr(), norm_eps, window, 1 if causal else 0, dtype_code(q),
        code, k_ptr, v_ptr, partition_size, workspace.data_ptr(), workspace.nbytes,
        _raw_stream(dev) if stream is None else _stream_on(stream, dev, "pa_diff_varlen_attn"))
    if st != PA_OK:
        raise PAError(st, "pa_diff_varlen_attn")


def pa_get_error_flags(clear: bool = True, stream=None) -> int:
    """Synchronise the stream and return the device error word (PA_ERRFLAG_* bits)."""
    flags = ctypes.c_uint32(0)
    st = _lib.pa_get_error_flags(ctypes.byref(flags), 1 if clear else 0, _stream(stream))
    if st not in (PA_OK, PA_ERR_BOUNDS, PA_ERR_TIMEOUT):
        _check(st, "pa_get_error_flags")
    return int(flags.value)


def pa_trace_enable(on: bool) -> None:
    _check(_lib.pa_trace_enable(1 if on else 0), "pa_trace_enable")


def pa_trace_read(kind: int, reset: bool = False):
    """(launches, total device ms) of one kernel kind since the last reset."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check(_lib.pa_trace_read(kind, ctypes.byref(n), ctypes.byref(ms), 1 if reset else 0), "pa_trace_read")
    return int(n.value), float(ms.value)


def workspace_tensor(nbytes: int, device=None) -> torch.Tensor:
    """A device byte buffer suitable as `workspace` (torch allocations are 256-byte aligned)."""
    return torch.empty(int(nbytes), dtype=torch.uint8, device="cuda" if device is None else device)
