"""Thin Python binding over libpa_gb300.so (the C ABI in include/pa.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, checks shapes and dtypes, and passes raw device pointers,
element strides and the current CUDA stream to the C entry point of the same
name.  All arithmetic runs in the library's sm_103a kernels; there is no
fallback path.  Importing this module loads the library and raises if it has
not been built (``python -m paged_kv_continuous_gb300.build``).

A call is enqueued on ``stream`` (default: the current stream), and an output
or workspace that it allocates because none was given belongs to that stream,
as if made under ``torch.cuda.stream(stream)``: wait for the stream before using
it on another, and tell the allocator (``record_stream``) of any but the one
that was current at the call.  The prepared calls (``*Call``) allocate on the
stream that is current when they are made; the first call on another stream
makes that one wait for it, which a call under capture cannot: make the call
object before the capture, capture behind a synchronize (as ``torch.cuda.graph``
does), and keep the object as long as the graph.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libpa_gb300.so")

PA_OK = 0
PA_DTYPE_BF16 = 0
PA_DTYPE_F32 = 1
PA_LAUNCH_PDL = 1  # programmatic dependent launch (see include/pa.h)
PA_LAUNCH_EARLY_KV = 2  # decode: K/V pages requested before the previous kernel completes
PA_COPY_BEFORE_WAIT = 4  # pa_copy: the bytes move before the previous kernel completes
DEVERR_BLOCK_INDEX = 1
DEVERR_SLOT_INDEX = 2
DEVERR_WAIT_TIMEOUT = 4
DEVERR_SHAPE = 8
DEVERR_POSITION = 16
DEVERR_PAGES = 32

EXPORTED = (
    "pa_abi_version", "pa_status_string", "pa_store_kv", "pa_decode_workspace_size",
    "pa_decode_default_splits", "pa_decode", "pa_decode_merge", "pa_prefill_varlen",
    "pa_decode_noalloc", "pa_rope_store_kv", "pa_store_kv_fp8", "pa_decode_fp8",
    "pa_store_decode", "pa_store_decode_fp8", "pa_prefill_store_varlen",
    "pa_rope_store_decode", "pa_get_device_error", "pa_copy", "pa_store_kv_fp8_block",
    "pa_decode_fp8_block", "pa_copy_pages", "pa_fork_pages", "pa_free_pages",
    "pa_compact_pages", "pa_prefill_fp8_block",
)


class PagedAttentionError(RuntimeError):
    pass


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise PagedAttentionError(
            f"{path} is missing: build it with `python -m paged_kv_continuous_gb300.build`")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz, u32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                 ctypes.c_float, ctypes.c_size_t, ctypes.c_uint32)
    lib.pa_abi_version.restype = i32
    lib.pa_abi_version.argtypes = []
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_status_string.argtypes = [i32]
    lib.pa_get_device_error.restype = i32
    lib.pa_get_device_error.argtypes = [P, P, i32, P]
    lib.pa_copy.restype = i32
    lib.pa_copy.argtypes = [P, P, i64, u32, P]
    lib.pa_store_kv.restype = i32
    lib.pa_store_kv.argtypes = [P, P, i64, i64, i64, i64, i64, P, P, i64, i32, i32, i32, P, P,
                                u32, P]
    lib.pa_rope_store_kv.restype = i32
    lib.pa_rope_store_kv.argtypes = [P, i64, P, i64, P, i64, P, i64, i64, i32, i32, i32, P, P,
                                     P, i64, P, P, i64, i32, P, P, u32, P]
    lib.pa_decode_workspace_size.restype = sz
    lib.pa_decode_workspace_size.argtypes = [i32, i32, i32]
    lib.pa_decode_default_splits.restype = i32
    lib.pa_decode_default_splits.argtypes = [i32, i32, i32]
    lib.pa_decode.restype = i32
    lib.pa_decode.argtypes = [P, i32, P, P, P, i64, P, i32, P, i32, i32, i32, i32, i32, f32,
                              i32, P, sz, u32, P]
    lib.pa_store_decode.restype = i32
    lib.pa_store_decode.argtypes = [P, i32, P, P, P, i64, i64, P, P, P, i64, P, i32, P, i32,
                                    i32, i32, i32, i32, f32, i32, P, sz, u32, P]
    lib.pa_rope_store_decode.restype = i32
    lib.pa_rope_store_decode.argtypes = [P, i32, P, P, P, i64, i64, P, P, P, i64, P, P, P, i64,
                                         P, i32, P, i32, i32, i32, i32, i32, f32, i32, P, sz,
                                         u32, P]
    lib.pa_store_decode_fp8.restype = i32
    lib.pa_store_decode_fp8.argtypes = [P, i32, P, P, P, i64, i64, P, P, P, P, P, i64, P, i32,
                                        P, i32, i32, i32, i32, i32, f32, i32, P, sz, u32, P]
    lib.pa_decode_fp8.restype = i32
    lib.pa_decode_fp8.argtypes = [P, i32, P, P, P, P, P, i64, P, i32, P, i32, i32, i32, i32,
                                  i32, f32, i32, P, sz, u32, P]
    lib.pa_store_kv_fp8.restype = i32
    lib.pa_store_kv_fp8.argtypes = [P, P, i64, i64, i64, i64, i64, P, P, P, P, i64, i32, i32,
                                    i32, P, P, u32, P]
    lib.pa_store_kv_fp8_block.restype = i32
    lib.pa_store_kv_fp8_block.argtypes = [P, P, i64, i64, i64, i64, P, i32, i32, P, P, P, P, i64,
                                          i32, i32, i32, P, i32, P, P, u32, P]
    lib.pa_decode_fp8_block.restype = i32
    lib.pa_decode_fp8_block.argtypes = [P, i32, P, P, P, P, P, i64, P, i32, P, i32, i32, i32,
                                        i32, i32, f32, i32, P, sz, u32, P]
    lib.pa_prefill_fp8_block.restype = i32
    lib.pa_prefill_fp8_block.argtypes = [P, i32, P, P, i32, i32, i32, P, P, P, P, i64, P, i32, P,
                                         i32, i32, i32, i32, f32, P, P]
    lib.pa_copy_pages.restype = i32
    lib.pa_copy_pages.argtypes = [P, i32, i64, P, P, i32, P, P, u32, P]
    lib.pa_fork_pages.restype = i32
    lib.pa_fork_pages.argtypes = [P, i32, P, i32, P, P, i32, P, i64, i32, P, P, P, P, u32, P]
    lib.pa_free_pages.restype = i32
    lib.pa_free_pages.argtypes = [P, i32, P, i32, P, i32, P, i64, i32, P, u32, P]
    lib.pa_compact_pages.restype = i32
    lib.pa_compact_pages.argtypes = [P, i32, P, i32, P, i64, i32, P, P, P, P, P, u32, P]
    lib.pa_decode_merge.restype = i32
    lib.pa_decode_merge.argtypes = [P, i32, P, sz, P, i32, i32, i32, i32, i32, P]
    lib.pa_decode_noalloc.restype = i32
    lib.pa_decode_noalloc.argtypes = [P, i32, P, P, P, i64, P, i32, P, i32, i32, i32, i32, i32,
                                      f32, i32, P, u32, P]
    lib.pa_prefill_varlen.restype = i32
    lib.pa_prefill_varlen.argtypes = [P, i32, P, P, i32, i32, i32, P, P, i64, P, i32, P, i32,
                                      i32, i32, i32, f32, P, P]
    lib.pa_prefill_store_varlen.restype = i32
    lib.pa_prefill_store_varlen.argtypes = [P, i32, P, P, P, i64, i64, P, P, i32, i32, i32, P,
                                            P, i64, P, i32, P, i32, i32, i32, i32, f32, P, P]
    return lib


lib = load_library()


def _check(status: int, what: str):
    if status != PA_OK:
        raise PagedAttentionError(f"{what}: {lib.pa_status_string(status).decode()} ({status})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class _on:
    """Where a call on ``stream`` allocates its default buffers: on that stream,
    so that filling, use and reuse of their memory follow one another.  Gives a
    function for those that the caller gets, which also tells the allocator of
    the stream that is current outside."""

    def __init__(self, stream):
        self._stream = stream

    def __enter__(self):
        if self._stream is not None:
            self._outside = torch.cuda.current_stream()
            self._inside = torch.cuda.stream(self._stream)
            self._inside.__enter__()
        return self._handed

    def __exit__(self, *exc):
        if self._stream is not None:
            self._inside.__exit__(*exc)

    def _handed(self, t):
        if self._stream is not None and self._outside != self._stream and \
                self._outside.device == t.device:
            t.record_stream(self._outside)
        return t


class _Defaults:
    """The buffers that a prepared call made for itself, on the stream that was
    current then.  Another stream that it is called on waits for that one
    (which may still fill them, or run what had their memory before), once, and
    the allocator is told of the stream."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        self.home = torch.cuda.current_stream(self.tensors[0].device)
        self.known = {self.home.cuda_stream}

    def share(self, stream):
        for t in self.tensors:
            t.record_stream(stream)
        if _capturing(stream) or _capturing(self.home):
            return  # the wait would become part of the capture, or break it
        stream.wait_stream(self.home)
        self.known.add(stream.cuda_stream)


def _capturing(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _need(t, dtype, name, dims=None):
    if not t.is_cuda:
        raise PagedAttentionError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise PagedAttentionError(f"{name} must be {dtype}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise PagedAttentionError(f"{name} must have {dims} dims, got {tuple(t.shape)}")


def _out_code(dtype):
    if dtype == torch.bfloat16:
        return PA_DTYPE_BF16
    if dtype == torch.float32:
        return PA_DTYPE_F32
    raise PagedAttentionError(f"unsupported output dtype {dtype}")


def store_kv(k, v, k_cache, v_cache, slot_mapping, error_flags=None, stream=None, pdl=False):
    """pa_store_kv: k/v bf16 [T, Hkv, D] (any token/head strides, unit dim
    stride) into the pools at slot_mapping (int32 [T]).  pdl: launch with
    PA_LAUNCH_PDL."""
    _need(k, torch.bfloat16, "k", 3)
    _need(v, torch.bfloat16, "v", 3)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise PagedAttentionError("k/v need a unit stride along head_dim")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise PagedAttentionError("pools must be contiguous")
    T, Hkv, D = k.shape
    NB, bs, Hkv2, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or v.shape != k.shape or v_cache.shape != k_cache.shape:
        raise PagedAttentionError("shape mismatch between k/v and the pools")
    if slot_mapping.shape[0] != T:
        raise PagedAttentionError("slot_mapping must have one entry per token")
    _check(lib.pa_store_kv(_ptr(k), _ptr(v), T, k.stride(0), k.stride(1), v.stride(0),
                           v.stride(1), _ptr(k_cache), _ptr(v_cache), NB, bs, Hkv, D,
                           _ptr(slot_mapping), _ptr(error_flags),
                           PA_LAUNCH_PDL if pdl else 0, _stream(stream)),
           "pa_store_kv")


def rope_store_kv(q, k, v, positions, cos_table, sin_table, k_cache, v_cache, slot_mapping,
                  q_out=None, error_flags=None, stream=None, pdl=False):
    """pa_rope_store_kv: rotate q (bf16 [T, Hq, D]) into q_out (new tensor,
    or q itself for in place) and k (bf16 [T, Hkv, D]) by the rotary tables
    (float32 [max_position, D/2]) at positions (int32 [T]); store the rotated
    k and the plain v at slot_mapping.  q/k/v may be views of a fused QKV
    buffer (any token stride; heads contiguous).  Returns q_out."""
    for t, n, d in ((q, "q", 3), (k, "k", 3), (v, "v", 3)):
        _need(t, torch.bfloat16, n, d)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise PagedAttentionError(f"{n} needs contiguous heads ([T, H, D], unit dim stride)")
    _need(positions, torch.int32, "positions", 1)
    _need(cos_table, torch.float32, "cos_table", 2)
    _need(sin_table, torch.float32, "sin_table", 2)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise PagedAttentionError("pools must be contiguous")
    if not (cos_table.is_contiguous() and sin_table.is_contiguous()):
        raise PagedAttentionError("rotary tables must be contiguous")
    T, Hq, D = q.shape
    _, Hkv, _ = k.shape
    NB, bs, Hkv2, D2 = k_cache.shape
    if k.shape != (T, Hkv, D) or v.shape != k.shape or (Hkv2, D2) != (Hkv, D) or \
            v_cache.shape != k_cache.shape:
        raise PagedAttentionError("shape mismatch between q/k/v and the pools")
    if cos_table.shape != sin_table.shape or cos_table.shape[1] != D // 2:
        raise PagedAttentionError("rotary tables must be [max_position, head_dim / 2]")
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise PagedAttentionError("positions and slot_mapping need one entry per token")
    if q_out is None:
        with _on(stream) as handed:
            q_out = handed(torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device))
    _need(q_out, torch.bfloat16, "q_out", 3)
    if q_out.shape != q.shape or q_out.stride(2) != 1 or q_out.stride(1) != D:
        raise PagedAttentionError("q_out must be [T, Hq, D] with contiguous heads")
    _check(lib.pa_rope_store_kv(_ptr(q), q.stride(0), _ptr(q_out), q_out.stride(0), _ptr(k),
                                k.stride(0), _ptr(v), v.stride(0), T, Hq, Hkv, D,
                                _ptr(positions), _ptr(cos_table), _ptr(sin_table),
                                cos_table.shape[0], _ptr(k_cache), _ptr(v_cache), NB, bs,
                                _ptr(slot_mapping), _ptr(error_flags),
                                PA_LAUNCH_PDL if pdl else 0, _stream(stream)),
           "pa_rope_store_kv")
    return q_out


def _device_index(device=None) -> int:
    if device is None:
        return torch.cuda.current_device()
    if isinstance(device, torch.device):
        return device.index if device.index is not None else torch.cuda.current_device()
    if isinstance(device, str):
        return _device_index(torch.device(device))
    return int(device)


def default_splits(num_q_heads: int, num_kv_heads: int, device=None) -> int:
    return int(lib.pa_decode_default_splits(_device_index(device), num_q_heads, num_kv_heads))


def decode_workspace(num_q_heads: int, num_kv_heads: int, num_splits: int = 0,
                     head_dim: int = 128, device=None):
    """A zeroed workspace for pa_decode (error word and counters start at zero)."""
    s = num_splits if num_splits > 0 else default_splits(num_q_heads, num_kv_heads, device)
    n = int(lib.pa_decode_workspace_size(s, num_q_heads, head_dim))
    if n == 0:
        raise PagedAttentionError("bad workspace request")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _decode_flags(pdl, early_kv):
    """Launch flags of the decode entry points.  early_kv (with pdl): the
    kernel requests its first K/V pages before the kernel launched just
    before it completes, so that kernel must not write the pools."""
    if early_kv and not pdl:
        raise PagedAttentionError("early_kv needs pdl")
    return (PA_LAUNCH_PDL if pdl else 0) | (PA_LAUNCH_EARLY_KV if early_kv else 0)


def decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
           out_dtype=torch.bfloat16, num_splits=0, workspace=None, stream=None, pdl=False,
           early_kv=False):
    """pa_decode: q bf16 [B, Hq, D] over the paged pools; returns out [B, Hq, D].
    pdl: launch with PA_LAUNCH_PDL (context_lens and block_tables must then
    not be written by the kernel launched just before).  early_kv (with pdl):
    PA_LAUNCH_EARLY_KV, the first K/V pages are requested before that kernel
    completes, so it must not write k_cache / v_cache either."""
    _need(q, torch.bfloat16, "q", 3)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    if not q.is_contiguous():
        raise PagedAttentionError("q must be contiguous")
    if block_tables.stride(1) != 1:
        raise PagedAttentionError("block_tables rows must be contiguous")
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    with _on(stream) as handed:
        if out is None:
            out = handed(torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
    _check(lib.pa_decode(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(k_cache),
                         _ptr(v_cache), NB, _ptr(block_tables), block_tables.stride(0),
                         _ptr(context_lens), B, Hq, Hkv, D, bs, float(scale), int(num_splits),
                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                         _decode_flags(pdl, early_kv), _stream(stream)), "pa_decode")
    return out


def store_decode(q, new_k, new_v, k_cache, v_cache, slot_mapping, block_tables, context_lens,
                 scale, out=None, out_dtype=torch.bfloat16, num_splits=0, workspace=None,
                 stream=None, pdl=False, early_kv=False):
    """pa_store_decode: one decode step in one kernel -- each sequence's new
    token (new_k / new_v bf16 [B, Hkv, D], heads contiguous) is stored at
    slot_mapping[b] and attended with the rest of the pool.  Returns out."""
    _need(q, torch.bfloat16, "q", 3)
    _need(new_k, torch.bfloat16, "new_k", 3)
    _need(new_v, torch.bfloat16, "new_v", 3)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    if not q.is_contiguous():
        raise PagedAttentionError("q must be contiguous")
    for t, n in ((new_k, "new_k"), (new_v, "new_v")):
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise PagedAttentionError(f"{n} needs contiguous heads")
    if block_tables.stride(1) != 1:
        raise PagedAttentionError("block_tables rows must be contiguous")
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    if tuple(new_k.shape) != (B, Hkv, D) or new_v.shape != new_k.shape or \
            slot_mapping.shape[0] != B:
        raise PagedAttentionError("new_k / new_v / slot_mapping need one row per sequence")
    with _on(stream) as handed:
        if out is None:
            out = handed(torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
    _check(lib.pa_store_decode(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(new_k),
                               _ptr(new_v), new_k.stride(0), new_v.stride(0), _ptr(slot_mapping),
                               _ptr(k_cache), _ptr(v_cache), NB, _ptr(block_tables),
                               block_tables.stride(0), _ptr(context_lens), B, Hq, Hkv, D, bs,
                               float(scale), int(num_splits), _ptr(workspace),
                               workspace.numel() * workspace.element_size(),
                               _decode_flags(pdl, early_kv), _stream(stream)),
           "pa_store_decode")
    return out


class StoreDecodeCall:
    """A prepared pa_store_decode: the tensors are checked once and the
    marshalled arguments kept, so each call is one foreign call.  The caller
    updates the tensors' contents in place between calls (as with the static
    buffers of a captured step) and keeps them alive; ``call(stream)`` then
    enqueues the step on ``stream`` (default: the current stream)."""

    def __init__(self, q, new_k, new_v, k_cache, v_cache, slot_mapping, block_tables,
                 context_lens, scale, out, num_splits=0, workspace=None, pdl=False,
                 early_kv=False):
        _need(q, torch.bfloat16, "q", 3)
        _need(new_k, torch.bfloat16, "new_k", 3)
        _need(new_v, torch.bfloat16, "new_v", 3)
        _need(k_cache, torch.bfloat16, "k_cache", 4)
        _need(v_cache, torch.bfloat16, "v_cache", 4)
        _need(slot_mapping, torch.int32, "slot_mapping", 1)
        _need(block_tables, torch.int32, "block_tables", 2)
        _need(context_lens, torch.int32, "context_lens", 1)
        if not q.is_contiguous():
            raise PagedAttentionError("q must be contiguous")
        for t, n in ((new_k, "new_k"), (new_v, "new_v")):
            if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
                raise PagedAttentionError(f"{n} needs contiguous heads")
        if block_tables.stride(1) != 1:
            raise PagedAttentionError("block_tables rows must be contiguous")
        B, Hq, D = q.shape
        NB, bs, Hkv, _ = k_cache.shape
        if tuple(new_k.shape) != (B, Hkv, D) or new_v.shape != new_k.shape or \
                slot_mapping.shape[0] != B:
            raise PagedAttentionError("new_k / new_v / slot_mapping need one row per sequence")
        if out.shape != (B, Hq, D) or not out.is_contiguous():
            raise PagedAttentionError("out must be a contiguous [B, Hq, D] tensor")
        self._defaults = None
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
            self._defaults = _Defaults([workspace])
        self._keep = (q, new_k, new_v, k_cache, v_cache, slot_mapping, block_tables,
                      context_lens, out, workspace)
        c = ctypes
        self._args = (
            c.c_void_p(out.data_ptr()), c.c_int32(_out_code(out.dtype)), c.c_void_p(q.data_ptr()),
            c.c_void_p(new_k.data_ptr()), c.c_void_p(new_v.data_ptr()),
            c.c_int64(new_k.stride(0)), c.c_int64(new_v.stride(0)),
            c.c_void_p(slot_mapping.data_ptr()), c.c_void_p(k_cache.data_ptr()),
            c.c_void_p(v_cache.data_ptr()), c.c_int64(NB), c.c_void_p(block_tables.data_ptr()),
            c.c_int32(block_tables.stride(0)), c.c_void_p(context_lens.data_ptr()), c.c_int32(B),
            c.c_int32(Hq), c.c_int32(Hkv), c.c_int32(D), c.c_int32(bs), c.c_float(scale),
            c.c_int32(num_splits), c.c_void_p(workspace.data_ptr()),
            c.c_size_t(workspace.numel() * workspace.element_size()),
            c.c_uint32(_decode_flags(pdl, early_kv)))
        self.out = out
        self.workspace = workspace

    def __call__(self, stream=None):
        if self._defaults is not None:
            s = torch.cuda.current_stream(self.workspace.device) if stream is None else stream
            if s.cuda_stream not in self._defaults.known:
                self._defaults.share(s)
        st = lib.pa_store_decode(*self._args, _stream(stream))
        if st != PA_OK:
            _check(st, "pa_store_decode")
        return self.out


class CopyCall:
    """A prepared pa_copy (dst <- src, checked once, as ``copy`` checks)."""

    def __init__(self, dst, src, pdl=False, before_wait=False):
        nbytes, flags = _copy_check(dst, src, pdl, before_wait)
        self._keep = (dst, src)
        self._args = (ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()),
                      ctypes.c_int64(nbytes), ctypes.c_uint32(flags))

    def __call__(self, stream=None):
        st = lib.pa_copy(*self._args, _stream(stream))
        if st != PA_OK:
            _check(st, "pa_copy")


def _copy_check(dst, src, pdl, before_wait):
    for t, n in ((dst, "dst"), (src, "src")):
        if not (t.is_cuda or t.is_pinned()):
            raise PagedAttentionError(f"{n} must be a CUDA tensor or pinned host memory")
        if not t.is_contiguous():
            raise PagedAttentionError(f"{n} must be contiguous")
    nbytes = dst.numel() * dst.element_size()
    if nbytes != src.numel() * src.element_size():
        raise PagedAttentionError("dst and src differ in size")
    if before_wait and not pdl:
        raise PagedAttentionError("before_wait needs pdl")
    return nbytes, (PA_LAUNCH_PDL if pdl else 0) | (PA_COPY_BEFORE_WAIT if before_wait else 0)


def copy(dst, src, pdl=False, before_wait=False, stream=None):
    """pa_copy: dst <- src (tensors of the same byte size, contiguous; each on
    the GPU or in pinned host memory).  pdl: launch with PA_LAUNCH_PDL;
    before_wait (with pdl): PA_COPY_BEFORE_WAIT, the bytes move before the
    kernel launched just before completes (it must not write src nor touch
    dst)."""
    nbytes, flags = _copy_check(dst, src, pdl, before_wait)
    _check(lib.pa_copy(_ptr(dst), _ptr(src), nbytes, flags, _stream(stream)), "pa_copy")


def rope_store_decode(q, new_k, new_v, k_cache, v_cache, slot_mapping, block_tables,
                      context_lens, scale, positions, cos_table, sin_table, out=None,
                      out_dtype=torch.bfloat16, num_splits=0, workspace=None, stream=None,
                      pdl=False, early_kv=False):
    """pa_rope_store_decode: store_decode with the rotary embedding of q and
    the new K rows at positions (int32 [B]) from cos_table / sin_table
    (float32 [max_position, D/2]).  q is not written.  Returns out."""
    _need(q, torch.bfloat16, "q", 3)
    _need(new_k, torch.bfloat16, "new_k", 3)
    _need(new_v, torch.bfloat16, "new_v", 3)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    _need(positions, torch.int32, "positions", 1)
    _need(cos_table, torch.float32, "cos_table", 2)
    _need(sin_table, torch.float32, "sin_table", 2)
    if not q.is_contiguous():
        raise PagedAttentionError("q must be contiguous")
    for t, n in ((new_k, "new_k"), (new_v, "new_v")):
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise PagedAttentionError(f"{n} needs contiguous heads")
    if block_tables.stride(1) != 1:
        raise PagedAttentionError("block_tables rows must be contiguous")
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    if tuple(new_k.shape) != (B, Hkv, D) or new_v.shape != new_k.shape or \
            slot_mapping.shape[0] != B or positions.shape[0] != B:
        raise PagedAttentionError(
            "new_k / new_v / slot_mapping / positions need one row per sequence")
    if cos_table.shape != sin_table.shape or cos_table.shape[1] != D // 2 or \
            not cos_table.is_contiguous() or not sin_table.is_contiguous():
        raise PagedAttentionError("cos_table / sin_table must be contiguous [max_position, D/2]")
    with _on(stream) as handed:
        if out is None:
            out = handed(torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
    _check(lib.pa_rope_store_decode(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(new_k),
                                    _ptr(new_v), new_k.stride(0), new_v.stride(0),
                                    _ptr(positions), _ptr(cos_table), _ptr(sin_table),
                                    cos_table.shape[0], _ptr(slot_mapping), _ptr(k_cache),
                                    _ptr(v_cache), NB, _ptr(block_tables),
                                    block_tables.stride(0), _ptr(context_lens), B, Hq, Hkv, D, bs,
                                    float(scale), int(num_splits), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _decode_flags(pdl, early_kv), _stream(stream)),
           "pa_rope_store_decode")
    return out


def fp8_pools(num_blocks, num_kv_heads, head_dim=128, block_size=16, device=None):
    """Empty FP8 pools: K uint8 [NB, bs, Hkv, D] (token-major), V uint8
    [NB, Hkv, D, bs] (dim-major inside a block)."""
    k = torch.empty((num_blocks, block_size, num_kv_heads, head_dim), dtype=torch.uint8,
                    device=device)
    v = torch.empty((num_blocks, num_kv_heads, head_dim, block_size), dtype=torch.uint8,
                    device=device)
    return k, v


def _need_fp8_pools(k_cache, v_cache, k_scale, v_scale):
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    _need(k_scale, torch.float32, "k_scale", 1)
    _need(v_scale, torch.float32, "v_scale", 1)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise PagedAttentionError("pools must be contiguous")
    NB, bs, Hkv, D = k_cache.shape
    if tuple(v_cache.shape) != (NB, Hkv, D, bs):
        raise PagedAttentionError("FP8 V pool must be [num_blocks, Hkv, D, block_size]")
    if k_scale.shape[0] != Hkv or v_scale.shape[0] != Hkv:
        raise PagedAttentionError("k_scale / v_scale need one entry per kv head")
    return NB, bs, Hkv, D


def store_kv_fp8(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, error_flags=None,
                 stream=None, pdl=False):
    """pa_store_kv_fp8: quantise k/v bf16 [T, Hkv, D] (any token/head
    strides) into the FP8 pools (see fp8_pools) at slot_mapping."""
    _need(k, torch.bfloat16, "k", 3)
    _need(v, torch.bfloat16, "v", 3)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise PagedAttentionError("k/v need a unit stride along head_dim")
    NB, bs, Hkv, D = _need_fp8_pools(k_cache, v_cache, k_scale, v_scale)
    T = k.shape[0]
    if tuple(k.shape) != (T, Hkv, D) or v.shape != k.shape or slot_mapping.shape[0] != T:
        raise PagedAttentionError("shape mismatch between k/v, the pools and slot_mapping")
    _check(lib.pa_store_kv_fp8(_ptr(k), _ptr(v), T, k.stride(0), k.stride(1), v.stride(0),
                               v.stride(1), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                               _ptr(v_scale), NB, bs, Hkv, D, _ptr(slot_mapping),
                               _ptr(error_flags), PA_LAUNCH_PDL if pdl else 0, _stream(stream)),
           "pa_store_kv_fp8")


def decode_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
               out=None, out_dtype=torch.bfloat16, num_splits=0, workspace=None, stream=None,
               pdl=False, early_kv=False):
    """pa_decode_fp8: q bf16 [B, Hq, D] over the FP8 pools with per-kv-head
    scales; returns out [B, Hq, D]."""
    _need(q, torch.bfloat16, "q", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    if not q.is_contiguous():
        raise PagedAttentionError("q must be contiguous")
    if block_tables.stride(1) != 1:
        raise PagedAttentionError("block_tables rows must be contiguous")
    NB, bs, Hkv, _ = _need_fp8_pools(k_cache, v_cache, k_scale, v_scale)
    B, Hq, D = q.shape
    with _on(stream) as handed:
        if out is None:
            out = handed(torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
    _check(lib.pa_decode_fp8(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(k_cache),
                             _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), NB,
                             _ptr(block_tables), block_tables.stride(0), _ptr(context_lens), B,
                             Hq, Hkv, D, bs, float(scale), int(num_splits), _ptr(workspace),
                             workspace.numel() * workspace.element_size(),
                             _decode_flags(pdl, early_kv), _stream(stream)), "pa_decode_fp8")
    return out


def store_decode_fp8(q, new_k, new_v, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                     block_tables, context_lens, scale, out=None, out_dtype=torch.bfloat16,
                     num_splits=0, workspace=None, stream=None, pdl=False,
                     early_kv=False):
    """pa_store_decode_fp8: store_decode over FP8 pools (see fp8_pools)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(new_k, torch.bfloat16, "new_k", 3)
    _need(new_v, torch.bfloat16, "new_v", 3)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    if not q.is_contiguous():
        raise PagedAttentionError("q must be contiguous")
    for t, n in ((new_k, "new_k"), (new_v, "new_v")):
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise PagedAttentionError(f"{n} needs contiguous heads")
    if block_tables.stride(1) != 1:
        raise PagedAttentionError("block_tables rows must be contiguous")
    NB, bs, Hkv, _ = _need_fp8_pools(k_cache, v_cache, k_scale, v_scale)
    B, Hq, D = q.shape
    if tuple(new_k.shape) != (B, Hkv, D) or new_v.shape != new_k.shape or \
            slot_mapping.shape[0] != B:
        raise PagedAttentionError("new_k / new_v / slot_mapping need one row per sequence")
    with _on(stream) as handed:
        if out is None:
            out = handed(torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
    _check(lib.pa_store_decode_fp8(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(new_k),
                                   _ptr(new_v), new_k.stride(0), new_v.stride(0),
                                   _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(k_scale), _ptr(v_scale), NB, _ptr(block_tables),
                                   block_tables.stride(0), _ptr(context_lens), B, Hq, Hkv, D, bs,
                                   float(scale), int(num_splits), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _decode_flags(pdl, early_kv), _stream(stream)),
           "pa_store_decode_fp8")
    return out


# A device's current stream (as an address) and the current device, without
# the wrapper objects that torch.cuda builds around them on every call
_raw_stream = torch._C._cuda_getCurrentRawStream if torch.cuda.is_available() else None
_current_device = torch._C._cuda_getDevice if torch.cuda.is_available() else None


class _Prepared:
    """A prepared call: the tensors are checked once and the marshalled
    arguments kept, so each call is one foreign call.  The caller updates the
    tensors' contents in place between calls and keeps their storage; the
    call is enqueued on ``stream`` (default: the current stream of the
    tensors' device, which also becomes the device of the launch)."""

    def _prepare(self, fn, what, args, keep, result=None, made=()):
        """made: the tensors among ``keep`` that the call allocated itself."""
        self._fn, self._what, self._keep, self._result = fn, what, keep, result
        # (pinned host memory, which the device reaches, counts for none)
        devices = {t.device for t in keep if t is not None and t.is_cuda}
        if len(devices) != 1:
            raise PagedAttentionError(f"{what}: tensors on different devices")
        self._device = devices.pop().index
        # marshalled once: a call converts nothing but the stream
        self._args = tuple(a if t is None else t(a) for a, t in zip(args, fn.argtypes))
        self._defaults = _Defaults(made) if made else None

    def __call__(self, stream=None):
        handle = _raw_stream(self._device) if stream is None else stream.cuda_stream
        if self._defaults is not None and handle not in self._defaults.known:
            self._defaults.share(torch.cuda.current_stream(self._device) if stream is None
                                 else stream)
        if _current_device() == self._device:
            status = self._fn(*self._args, handle)
        else:
            with torch.cuda.device(self._device):
                status = self._fn(*self._args, handle)
        if status != PA_OK:
            _check(status, self._what)
        return self._result


def _address(t):
    return None if t is None else t.data_ptr()


def _need_contiguous(t, dtype, name, shape=None, dims=None):
    _need(t, dtype, name, dims)
    if not t.is_contiguous():
        raise PagedAttentionError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise PagedAttentionError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _need_error_flags(t):
    if t is not None:
        _need(t, torch.int32, "error_flags")
        if t.numel() < 1:
            raise PagedAttentionError("error_flags must hold an int32 word")


def _need_table_rows(block_tables):
    """Contiguous rows that do not overlap, the last one with room for a whole
    row stride (the kernels know a row by its stride)."""
    _need(block_tables, torch.int32, "block_tables", 2)
    rows, width = block_tables.shape
    if not rows:
        return
    step = block_tables.stride(0)
    if width < 1 or (width > 1 and block_tables.stride(1) != 1) or step < width:
        raise PagedAttentionError("block_tables rows must be contiguous and apart")
    if 4 * (block_tables.storage_offset() + rows * step) > block_tables.untyped_storage().nbytes():
        raise PagedAttentionError("block_tables needs room for its last row's whole stride")


def _need_tables(block_tables, context_lens, batch):
    _need_table_rows(block_tables)
    _need_contiguous(context_lens, torch.int32, "context_lens", (batch,))
    if block_tables.shape[0] < batch:
        raise PagedAttentionError("block_tables needs one row per sequence")


def fp8_block_pools(num_blocks, num_kv_heads, head_dim=128, block_size=16, device=None):
    """Empty block-scaled FP8 pools: K and V as ``fp8_pools``, and the scale
    bytes k_scale / v_scale (uint8 [NB, Hkv], biased exponents)."""
    k, v = fp8_pools(num_blocks, num_kv_heads, head_dim, block_size, device)
    ks, vs = (torch.empty((num_blocks, num_kv_heads), dtype=torch.uint8, device=device)
              for _ in range(2))
    return k, v, ks, vs


def _need_fp8_block_pools(k_cache, v_cache, k_scale, v_scale):
    _need_contiguous(k_cache, torch.uint8, "k_cache", dims=4)
    NB, bs, Hkv, D = k_cache.shape
    _need_contiguous(v_cache, torch.uint8, "v_cache", (NB, Hkv, D, bs))
    _need_contiguous(k_scale, torch.uint8, "k_scale", (NB, Hkv))
    _need_contiguous(v_scale, torch.uint8, "v_scale", (NB, Hkv))
    return NB, bs, Hkv, D


class StoreKvFp8BlockCall(_Prepared):
    """A prepared pa_store_kv_fp8_block (arguments as ``store_kv_fp8_block``)."""

    def __init__(self, k, v, k_cache, v_cache, k_scale, v_scale, cu_seqlens, block_tables,
                 context_lens, error_flags=None, pdl=False):
        NB, bs, Hkv, D = _need_fp8_block_pools(k_cache, v_cache, k_scale, v_scale)
        _need(k, torch.bfloat16, "k", 3)
        _need(v, torch.bfloat16, "v", 3)
        if tuple(k.shape[1:]) != (Hkv, D) or v.shape != k.shape:
            raise PagedAttentionError("shape mismatch between k/v and the pools")
        if k.numel() and (k.stride(2) != 1 or v.stride(2) != 1):
            raise PagedAttentionError("k/v need a unit stride along head_dim")
        _need_contiguous(cu_seqlens, torch.int32, "cu_seqlens", dims=1)
        B = cu_seqlens.shape[0] - 1
        if B < 0:
            raise PagedAttentionError("cu_seqlens needs num_seqs + 1 entries")
        _need_tables(block_tables, context_lens, B)
        _need_error_flags(error_flags)
        self._prepare(
            lib.pa_store_kv_fp8_block, "pa_store_kv_fp8_block",
            (_address(k), _address(v), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
             _address(cu_seqlens), B, k.shape[0], _address(k_cache), _address(v_cache),
             _address(k_scale), _address(v_scale), NB, bs, Hkv, D, _address(block_tables),
             block_tables.stride(0), _address(context_lens), _address(error_flags),
             PA_LAUNCH_PDL if pdl else 0),
            (k, v, k_cache, v_cache, k_scale, v_scale, cu_seqlens, block_tables, context_lens,
             error_flags))


def store_kv_fp8_block(k, v, k_cache, v_cache, k_scale, v_scale, cu_seqlens, block_tables,
                       context_lens, error_flags=None, stream=None, pdl=False):
    """pa_store_kv_fp8_block: append k/v bf16 [T, Hkv, D] (any token/head
    strides, unit dim stride), packed by cu_seqlens (int32 [B + 1]), as the
    last positions of sequences of context_lens (int32 [B], the new tokens
    included), to block-scaled FP8 pools (see fp8_block_pools)."""
    StoreKvFp8BlockCall(k, v, k_cache, v_cache, k_scale, v_scale, cu_seqlens, block_tables,
                        context_lens, error_flags, pdl)(stream)


class DecodeFp8BlockCall(_Prepared):
    """A prepared pa_decode_fp8_block (arguments as ``decode_fp8_block``); the
    output tensor and, if none is given, the workspace are kept with it."""

    def __init__(self, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                 out, num_splits=0, workspace=None, pdl=False, early_kv=False):
        NB, bs, Hkv, D = _need_fp8_block_pools(k_cache, v_cache, k_scale, v_scale)
        _need_contiguous(q, torch.bfloat16, "q", dims=3)
        B, Hq, Dq = q.shape
        if Dq != D:
            raise PagedAttentionError("q and the pools differ in head_dim")
        _need_tables(block_tables, context_lens, B)
        code = _out_code(out.dtype)
        if not (out.is_cuda or out.is_pinned()):
            raise PagedAttentionError("out must be a CUDA tensor or pinned host memory")
        if out.shape != q.shape or not out.is_contiguous():
            raise PagedAttentionError("out must be a contiguous [B, Hq, D] tensor")
        made = ()
        if workspace is None:
            workspace = decode_workspace(Hq, Hkv, num_splits, D, q.device)
            made = (workspace,)
        _need_contiguous(workspace, workspace.dtype, "workspace")
        self.out, self.workspace = out, workspace
        self._prepare(
            lib.pa_decode_fp8_block, "pa_decode_fp8_block",
            (_address(out), code, _address(q), _address(k_cache), _address(v_cache),
             _address(k_scale), _address(v_scale), NB, _address(block_tables),
             block_tables.stride(0), _address(context_lens), B, Hq, Hkv, D, bs, float(scale),
             int(num_splits), _address(workspace), workspace.numel() * workspace.element_size(),
             _decode_flags(pdl, early_kv)),
            (q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out, workspace),
            out, made)


def decode_fp8_block(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                     out=None, out_dtype=torch.bfloat16, num_splits=0, workspace=None,
                     stream=None, pdl=False, early_kv=False):
    """pa_decode_fp8_block: q bf16 [B, Hq, D] over block-scaled FP8 pools
    (see fp8_block_pools); returns out [B, Hq, D]."""
    with _on(stream) as handed:
        if out is None:
            out = handed(torch.empty(q.shape, dtype=out_dtype, device=q.device))
        return DecodeFp8BlockCall(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                  context_lens, scale, out, num_splits, workspace, pdl,
                                  early_kv)(stream)


class PrefillFp8BlockCall(_Prepared):
    """A prepared pa_prefill_fp8_block (arguments as
    ``prefill_varlen_fp8_block``)."""

    def __init__(self, q, cu_seqlens, k_cache, v_cache, k_scale, v_scale, block_tables,
                 context_lens, scale, max_q_len, out, error_flags=None):
        NB, bs, Hkv, D = _need_fp8_block_pools(k_cache, v_cache, k_scale, v_scale)
        _need_contiguous(q, torch.bfloat16, "q", dims=3)
        T, Hq, Dq = q.shape
        if Dq != D:
            raise PagedAttentionError("q and the pools differ in head_dim")
        _need_contiguous(cu_seqlens, torch.int32, "cu_seqlens", dims=1)
        B = cu_seqlens.shape[0] - 1
        if B < 0:
            raise PagedAttentionError("cu_seqlens needs num_seqs + 1 entries")
        _need_tables(block_tables, context_lens, B)
        code = _out_code(out.dtype)
        _need_contiguous(out, out.dtype, "out", q.shape)
        _need_error_flags(error_flags)
        self.out = out
        self._prepare(
            lib.pa_prefill_fp8_block, "pa_prefill_fp8_block",
            (_address(out), code, _address(q), _address(cu_seqlens), B, T, int(max_q_len),
             _address(k_cache), _address(v_cache), _address(k_scale), _address(v_scale), NB,
             _address(block_tables), block_tables.stride(0), _address(context_lens), Hq, Hkv, D,
             bs, float(scale), _address(error_flags)),
            (q, cu_seqlens, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out,
             error_flags), out)


def prefill_varlen_fp8_block(q, cu_seqlens, k_cache, v_cache, k_scale, v_scale, block_tables,
                             context_lens, scale, max_q_len, out=None, out_dtype=torch.bfloat16,
                             error_flags=None, stream=None):
    """pa_prefill_fp8_block: q bf16 [T, Hq, D] packed by cu_seqlens (int32
    [N + 1]) over block-scaled FP8 pools that hold the chunks' own keys too
    (store_kv_fp8_block first); returns out [T, Hq, D]."""
    if out is None:
        with _on(stream) as handed:
            out = handed(torch.empty(q.shape, dtype=out_dtype, device=q.device))
    return PrefillFp8BlockCall(q, cu_seqlens, k_cache, v_cache, k_scale, v_scale, block_tables,
                               context_lens, scale, max_q_len, out, error_flags)(stream)


class _PagePool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64)]


class PagePools:
    """The pools whose pages move together (K, V and scale tensors of every
    layer, any dtype): contiguous CUDA tensors with one page per index of the
    first dimension, checked once.  Keeps the tensors alive."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        if not self.tensors:
            raise PagedAttentionError("PagePools needs at least one pool")
        self.num_blocks = self.tensors[0].shape[0] if self.tensors[0].dim() else 0
        self.array = (_PagePool * len(self.tensors))()
        for entry, t in zip(self.array, self.tensors):
            if not t.is_cuda or not t.is_contiguous() or t.dim() < 1:
                raise PagedAttentionError("pools must be contiguous CUDA tensors")
            if t.shape[0] != self.num_blocks:
                raise PagedAttentionError("pools must have the same number of pages")
            if t.numel() == 0:
                raise PagedAttentionError("pools must not be empty")
            entry.base = t.data_ptr()
            entry.page_bytes = t.numel() // self.num_blocks * t.element_size()


class CopyPagesCall(_Prepared):
    """A prepared pa_copy_pages (arguments as ``copy_pages``)."""

    def __init__(self, pools, src, dst, count=None, error_flags=None, pdl=False):
        _need_contiguous(src, torch.int32, "src", dims=1)
        _need_contiguous(dst, torch.int32, "dst", src.shape)
        if count is not None:
            _need_contiguous(count, torch.int32, "count")
            if count.numel() < 1:
                raise PagedAttentionError("count must hold an int32 word")
        _need_error_flags(error_flags)
        self.pools = pools
        self._prepare(
            lib.pa_copy_pages, "pa_copy_pages",
            (ctypes.addressof(pools.array), len(pools.tensors), pools.num_blocks, _address(src),
             _address(dst), src.shape[0], _address(count), _address(error_flags),
             PA_LAUNCH_PDL if pdl else 0),
            (*pools.tensors, src, dst, count, error_flags))


def copy_pages(pools, src, dst, count=None, error_flags=None, stream=None, pdl=False):
    """pa_copy_pages: in every pool of ``pools`` (a PagePools), page dst[i]
    becomes a copy of page src[i] (int32 [n]; src[i] < 0: skipped); with
    ``count`` (int32 CUDA tensor) only the first count[0] pairs."""
    CopyPagesCall(pools, src, dst, count, error_flags, pdl)(stream)


def _need_rows(block_tables, context_lens, ref_counts, error_flags):
    _need_table_rows(block_tables)
    rows = block_tables.shape[0]
    if rows and block_tables.stride(0) != block_tables.shape[1]:
        # a row is written up to its stride
        raise PagedAttentionError("block_tables must be contiguous")
    _need_contiguous(context_lens, torch.int32, "context_lens", (rows,))
    _need_contiguous(ref_counts, torch.int32, "ref_counts", dims=1)
    _need_error_flags(error_flags)
    return rows, ref_counts.shape[0]


def _i32_out(t, n, name, like):
    if t is None:
        return torch.empty(n, dtype=torch.int32, device=like.device)
    _need_contiguous(t, torch.int32, name, (n,))
    return t


class ForkPagesCall(_Prepared):
    """A prepared pa_fork_pages (arguments as ``fork_pages``); ``copy_src``,
    ``copy_dst`` and ``forked`` hold the results of the latest call."""

    def __init__(self, block_tables, context_lens, parents, children, ref_counts, copy_src=None,
                 copy_dst=None, forked=None, error_flags=None, pdl=False, block_size=16):
        rows, NB = _need_rows(block_tables, context_lens, ref_counts, error_flags)
        _need_contiguous(parents, torch.int32, "parents", dims=1)
        n = parents.shape[0]
        _need_contiguous(children, torch.int32, "children", (n,))
        self.copy_src = _i32_out(copy_src, n, "copy_src", parents)
        self.copy_dst = _i32_out(copy_dst, n, "copy_dst", parents)
        self.forked = _i32_out(forked, n, "forked", parents)
        result = (self.copy_src, self.copy_dst, self.forked)
        made = [t for t, given in zip(result, (copy_src, copy_dst, forked)) if given is None]
        self._prepare(
            lib.pa_fork_pages, "pa_fork_pages",
            (_address(block_tables), block_tables.stride(0), _address(context_lens), rows,
             _address(parents), _address(children), n, _address(ref_counts), NB, block_size,
             *map(_address, result), _address(error_flags), PA_LAUNCH_PDL if pdl else 0),
            (block_tables, context_lens, parents, children, ref_counts, *result, error_flags),
            result, made)


def fork_pages(block_tables, context_lens, parents, children, ref_counts, copy_src=None,
               copy_dst=None, forked=None, error_flags=None, stream=None, pdl=False):
    """pa_fork_pages: row children[i] of the tables becomes a copy of row
    parents[i] (int32 [n]) that shares its full pages; the part-filled last
    page gets a free page, to be filled by ``copy_pages(pools, copy_src,
    copy_dst)``.  Returns (copy_src, copy_dst, forked), int32 [n] each."""
    with _on(stream) as handed:
        out = ForkPagesCall(block_tables, context_lens, parents, children, ref_counts, copy_src,
                            copy_dst, forked, error_flags, pdl)(stream)
        return tuple(map(handed, out))


class FreePagesCall(_Prepared):
    """A prepared pa_free_pages (arguments as ``free_pages``)."""

    def __init__(self, block_tables, context_lens, seqs, ref_counts, error_flags=None, pdl=False,
                 block_size=16):
        rows, NB = _need_rows(block_tables, context_lens, ref_counts, error_flags)
        _need_contiguous(seqs, torch.int32, "seqs", dims=1)
        self._prepare(
            lib.pa_free_pages, "pa_free_pages",
            (_address(block_tables), block_tables.stride(0), _address(context_lens), rows,
             _address(seqs), seqs.shape[0], _address(ref_counts), NB, block_size,
             _address(error_flags), PA_LAUNCH_PDL if pdl else 0),
            (block_tables, context_lens, seqs, ref_counts, error_flags))


def free_pages(block_tables, context_lens, seqs, ref_counts, error_flags=None, stream=None,
               pdl=False):
    """pa_free_pages: rows seqs (int32 [n]) of the tables let their pages go
    and become empty."""
    FreePagesCall(block_tables, context_lens, seqs, ref_counts, error_flags, pdl)(stream)


class CompactPagesCall(_Prepared):
    """A prepared pa_compact_pages (arguments as ``compact_pages``);
    ``copy_src``, ``copy_dst``, ``counts`` and ``remap`` hold the results of
    the latest call."""

    def __init__(self, block_tables, context_lens, ref_counts, copy_src=None, copy_dst=None,
                 counts=None, remap=None, error_flags=None, pdl=False, block_size=16):
        rows, NB = _need_rows(block_tables, context_lens, ref_counts, error_flags)
        self.copy_src = _i32_out(copy_src, NB // 2, "copy_src", ref_counts)
        self.copy_dst = _i32_out(copy_dst, NB // 2, "copy_dst", ref_counts)
        self.counts = _i32_out(counts, 2, "counts", ref_counts)
        self.remap = _i32_out(remap, NB, "remap", ref_counts)
        result = (self.copy_src, self.copy_dst, self.counts, self.remap)
        made = [t for t, given in zip(result, (copy_src, copy_dst, counts, remap))
                if given is None]
        self._prepare(
            lib.pa_compact_pages, "pa_compact_pages",
            (_address(block_tables), block_tables.stride(0), _address(context_lens), rows,
             _address(ref_counts), NB, block_size, *map(_address, result),
             _address(error_flags), PA_LAUNCH_PDL if pdl else 0),
            (block_tables, context_lens, ref_counts, *result, error_flags), result, made)


def compact_pages(block_tables, context_lens, ref_counts, copy_src=None, copy_dst=None,
                  counts=None, remap=None, error_flags=None, stream=None, pdl=False):
    """pa_compact_pages: plan the move of the live pages to the front of the
    pool and bring tables and counts up to date; ``copy_pages(pools, copy_src,
    copy_dst, count=counts)`` then moves the contents.  Returns (copy_src,
    copy_dst [NB / 2], counts [moves, live pages], remap [NB]), int32."""
    with _on(stream) as handed:
        out = CompactPagesCall(block_tables, context_lens, ref_counts, copy_src, copy_dst,
                               counts, remap, error_flags, pdl)(stream)
        return tuple(map(handed, out))


def decode_merge(out, workspace, context_lens, num_splits, block_size=16, stream=None):
    """pa_decode_merge over a workspace filled by pa_decode (or by hand)."""
    B, Hq, D = out.shape
    _check(lib.pa_decode_merge(_ptr(out), _out_code(out.dtype), _ptr(workspace),
                               workspace.numel() * workspace.element_size(),
                               _ptr(context_lens), B, Hq, D, block_size, int(num_splits),
                               _stream(stream)), "pa_decode_merge")
    return out


def prefill_varlen(q, cu_seqlens, k_cache, v_cache, block_tables, context_lens, scale,
                   max_q_len, out=None, out_dtype=torch.bfloat16, error_flags=None,
                   stream=None):
    """pa_prefill_varlen: q bf16 [T, Hq, D] packed by cu_seqlens (int32 [N+1])."""
    _need(q, torch.bfloat16, "q", 3)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    T, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    if out is None:
        with _on(stream) as handed:
            out = handed(torch.empty((T, Hq, D), dtype=out_dtype, device=q.device))
    _check(lib.pa_prefill_varlen(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(cu_seqlens),
                                 cu_seqlens.shape[0] - 1, T, int(max_q_len), _ptr(k_cache),
                                 _ptr(v_cache), NB, _ptr(block_tables), block_tables.stride(0),
                                 _ptr(context_lens), Hq, Hkv, D, bs, float(scale),
                                 _ptr(error_flags), _stream(stream)), "pa_prefill_varlen")
    return out


def prefill_store_varlen(q, new_k, new_v, slot_mapping, cu_seqlens, k_cache, v_cache,
                         block_tables, context_lens, scale, max_q_len, out=None,
                         out_dtype=torch.bfloat16, error_flags=None, stream=None):
    """pa_prefill_store_varlen: the chunks' K/V rows (new_k / new_v bf16
    [T, Hkv, D], heads contiguous) stored at slot_mapping (int32 [T]) and
    attended, in one kernel; otherwise as prefill_varlen."""
    _need(q, torch.bfloat16, "q", 3)
    _need(new_k, torch.bfloat16, "new_k", 3)
    _need(new_v, torch.bfloat16, "new_v", 3)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    for t, n in ((new_k, "new_k"), (new_v, "new_v")):
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise PagedAttentionError(f"{n} needs contiguous heads")
    T, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    if tuple(new_k.shape) != (T, Hkv, D) or new_v.shape != new_k.shape or \
            slot_mapping.shape[0] != T:
        raise PagedAttentionError("new_k / new_v / slot_mapping need one row per token")
    if out is None:
        with _on(stream) as handed:
            out = handed(torch.empty((T, Hq, D), dtype=out_dtype, device=q.device))
    _check(lib.pa_prefill_store_varlen(_ptr(out), _out_code(out.dtype), _ptr(q), _ptr(new_k),
                                       _ptr(new_v), new_k.stride(0), new_v.stride(0),
                                       _ptr(slot_mapping), _ptr(cu_seqlens),
                                       cu_seqlens.shape[0] - 1, T, int(max_q_len), _ptr(k_cache),
                                       _ptr(v_cache), NB, _ptr(block_tables),
                                       block_tables.stride(0), _ptr(context_lens), Hq, Hkv, D, bs,
                                       float(scale), _ptr(error_flags), _stream(stream)),
           "pa_prefill_store_varlen")
    return out


def read_error_word(buf, clear=False, stream=None) -> int:
    """The int32 error word at the start of ``buf`` (a decode workspace or an
    error_flags tensor), read through pa_get_device_error: the copy is
    enqueued on ``stream`` and the stream synchronised; ``clear`` resets the
    word to 0 after the copy."""
    if not buf.is_cuda or buf.numel() * buf.element_size() < 4:
        raise PagedAttentionError("error word must be a CUDA tensor of at least 4 bytes")
    flags = ctypes.c_int32(0)
    _check(lib.pa_get_device_error(_ptr(buf), ctypes.byref(flags), 1 if clear else 0,
                                   _stream(stream)), "pa_get_device_error")
    return int(flags.value)
