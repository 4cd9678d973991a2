"""Thin ctypes binding of libpa.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
computation of its own: it reads shapes off the tensors, checks that they are
contiguous CUDA tensors of the right dtype, and passes raw device pointers and
the current CUDA stream to the library.  There is no fallback: if the CUDA
library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_388_b200.build` "
        "(nvcc, sm_100a).  There is no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)

P = ctypes.c_void_p
I = ctypes.c_int
F = ctypes.c_float
SZ = ctypes.c_size_t

_lib.pa_reshape_and_cache.restype = I
_lib.pa_reshape_and_cache.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P]
_lib.pa_copy_blocks.restype = I
_lib.pa_copy_blocks.argtypes = [P, P, P, I, I, I, I, I, I, P]
_lib.pa_reshape_and_cache_fp8.restype = I
_lib.pa_reshape_and_cache_fp8.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, F, P]
_lib.pa_decode_fp8.restype = I
_lib.pa_decode_fp8.argtypes = [P, P, P, P, P, I, P, I, I, I, I, I, I, F, F, F, I, I, P, SZ, P]
_lib.pa_decode_fp8_rows.restype = I
_lib.pa_decode_fp8_rows.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, F, F, F, I, I, I,
                                    P, SZ, P]
_lib.pa_decode_fp8_rows_workspace_size.restype = SZ
_lib.pa_decode_fp8_rows_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
_lib.pa_swap_blocks.restype = I
_lib.pa_swap_blocks.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, P]
_lib.pa_decode_workspace_size.restype = SZ
_lib.pa_decode_workspace_size.argtypes = [I, I, I, I, I, I, I]
_lib.pa_decode.restype = I
_lib.pa_decode.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, F, I, I, I, P, SZ, P]
_lib.pa_decode_noalloc.restype = I
_lib.pa_decode_noalloc.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, F, I, I, I, P]
_lib.pa_decode_shared_prefix.restype = I
_lib.pa_decode_shared_prefix.argtypes = [P, P, P, P, P, I, P, I, P, P, I, I, I, I, I, I, I, F, I, I,
                                         P, SZ, P]
_lib.pa_decode_shared_prefix_workspace_size.restype = SZ
_lib.pa_decode_shared_prefix_workspace_size.argtypes = [I, I, I, I, I, I]
_lib.pa_decode_shared_prefix_fp8.restype = I
_lib.pa_decode_shared_prefix_fp8.argtypes = [P, P, P, P, P, I, P, I, P, P, I, I, I, I, I, I, I, F,
                                             F, F, I, I, I, P, SZ, P]
_lib.pa_decode_shared_prefix_fp8_workspace_size.restype = SZ
_lib.pa_decode_shared_prefix_fp8_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I]
L = ctypes.c_int64
_lib.pa_latent_write.restype = I
_lib.pa_latent_write.argtypes = [P, P, P, P, I, L, L, I, I, I, I, I, P]
_lib.pa_latent_decode.restype = I
_lib.pa_latent_decode.argtypes = [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, F, I, I, P, SZ, P]
_lib.pa_latent_decode_workspace_size.restype = SZ
_lib.pa_latent_decode_workspace_size.argtypes = [I, I, I, I]
_lib.pa_latent_prefill.restype = I
_lib.pa_latent_prefill.argtypes = [P, P, P, P, P, P, L, L, L, L, L, P, P, I, I, I, I, I, I, I, I, F,
                                   I, I, P, SZ, P]
_lib.pa_latent_prefill_workspace_size.restype = SZ
_lib.pa_latent_prefill_workspace_size.argtypes = [I, I, I, I, I]
_lib.pa_table_step.restype = I
_lib.pa_table_step.argtypes = [P, I, P, P, P, P, P, I, I, I, P, I, P, P, P, P, I, P, SZ, P]
_lib.pa_table_compact.restype = I
_lib.pa_table_compact.argtypes = [P, I, P, P, I, I, I, P, P, P, P, I, P, SZ, P]
_lib.pa_table_workspace_size.restype = SZ
_lib.pa_table_workspace_size.argtypes = [I, I, I]
_lib.pa_noalloc_scratch_bytes.restype = SZ
_lib.pa_noalloc_scratch_bytes.argtypes = []
_lib.pa_get_device_error.restype = I
_lib.pa_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), P]
_lib.pa_status_string.restype = ctypes.c_char_p
_lib.pa_status_string.argtypes = [I]
_lib.pa_abi_version.restype = I
_lib.pa_abi_version.argtypes = []

PA_F32, PA_F16, PA_BF16, PA_FP8_E4M3 = 0, 1, 2, 3
_DT = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16,
       torch.uint8: PA_FP8_E4M3, torch.float8_e4m3fn: PA_FP8_E4M3}

PA_DEVERR_BLOCK_ID = 0x1
PA_DEVERR_SLOT = 0x2
PA_DEVERR_CONTEXT_LEN = 0x4
PA_DEVERR_QUERY_LEN = 0x8
PA_DEVERR_TIMEOUT = 0x10
PA_DEVERR_PREFIX = 0x20
PA_DEVERR_STAGING = 0x40
PA_DEVERR_POOL = 0x80
PA_DEVERR_TABLE = 0x100


class PAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib.pa_status_string(status).decode()} ({status})")


def library():
    """The loaded ctypes library (for tests that call entry points directly)."""
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle, without a Stream object
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dev(t, name, dtype=None, cur=None):
    """A contiguous CUDA tensor on the current device (the library launches on
    the current device and would otherwise dereference another GPU's memory).
    ``cur``: that device's index, where the caller has read it."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if cur is None:
        cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{cur}; "
                         "call under torch.cuda.device(...) of the tensors' device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _shape(cond, what):
    if not cond:
        raise ValueError(what)


def _cache_shapes(k_cache, v_cache):
    """(num_blocks, num_kv_heads, block_size, head_dim) of a pair of caches."""
    _shape(k_cache.dim() == 4, "k_cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    _shape(tuple(v_cache.shape) == tuple(k_cache.shape), "k_cache and v_cache shapes disagree")
    return tuple(k_cache.shape)


def _new_token_shapes(key, value, k_cache, v_cache, slot_mapping):
    nb, hk, bs, d = _cache_shapes(k_cache, v_cache)
    _shape(key.dim() == 3 and tuple(key.shape[1:]) == (hk, d),
           f"key must be [num_tokens, {hk}, {d}] to match the caches, got {tuple(key.shape)}")
    _shape(tuple(value.shape) == tuple(key.shape), "key and value shapes disagree")
    _shape(slot_mapping.dim() == 1 and slot_mapping.shape[0] == key.shape[0],
           "slot_mapping must hold one slot per key/value token")
    return nb, hk, bs, d


def _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc=None):
    """Shapes of a decode call; every tensor must agree with the others."""
    nb, hk, bs, d = _cache_shapes(k_cache, v_cache)
    _shape(q.dim() == 3 and q.shape[2] == d, f"q must be [tokens, heads, {d}] to match the caches")
    _shape(tuple(out.shape) == tuple(q.shape), "out and q shapes disagree")
    tq, h, _ = q.shape
    _shape(h % hk == 0, "num_heads must be a multiple of num_kv_heads")
    _shape(block_tables.dim() == 2, "block_tables must be [num_seqs, max_blocks_per_seq]")
    s, mbps = block_tables.shape
    _shape(context_lens.dim() == 1 and context_lens.shape[0] == s,
           "block_tables and context_lens disagree on the number of sequences")
    if query_start_loc is None:
        _shape(tq == s, "without query_start_loc q must hold one row per sequence")
    else:
        _shape(query_start_loc.dim() == 1 and query_start_loc.shape[0] == s + 1,
               "query_start_loc must have num_seqs + 1 entries")
    return tq, h, d, nb, hk, bs, s, mbps


def _check(rc, what):
    if rc != 0:
        raise PAError(rc, what)


def pa_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, stream=None):
    """key/value [T, Hk, D]; caches [NB, Hk, bs, D]; slot_mapping int64 [T]."""
    nb, hk, bs, d = _new_token_shapes(key, value, k_cache, v_cache, slot_mapping)
    _dev(key, "key")
    _dev(value, "value", key.dtype)
    _dev(k_cache, "k_cache", key.dtype)
    _dev(v_cache, "v_cache", key.dtype)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    rc = _lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(slot_mapping), key.shape[0], hk, d, bs, nb,
                                   _DT[key.dtype], _stream(stream))
    _check(rc, "pa_reshape_and_cache")


def pa_copy_blocks(k_cache, v_cache, block_mapping, stream=None):
    """block_mapping int64 [P, 2] of (src, dst) physical block ids."""
    nb, hk, bs, d = _cache_shapes(k_cache, v_cache)
    _shape(block_mapping.dim() == 2 and block_mapping.shape[1] == 2,
           "block_mapping must be [num_pairs, 2]")
    _dev(k_cache, "k_cache")
    _dev(v_cache, "v_cache", k_cache.dtype)
    _dev(block_mapping, "block_mapping", torch.int64)
    rc = _lib.pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_mapping),
                             block_mapping.shape[0], hk, d, bs, nb, _DT[k_cache.dtype],
                             _stream(stream))
    _check(rc, "pa_copy_blocks")


def pa_reshape_and_cache_fp8(key, value, k_cache, v_cache, slot_mapping, k_scale, v_scale,
                             stream=None):
    """key/value [T, Hk, D] (fp32/fp16/bf16); caches uint8 [NB, Hk, bs, D] of
    E4M3 codes; slot_mapping int64 [T]."""
    nb, hk, bs, d = _new_token_shapes(key, value, k_cache, v_cache, slot_mapping)
    _dev(key, "key")
    _dev(value, "value", key.dtype)
    _dev(k_cache, "k_cache", torch.uint8)
    _dev(v_cache, "v_cache", torch.uint8)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    rc = _lib.pa_reshape_and_cache_fp8(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(slot_mapping), key.shape[0], hk, d, bs, nb,
                                       _DT[key.dtype], float(k_scale), float(v_scale),
                                       _stream(stream))
    _check(rc, "pa_reshape_and_cache_fp8")


def pa_decode_fp8_rows_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                      max_context_len, max_blocks_per_seq, staged_blocks) -> int:
    return int(_lib.pa_decode_fp8_rows_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                      block_size, max_context_len,
                                                      max_blocks_per_seq, staged_blocks))


def pa_decode_fp8(out, q, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale,
                  max_context_len=0, workspace=None, query_start_loc=None, max_query_len=1,
                  staged_blocks=0, stream=None):
    """out/q [S, H, D] fp16/bf16; caches uint8 E4M3 codes [NB, Hk, bs, D];
    workspace: uint8 CUDA tensor of >= pa_decode_workspace_size(...) bytes.
    With query_start_loc (chunked-prefill rows as in pa_decode) the call is
    pa_decode_fp8_rows: staged_blocks bounds the blocks of the sequences with
    more than one row (batch.staged_blocks_needed), and the workspace must hold
    pa_decode_fp8_rows_workspace_size(...) bytes."""
    tq, h, d, nb, hk, bs, s, mbps = _decode_shapes(out, q, k_cache, v_cache, block_tables,
                                                   context_lens, query_start_loc)
    if query_start_loc is not None:
        _dev(query_start_loc, "query_start_loc", torch.int32)
    _dev(q, "q")
    _dev(out, "out", q.dtype)
    _dev(k_cache, "k_cache", torch.uint8)
    _dev(v_cache, "v_cache", torch.uint8)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    if workspace is not None:
        _dev(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if query_start_loc is not None:
        pa_decode_fp8_rows(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                           scale, k_scale, v_scale, max_query_len, staged_blocks,
                           max_context_len=max_context_len, workspace=workspace, stream=stream)
        return
    rc = _lib.pa_decode_fp8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                            mbps, _ptr(context_lens), s, h, hk, d, bs, nb, float(scale),
                            float(k_scale), float(v_scale), int(max_context_len), _DT[q.dtype],
                            _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "pa_decode_fp8")


def pa_decode_fp8_rows(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                       scale, k_scale, v_scale, max_query_len, staged_blocks, max_context_len=0,
                       workspace=None, stream=None):
    """pa_decode_fp8 over a batch with chunked-prefill rows: q/out [Tq, H, D],
    query_start_loc int32 [S + 1]; staged_blocks bounds the blocks of the
    sequences with more than one row; workspace uint8 of
    >= pa_decode_fp8_rows_workspace_size(...) bytes."""
    tq, h, d, nb, hk, bs, s, mbps = _decode_shapes(out, q, k_cache, v_cache, block_tables,
                                                   context_lens, query_start_loc)
    _dev(q, "q")
    _dev(out, "out", q.dtype)
    _dev(k_cache, "k_cache", torch.uint8)
    _dev(v_cache, "v_cache", torch.uint8)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    _dev(query_start_loc, "query_start_loc", torch.int32)
    if workspace is not None:
        _dev(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_decode_fp8_rows(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(block_tables), mbps, _ptr(context_lens),
                                 _ptr(query_start_loc), s, tq, int(max_query_len), h, hk, d, bs,
                                 nb, float(scale), float(k_scale), float(v_scale),
                                 int(max_context_len), int(staged_blocks), _DT[q.dtype],
                                 _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "pa_decode_fp8_rows")


def pa_swap_blocks(dst_k, dst_v, src_k, src_v, block_mapping, stream=None):
    """Copy blocks (src, dst) of block_mapping int64 [P, 2] from the
    (src_k, src_v) pool into the (dst_k, dst_v) pool.  Pools and mapping may
    be CUDA tensors or pinned CPU tensors (not pageable ones)."""
    for name, t in (("dst_k", dst_k), ("dst_v", dst_v), ("src_k", src_k), ("src_v", src_v),
                    ("block_mapping", block_mapping)):
        if t.is_cuda:
            _dev(t, name)
        elif not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if block_mapping.dtype != torch.int64:
        raise ValueError("block_mapping must be int64")
    if not (dst_k.dtype == dst_v.dtype == src_k.dtype == src_v.dtype):
        raise ValueError("pools must share one dtype")
    nd, hk, bs, d = dst_k.shape
    ns = src_k.shape[0]
    if tuple(src_k.shape[1:]) != (hk, bs, d) or src_v.shape != src_k.shape or dst_v.shape != dst_k.shape:
        raise ValueError("pool shapes disagree")
    rc = _lib.pa_swap_blocks(_ptr(dst_k), _ptr(dst_v), _ptr(src_k), _ptr(src_v),
                             _ptr(block_mapping), block_mapping.shape[0], hk, d, bs, ns, nd,
                             _DT[dst_k.dtype], _stream(stream))
    _check(rc, "pa_swap_blocks")


def pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                             max_context_len, kv_split_tokens=0) -> int:
    return int(_lib.pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                             block_size, max_context_len, kv_split_tokens))


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale,
              query_start_loc=None, max_query_len=1, max_context_len=0, kv_split_tokens=0,
              workspace=None, stream=None):
    """out/q [Tq, H, D]; caches [NB, Hk, bs, D]; block_tables int32 [S, mbps];
    context_lens int32 [S]; query_start_loc int32 [S+1] or None; workspace: a
    uint8 CUDA tensor of >= pa_decode_workspace_size(...) bytes (or None when
    that size is 0)."""
    tq, h, d, nb, hk, bs, s, mbps = _decode_shapes(out, q, k_cache, v_cache, block_tables,
                                                   context_lens, query_start_loc)
    _dev(q, "q")
    _dev(out, "out", q.dtype)
    _dev(k_cache, "k_cache", q.dtype)
    _dev(v_cache, "v_cache", q.dtype)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    if query_start_loc is not None:
        _dev(query_start_loc, "query_start_loc", torch.int32)
    if workspace is not None:
        _dev(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                        mbps, _ptr(context_lens), _ptr(query_start_loc), s, tq,
                        int(max_query_len), h, hk, d, bs, nb, float(scale), int(max_context_len),
                        int(kv_split_tokens), _DT[q.dtype], _ptr(workspace), ws_bytes,
                        _stream(stream))
    _check(rc, "pa_decode")


def pa_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                      query_start_loc=None, max_query_len=1, max_context_len=0, kv_split_tokens=0,
                      stream=None):
    """pa_decode with the library's static scratch instead of a workspace, for
    callers that cannot allocate device memory.  Calls must not overlap on
    the GPU (they share the scratch); make the first call on a device before
    any stream capture."""
    tq, h, d, nb, hk, bs, s, mbps = _decode_shapes(out, q, k_cache, v_cache, block_tables,
                                                   context_lens, query_start_loc)
    _dev(q, "q")
    _dev(out, "out", q.dtype)
    _dev(k_cache, "k_cache", q.dtype)
    _dev(v_cache, "v_cache", q.dtype)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    if query_start_loc is not None:
        _dev(query_start_loc, "query_start_loc", torch.int32)
    rc = _lib.pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                _ptr(block_tables), mbps, _ptr(context_lens), _ptr(query_start_loc),
                                s, tq, int(max_query_len), h, hk, d, bs, nb, float(scale),
                                int(max_context_len), int(kv_split_tokens), _DT[q.dtype],
                                _stream(stream))
    _check(rc, "pa_decode_noalloc")


def pa_decode_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                           max_context_len) -> int:
    return int(_lib.pa_decode_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                           head_dim, block_size, max_context_len))


def pa_decode_shared_prefix(out, q, k_cache, v_cache, block_tables, context_lens, group_start,
                            group_shared_blocks, scale, max_group_size=0, max_context_len=0,
                            workspace=None, stream=None):
    """Decode with shared-prefix groups.  out/q [S, H, D]; group_start int32
    [G+1] and group_shared_blocks int32 [G] on the device; workspace: uint8
    CUDA tensor of >= pa_decode_shared_prefix_workspace_size(...) bytes."""
    s, h, d, nb, hk, bs, _, mbps = _decode_shapes(out, q, k_cache, v_cache, block_tables,
                                                  context_lens)
    _shape(group_start.dim() == 1 and group_shared_blocks.dim() == 1 and
           group_start.shape[0] == group_shared_blocks.shape[0] + 1,
           "group_start must have one more entry than group_shared_blocks")
    _dev(q, "q")
    _dev(out, "out", q.dtype)
    _dev(k_cache, "k_cache", q.dtype)
    _dev(v_cache, "v_cache", q.dtype)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    _dev(group_start, "group_start", torch.int32)
    _dev(group_shared_blocks, "group_shared_blocks", torch.int32)
    if workspace is not None:
        _dev(workspace, "workspace")
    g = group_shared_blocks.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_decode_shared_prefix(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(block_tables), mbps, _ptr(context_lens), s,
                                      _ptr(group_start), _ptr(group_shared_blocks), g,
                                      int(max_group_size), h, hk, d, bs, nb, float(scale),
                                      int(max_context_len), _DT[q.dtype], _ptr(workspace),
                                      ws_bytes, _stream(stream))
    _check(rc, "pa_decode_shared_prefix")


def pa_decode_shared_prefix_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                               block_size, max_context_len, max_blocks_per_seq,
                                               num_groups, staged_blocks) -> int:
    return int(_lib.pa_decode_shared_prefix_fp8_workspace_size(
        num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
        max_blocks_per_seq, num_groups, staged_blocks))


def pa_decode_shared_prefix_fp8(out, q, k_cache, v_cache, block_tables, context_lens, group_start,
                                group_shared_blocks, scale, k_scale, v_scale, staged_blocks,
                                max_group_size=0, max_context_len=0, workspace=None, stream=None):
    """pa_decode_shared_prefix over FP8 (E4M3) caches (uint8 codes); out/q
    fp16/bf16 [S, H, D]; staged_blocks bounds the groups' shared blocks
    (their sum); workspace uint8 of
    >= pa_decode_shared_prefix_fp8_workspace_size(...) bytes."""
    s, h, d, nb, hk, bs, _, mbps = _decode_shapes(out, q, k_cache, v_cache, block_tables,
                                                  context_lens)
    _shape(group_start.dim() == 1 and group_shared_blocks.dim() == 1 and
           group_start.shape[0] == group_shared_blocks.shape[0] + 1,
           "group_start must have one more entry than group_shared_blocks")
    _dev(q, "q")
    _dev(out, "out", q.dtype)
    _dev(k_cache, "k_cache", torch.uint8)
    _dev(v_cache, "v_cache", torch.uint8)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    _dev(group_start, "group_start", torch.int32)
    _dev(group_shared_blocks, "group_shared_blocks", torch.int32)
    if workspace is not None:
        _dev(workspace, "workspace")
    g = group_shared_blocks.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_decode_shared_prefix_fp8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(block_tables), mbps, _ptr(context_lens), s,
                                          _ptr(group_start), _ptr(group_shared_blocks), g,
                                          int(max_group_size), h, hk, d, bs, nb, float(scale),
                                          float(k_scale), float(v_scale), int(max_context_len),
                                          int(staged_blocks), _DT[q.dtype], _ptr(workspace),
                                          ws_bytes, _stream(stream))
    _check(rc, "pa_decode_shared_prefix_fp8")


def _here(t, name):
    """The current device's index, read once a call (t: any of its tensors)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch.cuda.current_device()


def _dev_rows(t, name, dtype, cur):
    """A CUDA tensor on the current device whose last dimension is contiguous;
    returns its element strides before it (a dimension of one row or head
    counts as packed: torch leaves its stride arbitrary)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{cur}; "
                         "call under torch.cuda.device(...) of the tensors' device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if 0 in shape or 1 in shape:
        strides, packed = list(strides), 1
        for i in range(len(shape) - 1, -1, -1):
            if shape[i] <= 1:
                strides[i] = packed
            packed *= max(shape[i], 1)
    if strides[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if t.data_ptr() % 16 or strides[0] % 8 or strides[-2] % 8:  # two or three dimensions
        raise ValueError(f"rows of {name} must start on 16-byte boundaries")
    return strides[:-1]


def _latent_shape(latent_cache):
    """(num_blocks, block_size, row width) of a latent cache."""
    if not (latent_cache.dim() == 3):
        raise ValueError("latent_cache must be [num_blocks, block_size, latent_dim + rope_dim]")
    return tuple(latent_cache.shape)


def pa_latent_write(latent, rope, latent_cache, slot_mapping, stream=None):
    """latent [T, R] and rope [T, Dr] (rows may be strided slices); latent_cache
    [NB, bs, R + Dr]; slot_mapping int64 [T], negative slots are skipped."""
    nb, bs, w = _latent_shape(latent_cache)
    if not (latent.dim() == 2 and rope.dim() == 2 and latent.shape[0] == rope.shape[0]):
        raise ValueError("latent and rope must hold one row per token")
    if not (latent.shape[1] + rope.shape[1] == w):
        raise ValueError(f"latent and rope rows must add up to the cache's {w} values")
    if not (slot_mapping.dim() == 1 and slot_mapping.shape[0] == latent.shape[0]):
        raise ValueError("slot_mapping must hold one slot per token")
    cur = _here(latent_cache, "latent_cache")
    _dev(latent_cache, "latent_cache", None, cur)
    ls, = _dev_rows(latent, "latent", latent_cache.dtype, cur)
    rs, = _dev_rows(rope, "rope", latent_cache.dtype, cur)
    _dev(slot_mapping, "slot_mapping", torch.int64, cur)
    rc = _lib.pa_latent_write(_ptr(latent), _ptr(rope), _ptr(latent_cache), _ptr(slot_mapping),
                              latent.shape[0], ls, rs, latent.shape[1], rope.shape[1], bs, nb,
                              _DT.get(latent_cache.dtype, -1), _stream(stream))
    _check(rc, "pa_latent_write")


def pa_latent_decode_workspace_size(num_seqs, max_query_len, num_heads, latent_dim) -> int:
    return int(_lib.pa_latent_decode_workspace_size(num_seqs, max_query_len, num_heads, latent_dim))


def pa_latent_decode(out, lse, q, latent_cache, block_tables, context_lens, scale,
                     query_start_loc=None, max_query_len=1, max_context_len=0, workspace=None,
                     stream=None):
    """out [Tq, H, R]; lse float32 [Tq, H] or None; q [Tq, H, R + Dr];
    latent_cache [NB, bs, R + Dr]; block_tables int32 [S, mbps]; context_lens
    int32 [S]; query_start_loc int32 [S + 1] or None; workspace: uint8 CUDA
    tensor of >= pa_latent_decode_workspace_size(...) bytes."""
    nb, bs, w = _latent_shape(latent_cache)
    if not (q.dim() == 3 and q.shape[2] == w):
        raise ValueError(f"q must be [tokens, heads, {w}] to match the cache")
    tq, h, _ = q.shape
    if not (out.dim() == 3 and tuple(out.shape[:2]) == (tq, h) and out.shape[2] < w):
        raise ValueError("out must be [tokens, heads, latent_dim]")
    r = out.shape[2]
    if not (lse is None or tuple(lse.shape) == (tq, h)):
        raise ValueError("lse must be [tokens, heads]")
    if not (block_tables.dim() == 2):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    s, mbps = block_tables.shape
    if not (context_lens.dim() == 1 and context_lens.shape[0] == s):
        raise ValueError("block_tables and context_lens disagree on the number of sequences")
    if query_start_loc is None:
        if not (tq == s):
            raise ValueError("without query_start_loc q must hold one row per sequence")
    else:
        if not (query_start_loc.dim() == 1 and query_start_loc.shape[0] == s + 1):
            raise ValueError("query_start_loc must have num_seqs + 1 entries")
    cur = _here(q, "q")
    if query_start_loc is not None:
        _dev(query_start_loc, "query_start_loc", torch.int32, cur)
    _dev(q, "q", None, cur)
    _dev(out, "out", q.dtype, cur)
    _dev(latent_cache, "latent_cache", q.dtype, cur)
    _dev(block_tables, "block_tables", torch.int32, cur)
    _dev(context_lens, "context_lens", torch.int32, cur)
    if lse is not None:
        _dev(lse, "lse", torch.float32, cur)
    if workspace is not None:
        _dev(workspace, "workspace", None, cur)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_latent_decode(_ptr(out), _ptr(lse), _ptr(q), _ptr(latent_cache),
                               _ptr(block_tables), mbps, _ptr(context_lens), _ptr(query_start_loc),
                               s, tq, int(max_query_len), h, r, w - r, bs, nb, float(scale),
                               int(max_context_len), _DT.get(q.dtype, -1), _ptr(workspace),
                               ws_bytes, _stream(stream))
    _check(rc, "pa_latent_decode")


def pa_latent_prefill_workspace_size(num_seqs, num_q_tokens, num_k_tokens, num_heads,
                                     nope_dim) -> int:
    return int(_lib.pa_latent_prefill_workspace_size(num_seqs, num_q_tokens, num_k_tokens, num_heads,
                                                     nope_dim))


def pa_latent_prefill(out, lse, q, k, k_rope, v, query_start_loc, context_start_loc, scale,
                      max_query_len, causal=True, workspace=None, stream=None):
    """out [Tq, H, Dv]; lse float32 [Tq, H] or None; q [Tq, H, Dn + Dr]; k
    [Tk, H, Dn], v [Tk, H, Dv] and k_rope [Tk, Dr] (tokens and heads may be
    strided); query_start_loc and context_start_loc int32 [S + 1]; workspace:
    uint8 CUDA tensor of >= pa_latent_prefill_workspace_size(...) bytes."""
    if not (q.dim() == 3 and k.dim() == 3 and v.dim() == 3 and k_rope.dim() == 2):
        raise ValueError("q, k and v must be [tokens, heads, dim], k_rope [tokens, dim]")
    tq, h, dq = q.shape
    tk, _, dn = k.shape
    dr, dv = k_rope.shape[1], v.shape[2]
    if not (dn + dr == dq):
        raise ValueError("q rows must hold nope_dim + rope_dim values")
    if not (k.shape[1] == h and tuple(v.shape[:2]) == (tk, h) and k_rope.shape[0] == tk):
        raise ValueError("k, v and k_rope must hold the same tokens, k and v q's heads")
    if not (tuple(out.shape) == (tq, h, dv)):
        raise ValueError("out must be [tokens, heads, v_dim]")
    if not (lse is None or tuple(lse.shape) == (tq, h)):
        raise ValueError("lse must be [tokens, heads]")
    if not (query_start_loc.dim() == 1 and
            query_start_loc.shape[0] >= 1 and
            query_start_loc.shape == context_start_loc.shape):
        raise ValueError("query_start_loc and context_start_loc must have num_seqs + 1 entries each")
    cur = _here(q, "q")
    _dev(q, "q", None, cur)
    _dev(out, "out", q.dtype, cur)
    ks, kh = _dev_rows(k, "k", q.dtype, cur)
    vs, vh = _dev_rows(v, "v", q.dtype, cur)
    krs, = _dev_rows(k_rope, "k_rope", q.dtype, cur)
    if lse is not None:
        _dev(lse, "lse", torch.float32, cur)
    _dev(query_start_loc, "query_start_loc", torch.int32, cur)
    _dev(context_start_loc, "context_start_loc", torch.int32, cur)
    if workspace is not None:
        _dev(workspace, "workspace", None, cur)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_latent_prefill(_ptr(out), _ptr(lse), _ptr(q), _ptr(k), _ptr(k_rope), _ptr(v),
                                ks, kh, krs, vs, vh, _ptr(query_start_loc),
                                _ptr(context_start_loc), query_start_loc.shape[0] - 1, tq, tk,
                                int(max_query_len), h, dn, dr, dv, float(scale),
                                1 if causal else 0, _DT.get(q.dtype, -1), _ptr(workspace),
                                ws_bytes, _stream(stream))
    _check(rc, "pa_latent_prefill")


def _table_shapes(block_tables, context_lens, ref_counts):
    if not (block_tables.dim() == 2):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    if context_lens.dim() != 1 or context_lens.shape[0] != block_tables.shape[0]:
        raise ValueError("block_tables and context_lens disagree on the number of sequences")
    if not (ref_counts.dim() == 1):
        raise ValueError("ref_counts must be [num_blocks]")
    cur = _here(block_tables, "block_tables")
    _dev(block_tables, "block_tables", torch.int32, cur)
    _dev(context_lens, "context_lens", torch.int32, cur)
    _dev(ref_counts, "ref_counts", torch.int32, cur)
    return (*block_tables.shape, ref_counts.shape[0], cur)


def _pool_args(pools, num_blocks, cur):
    """Host arrays of the pools' addresses and block bytes."""
    n = len(pools)
    if n == 0:
        return None, None, 0
    ptrs, sizes = (P * n)(), (L * n)()
    for i, t in enumerate(pools):
        _dev(t, "pool", None, cur)
        if not (t.dim() >= 1 and t.shape[0] == num_blocks):
            raise ValueError(f"a pool must hold {num_blocks} blocks, got {tuple(t.shape)}")
        ptrs[i] = t.data_ptr()
        sizes[i] = t.nbytes // num_blocks
    return ptrs, sizes, n


def pa_table_workspace_size(num_seqs, max_blocks_per_seq, num_blocks) -> int:
    return int(_lib.pa_table_workspace_size(num_seqs, max_blocks_per_seq, num_blocks))


def pa_table_step(block_tables, context_lens, ref_counts, append, block_size, slot_mapping,
                  query_start_loc, copy_pairs, release=None, fork_src=None, pools=(),
                  workspace=None, stream=None):
    """block_tables int32 [S, W], context_lens int32 [S] and ref_counts int32
    [NB], updated in place; append, release, fork_src int32 [S]; slot_mapping
    int64 [max_new_tokens], query_start_loc int32 [S + 1] and copy_pairs int64
    [S, 2] are written; pools: CUDA tensors [NB, ...] whose blocks follow."""
    s, w, nb, cur = _table_shapes(block_tables, context_lens, ref_counts)
    if not (slot_mapping.dim() == 1):
        raise ValueError("slot_mapping must be [max_new_tokens]")
    if not (tuple(query_start_loc.shape) == (s + 1,)):
        raise ValueError("query_start_loc must have num_seqs + 1 entries")
    if not (tuple(copy_pairs.shape) == (s, 2)):
        raise ValueError("copy_pairs must be [num_seqs, 2]")
    _dev(slot_mapping, "slot_mapping", torch.int64, cur)
    _dev(query_start_loc, "query_start_loc", torch.int32, cur)
    _dev(copy_pairs, "copy_pairs", torch.int64, cur)
    if workspace is not None:
        _dev(workspace, "workspace", None, cur)
    _table_step((s, w, nb, cur), block_tables, context_lens, ref_counts, append, block_size,
                slot_mapping, query_start_loc, copy_pairs, release, fork_src, pools, workspace,
                stream)


def _table_step(sizes, block_tables, context_lens, ref_counts, append, block_size, slot_mapping,
                query_start_loc, copy_pairs, release, fork_src, pools, workspace, stream):
    """pa_table_step with tables checked (sizes: _table_shapes') and outputs and
    workspace that are the caller's own."""
    s, w, nb, cur = sizes
    for name, t in (("append", append), ("release", release), ("fork_src", fork_src)):
        if t is not None:
            if t.dim() != 1 or t.shape[0] != s:
                raise ValueError(f"{name} must hold one entry per sequence")
            _dev(t, name, torch.int32, cur)
    ptrs, block_bytes, n = _pool_args(pools, nb, cur)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_table_step(_ptr(block_tables), w, _ptr(context_lens), _ptr(ref_counts),
                            _ptr(release), _ptr(fork_src), _ptr(append), s, nb, int(block_size),
                            _ptr(slot_mapping), slot_mapping.shape[0], _ptr(query_start_loc),
                            _ptr(copy_pairs), ptrs, block_bytes, n, _ptr(workspace), ws_bytes,
                            _stream(stream))
    _check(rc, "pa_table_step")


def pa_table_compact(block_tables, context_lens, ref_counts, block_size, num_live, block_moves,
                     pools=(), workspace=None, stream=None):
    """Move the used blocks to ids [0, live): block_tables, ref_counts and the
    pools' blocks are updated in place; num_live int32 [1] and block_moves
    int64 [max(1, NB // 2), 2] are written."""
    s, w, nb, cur = _table_shapes(block_tables, context_lens, ref_counts)
    if not (tuple(num_live.shape) == (1,)):
        raise ValueError("num_live must be [1]")
    if not (tuple(block_moves.shape) == (max(1, nb // 2), 2)):
        raise ValueError("block_moves must be [max(1, num_blocks // 2), 2]")
    _dev(num_live, "num_live", torch.int32, cur)
    _dev(block_moves, "block_moves", torch.int64, cur)
    if workspace is not None:
        _dev(workspace, "workspace", None, cur)
    _table_compact((s, w, nb, cur), block_tables, context_lens, ref_counts, block_size, num_live,
                   block_moves, pools, workspace, stream)


def _table_compact(sizes, block_tables, context_lens, ref_counts, block_size, num_live, block_moves,
                   pools, workspace, stream):
    """pa_table_compact, as _table_step."""
    s, w, nb, cur = sizes
    ptrs, block_bytes, n = _pool_args(pools, nb, cur)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.pa_table_compact(_ptr(block_tables), w, _ptr(context_lens), _ptr(ref_counts), s, nb,
                               int(block_size), _ptr(num_live), _ptr(block_moves), ptrs, block_bytes,
                               n, _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "pa_table_compact")


def pa_noalloc_scratch_bytes() -> int:
    return int(_lib.pa_noalloc_scratch_bytes())


def pa_get_device_error(stream=None) -> int:
    """Synchronise the stream, return and clear the device error word."""
    code = ctypes.c_uint(0)
    rc = _lib.pa_get_device_error(ctypes.byref(code), _stream(stream))
    _check(rc, "pa_get_device_error")
    return int(code.value)


def pa_abi_version() -> int:
    return int(_lib.pa_abi_version())
