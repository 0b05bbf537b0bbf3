"""Python binding of libpkv.so — paged KV-cache decode attention for GB300 (sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA library
(see include/pkv.h for the contract of each call).  torch supplies device memory
and streams.  There is no CPU fallback: the calls raise if the library is not
built or a tensor is not on a CUDA device.

Functions (same names as the C entry points without the ``pkv_`` prefix):
``kv_append``, ``paged_decode_attn``, ``paged_decode_attn_window``,
``paged_decode_attn_noalloc``, ``kv_quant_append_int4``, ``paged_decode_attn_int4``,
``paged_decode_attn_int4_window``, ``rope_shift_k``, ``copy_blocks``, ``kv_deviation``,
``select_top``, ``kv_fuse``, ``recompute_ratio``, ``select_count``, ``probe_read``,
``probe_copy``, ``layer_window`` (as ``layer_windows``), ``rope_append``, ``rope_qk``,
``kv_quant_append_q8``, ``paged_decode_attn_q8``, ``paged_decode_attn_mass``, ``kv_evict``,
``paged_tree_attn``, ``kv_tree_accept``, ``latent_append``, ``paged_latent_attn``, plus
``rope_table`` (``pkv_rope_init``), ``decode_workspace_bytes`` and the other ``*_workspace_bytes``,
``alloc_int4_cache``, ``alloc_q8_cache``, ``alloc_evict_state`` and ``BlockManager`` (the ``pkv_bm_*`` calls of
include/pkv_bm.h).
"""
from __future__ import annotations

import ctypes
import functools
import importlib
import os
from dataclasses import dataclass

import torch

from ._build import CALLS as CALLS_PATH, LIB as LIB_PATH, build_library, calls_current

PKV_OUT_BF16 = 0
PKV_OUT_F32 = 1
DEV_BAD_BLOCK, DEV_BAD_SLOT, DEV_BAD_CTX, DEV_TIMEOUT, DEV_BAD_TREE = 1, 2, 4, 8, 16

_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_SIGS = {
    "pkv_status_str": (ctypes.c_char_p, [_I]),
    "pkv_last_cuda_error": (_I, []),
    "pkv_kv_append": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P]),
    "pkv_decode_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "pkv_paged_decode_attn": (_I, [_P, _P, _P, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I,
                                   _P, _I, _P, ctypes.c_size_t, _P, _P]),
    "pkv_kv_quant_append_int4": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "pkv_int4_record_bytes": (ctypes.c_size_t, [_I, _I]),
    "pkv_paged_decode_attn_int4": (_I, [_P, _P, _P, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I,
                                        _P, _I, _P, ctypes.c_size_t, _P, _P]),
    "pkv_rope_shift_k": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_double, _P, _P]),
    "pkv_paged_decode_attn_noalloc": (_I, [_P, _P, _P, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I,
                                           _P, _I, _P, _P]),
    "pkv_paged_decode_attn_window": (_I, [_P, _P, _P, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I, _I,
                                          _P, _I, _P, ctypes.c_size_t, _P, _P]),
    "pkv_paged_decode_attn_int4_window": (_I, [_P, _P, _P, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I,
                                               _I, _P, _I, _P, ctypes.c_size_t, _P, _P]),
    # rotary positions, the 8-bit cache, accounted attention and eviction
    "pkv_rope_init": (_I, [_P, _P]),
    "pkv_rope_append": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _I, _P, _P, _L, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "pkv_rope_qk": (_I, [_P, _L, _P, _L, _P, _I, _P, _P, _L, _P, _L, _I, _I, _I, _P]),
    "pkv_q8_record_bytes": (ctypes.c_size_t, [_I, _I]),
    "pkv_kv_quant_append_q8": (_I, [_P, _L, _P, _L, _P, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "pkv_q8_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "pkv_paged_decode_attn_q8": (_I, [_P, _P, _I, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I, _I,
                                      _P, _I, _P, ctypes.c_size_t, _P, _P]),
    "pkv_mass_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "pkv_paged_decode_attn_mass": (_I, [_P, _P, _P, _P, _I, _P, ctypes.c_float, _I, _I, _I, _I, _I, _I,
                                        _P, _I, _P, _L, _P, ctypes.c_size_t, _P, _P]),
    "pkv_evict_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "pkv_kv_evict": (_I, [_P, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _L, _P, _I, _I, _I, _I, _I,
                          _P, ctypes.c_size_t, _P, _P]),
    # drafted tokens and the latent cache
    "pkv_tree_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "pkv_paged_tree_attn": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _I, ctypes.c_float, _I, _I, _I, _I, _I, _I, _I,
                                 _P, _I, _P, ctypes.c_size_t, _P, _P]),
    "pkv_kv_tree_accept": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _P, _P]),
    "pkv_latent_append": (_I, [_P, _L, _P, _L, _L, _P, _P, _I, _P, _P, ctypes.c_float, _P, _L, _L, _P, _I, _I, _I, _I, _I,
                               _P, _P]),
    "pkv_latent_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "pkv_paged_latent_attn": (_I, [_P, _P, _P, _I, _P, _P, _P, _I, ctypes.c_float, _I, _I, _I, _I, _I, _I, _I,
                                   _P, _I, _P, ctypes.c_size_t, _P, _P]),
    # block manager (host) and its copy executor
    "pkv_bm_create": (_P, [_I, _I, _I, _I, _I]),
    "pkv_bm_destroy": (None, [_P]),
    "pkv_bm_add_sequence": (_I, [_P, ctypes.c_int64, _P, _I, _P, _I, _P, _I]),
    "pkv_bm_append_tokens": (_I, [_P, _P, _P, _I, _P, _P]),
    "pkv_bm_append_drafts": (_I, [_P, ctypes.c_int64, _I, _P]),
    "pkv_bm_accept_drafts": (_I, [_P, ctypes.c_int64, _P, _I]),
    "pkv_bm_release": (_I, [_P, ctypes.c_int64]),
    "pkv_bm_slide_window": (_I, [_P, ctypes.c_int64, _I]),
    "pkv_bm_evict": (_I, [_P, ctypes.c_int64, _I]),
    "pkv_bm_tables": (_I, [_P, _P, _I, _P, _I, _P]),
    "pkv_bm_take_copies": (_I, [_P, _P, _I]),
    "pkv_bm_pending_copies": (_I, [_P]),
    "pkv_bm_counts": (None, [_P, _P]),
    "pkv_copy_blocks": (_I, [_P, _I, _P, _P, _I, _P, _P, _I, ctypes.c_size_t, _P]),
    # CacheBlend's model-free steps
    "pkv_kv_deviation": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "pkv_select_top": (_I, [_P, _P, _P, _I, _P, _P]),
    "pkv_kv_fuse": (_I, [_P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P]),
    "pkv_recompute_ratio": (ctypes.c_double, [ctypes.c_double, ctypes.c_double]),
    "pkv_select_count": (_I, [ctypes.c_double, _I]),
    "pkv_selftest_wait": (_I, [_I, _I, _P, _P]),
    "pkv_layer_window": (_I, [_P, _I, _I]),
    "pkv_probe_read": (_I, [_P, ctypes.c_size_t, _P, _P]),
    "pkv_probe_copy": (_I, [_P, _P, ctypes.c_size_t, _P]),
}
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024


class PkvError(RuntimeError):
    pass


def lib(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libpkv.so (fails loudly if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            if not build_if_missing:
                raise PkvError(f"{LIB_PATH} is missing: build it with paged_kv_cache_175_gb300._build.build_library()")
            build_library()
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _check(name: str, status: int):
    if status != 0:
        msg = lib().pkv_status_str(status).decode()
        extra = f" (cuda error {lib().pkv_last_cuda_error()})" if status == -3 else ""
        raise PkvError(f"{name}: {msg}{extra}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise PkvError("tensors must be contiguous CUDA tensors")


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def kv_append(k, v, slot_mapping, k_pool, v_pool, err=None, stream=None):
    """Write k, v [n_tok][n_kv][d] (bf16) into the pools at slot_mapping (int64)."""
    _cuda(k, v, slot_mapping, k_pool, v_pool, err)
    assert k.dtype == v.dtype == k_pool.dtype == v_pool.dtype == torch.bfloat16
    assert slot_mapping.dtype == torch.int64
    num_blocks, n_kv, bs, d = k_pool.shape
    _check("kv_append", lib().pkv_kv_append(_ptr(k), _ptr(v), _ptr(slot_mapping), k.shape[0], _ptr(k_pool),
                                            _ptr(v_pool), num_blocks, bs, n_kv, d, _ptr(err), _stream(stream)))


def decode_workspace_bytes(batch, n_h, n_kv, head_dim, block_size, int4=False) -> int:
    n = lib().pkv_decode_workspace_bytes(batch, n_h, n_kv, head_dim, block_size, 1 if int4 else 0)
    if n == 0 and batch > 0:
        raise PkvError("decode_workspace_bytes: invalid shape or no device")
    return n


# Buffers that a call makes itself come from the pool of the stream it runs on: a block just freed on another
# stream may still be in use by work queued there, which nothing makes this stream wait for.
def _scratch(nbytes, device, stream):
    """A workspace of nbytes for a call on `stream`, which alone uses it."""
    if nbytes == 0:
        raise PkvError("unsupported shape or no device")
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream`; it may be used on the current stream, too (once that waits)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    if out.is_cuda:
        out.record_stream(torch.cuda.current_stream(out.device))
    return out


def _out(q, out, out_dtype, stream):
    if out is None:
        out = _empty(q.shape, out_dtype, q.device, stream)
    assert out.shape == q.shape and out.dtype in (torch.bfloat16, torch.float32)
    return out, (PKV_OUT_F32 if out.dtype == torch.float32 else PKV_OUT_BF16)


def paged_decode_attn(q, k_pool, v_pool, block_tables, context_lens, scale, out=None, out_dtype=torch.bfloat16,
                      workspace=None, err=None, stream=None):
    """Decode attention over a paged bf16 cache; returns out [B][n_h][d]."""
    return _decode_bf16(q, k_pool, v_pool, block_tables, context_lens, scale, 0, out, out_dtype, workspace, err,
                        stream)


def paged_decode_attn_window(q, k_pool, v_pool, block_tables, context_lens, scale, window, out=None,
                             out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """Decode attention over the last `window` tokens of each context (0: all of it)."""
    return _decode_bf16(q, k_pool, v_pool, block_tables, context_lens, scale, int(window), out, out_dtype,
                        workspace, err, stream)


def layer_windows(max_attention_window, n_layers):
    """Attention window of each of n_layers layers from a max_attention_window list
    (pkv_layer_window: the list repeated over the layers)."""
    import numpy as np
    w = np.ascontiguousarray(max_attention_window, dtype=np.int32).reshape(-1)
    out = [lib().pkv_layer_window(w.ctypes.data, len(w), i) for i in range(max(int(n_layers), 1))]
    if any(x < 0 for x in out):
        raise ValueError("max_attention_window must be a non-empty list of positive token counts")
    return out[:int(n_layers)]


def _decode_bf16(q, k_pool, v_pool, block_tables, context_lens, scale, window, out, out_dtype, workspace, err,
                 stream):
    _cuda(q, k_pool, v_pool, block_tables, context_lens, out, workspace, err)
    assert q.dtype == k_pool.dtype == v_pool.dtype == torch.bfloat16
    assert block_tables.dtype == context_lens.dtype == torch.int32
    B, n_h, d = q.shape
    num_blocks, n_kv, bs, d2 = k_pool.shape
    assert d2 == d and v_pool.shape == k_pool.shape
    out, od = _out(q, out, out_dtype, stream)
    need = decode_workspace_bytes(B, n_h, n_kv, d, bs)
    if workspace is None:
        workspace = _scratch(max(need, 256), q.device, stream)
    if window == 0:
        _check("paged_decode_attn", lib().pkv_paged_decode_attn(
            _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
            float(scale), B, n_h, n_kv, d, bs, num_blocks, _ptr(out), od, _ptr(workspace), workspace.numel(),
            _ptr(err), _stream(stream)))
    else:
        _check("paged_decode_attn_window", lib().pkv_paged_decode_attn_window(
            _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
            float(scale), window, B, n_h, n_kv, d, bs, num_blocks, _ptr(out), od, _ptr(workspace),
            workspace.numel(), _ptr(err), _stream(stream)))
    return out


def paged_decode_attn_noalloc(q, k_pool, v_pool, block_tables, context_lens, scale, out=None,
                              out_dtype=torch.bfloat16, err=None, stream=None):
    """paged_decode_attn with the library's fixed internal scratch instead of a workspace
    (for callers that cannot allocate device memory; concurrent calls must not overlap)."""
    _cuda(q, k_pool, v_pool, block_tables, context_lens, out, err)
    assert q.dtype == k_pool.dtype == v_pool.dtype == torch.bfloat16
    assert block_tables.dtype == context_lens.dtype == torch.int32
    B, n_h, d = q.shape
    num_blocks, n_kv, bs, d2 = k_pool.shape
    assert d2 == d and v_pool.shape == k_pool.shape
    assert block_tables.dim() == 2 and block_tables.shape[0] == B and context_lens.shape == (B,)
    out, od = _out(q, out, out_dtype, stream)
    _check("paged_decode_attn_noalloc", lib().pkv_paged_decode_attn_noalloc(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
        float(scale), B, n_h, n_kv, d, bs, num_blocks, _ptr(out), od, _ptr(err), _stream(stream)))
    return out


def int4_record_bytes(block_size, head_dim) -> int:
    """Bytes of one (block, kv head) record of the INT4 cache (0 for an unsupported shape)."""
    return int(lib().pkv_int4_record_bytes(int(block_size), int(head_dim)))


@dataclass
class Int4CacheTensors:
    """INT4 paged cache: one record per (block, kv head) -- K codes, V codes, K scale and
    min rows, V (scale, min) per token -- plus the bf16 K rows of unfinished blocks.  The
    four fields of the records are exposed as views."""
    records: torch.Tensor     # uint8 [num_blocks][n_kv][int4_record_bytes(bs, d)]
    k_tail: torch.Tensor      # bf16  [tail_rows][n_kv][bs][d]

    @property
    def shape(self):
        _, n_kv, bs, d = self.k_tail.shape
        return self.records.shape[0], n_kv, bs, d

    def _field(self, start, size):
        return self.records[:, :, start:start + size]

    @property
    def k_codes(self):         # uint8 [num_blocks][n_kv][bs][d/2]
        nb, n_kv, bs, d = self.shape
        return self._field(0, bs * d // 2).view(nb, n_kv, bs, d // 2)

    @property
    def v_codes(self):         # uint8 [num_blocks][n_kv][bs][d/2]
        nb, n_kv, bs, d = self.shape
        return self._field(bs * d // 2, bs * d // 2).view(nb, n_kv, bs, d // 2)

    @property
    def k_meta(self):          # fp16 [num_blocks][n_kv][2][d]: scale row, min row
        nb, n_kv, bs, d = self.shape
        return self._field(bs * d, 4 * d).view(torch.float16).view(nb, n_kv, 2, d)

    @property
    def v_meta(self):          # fp16 [num_blocks][n_kv][bs][2]: (scale, min) per token
        nb, n_kv, bs, d = self.shape
        return self._field(bs * d + 4 * d, 4 * bs).view(torch.float16).view(nb, n_kv, bs, 2)


def alloc_int4_cache(num_blocks, n_kv, block_size, head_dim, tail_rows, device="cuda") -> Int4CacheTensors:
    rec = int4_record_bytes(block_size, head_dim)
    if rec == 0:
        raise ValueError(f"INT4 cache: unsupported block_size {block_size} / head_dim {head_dim}")
    return Int4CacheTensors(torch.zeros(num_blocks, n_kv, rec, dtype=torch.uint8, device=device),
                            torch.zeros(tail_rows, n_kv, block_size, head_dim, dtype=torch.bfloat16, device=device))


def kv_quant_append_int4(k, v, slot_mapping, tail_seq, cache: Int4CacheTensors, err=None, stream=None):
    """Quantize-on-append of k, v [n_tok][n_kv][d] into the INT4 cache."""
    _cuda(k, v, slot_mapping, tail_seq, cache.records, cache.k_tail, err)
    assert k.dtype == v.dtype == torch.bfloat16 and slot_mapping.dtype == torch.int64
    assert tail_seq.dtype == torch.int32
    nb, n_kv, bs, d = cache.shape
    _check("kv_quant_append_int4", lib().pkv_kv_quant_append_int4(
        _ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(tail_seq), k.shape[0], _ptr(cache.records), _ptr(cache.k_tail),
        cache.k_tail.shape[0], nb, bs, n_kv, d, _ptr(err), _stream(stream)))


def paged_decode_attn_int4(q, cache: Int4CacheTensors, block_tables, context_lens, scale, out=None,
                           out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """Decode attention over the INT4 cache; the batch index is the tail row."""
    return _decode_int4(q, cache, block_tables, context_lens, scale, 0, out, out_dtype, workspace, err, stream)


def paged_decode_attn_int4_window(q, cache: Int4CacheTensors, block_tables, context_lens, scale, window, out=None,
                                  out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """INT4 decode attention over the last `window` tokens of each context (0: all of it)."""
    return _decode_int4(q, cache, block_tables, context_lens, scale, int(window), out, out_dtype, workspace, err,
                        stream)


def _decode_int4(q, cache, block_tables, context_lens, scale, window, out, out_dtype, workspace, err, stream):
    _cuda(q, block_tables, context_lens, out, workspace, err)
    assert q.dtype == torch.bfloat16
    B, n_h, d = q.shape
    nb, n_kv, bs, d2 = cache.shape
    assert d2 == d and cache.k_tail.shape[0] >= B
    out, od = _out(q, out, out_dtype, stream)
    need = decode_workspace_bytes(B, n_h, n_kv, d, bs, int4=True)
    if workspace is None:
        workspace = _scratch(max(need, 256), q.device, stream)
    if window == 0:
        _check("paged_decode_attn_int4", lib().pkv_paged_decode_attn_int4(
            _ptr(q), _ptr(cache.records), _ptr(cache.k_tail), _ptr(block_tables), block_tables.shape[1],
            _ptr(context_lens), float(scale), B, n_h, n_kv, d, bs, nb, _ptr(out), od, _ptr(workspace), workspace.numel(), _ptr(err), _stream(stream)))
    else:
        _check("paged_decode_attn_int4_window", lib().pkv_paged_decode_attn_int4_window(
            _ptr(q), _ptr(cache.records), _ptr(cache.k_tail), _ptr(block_tables), block_tables.shape[1],
            _ptr(context_lens), float(scale), window, B, n_h, n_kv, d, bs, nb, _ptr(out), od, _ptr(workspace), workspace.numel(), _ptr(err),
            _stream(stream)))
    return out


def rope_shift_k(k_pool, block_ids, deltas, rope_base=10000.0, err=None, stream=None):
    """Rotate every key of block block_ids[i] by position deltas[i] in place."""
    _cuda(k_pool, block_ids, deltas, err)
    assert k_pool.dtype == torch.bfloat16 and block_ids.dtype == deltas.dtype == torch.int32
    num_blocks, n_kv, bs, d = k_pool.shape
    _check("rope_shift_k", lib().pkv_rope_shift_k(_ptr(k_pool), _ptr(block_ids), _ptr(deltas), block_ids.numel(),
                                                  num_blocks, n_kv, bs, d, float(rope_base), _ptr(err),
                                                  _stream(stream)))


# ---------------------------------------------------------------------------------------------
# Rotary positions, the 8-bit cache, accounted attention and eviction (pkv.h).
ROPE_SCALINGS = ("none", "linear", "ntk", "parts", "yarn")
Q8_FORMATS = ("e4m3", "int8")


class _RopeConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("amplitude", ctypes.c_double)]


class RopeTable(ctypes.Structure):
    """Angle table of a rotary embedding (rope_table); plain data, not to be changed."""
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("turns", ctypes.c_uint64 * 64)]


@functools.lru_cache(maxsize=64)
def rope_table(head_dim, rotary_dim=None, base=10000.0, interleaved=False, scaling="none", factor=1.0,
               original_len=0.0, low=1.0, high=32.0, amplitude=0.0) -> RopeTable:
    """The angle table for rope_append / rope_qk: rotary_dim channels of head_dim (all by default) in
    half or interleaved pairs, with a scaling for contexts `factor` times original_len (pkv_rope_init)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {ROPE_SCALINGS}")
    c = _RopeConfig(int(head_dim), int(head_dim if rotary_dim is None else rotary_dim), 1 if interleaved else 0,
                    ROPE_SCALINGS.index(scaling), float(base), float(factor), float(original_len), float(low),
                    float(high), float(amplitude))
    t = RopeTable()
    _check("rope_init", lib().pkv_rope_init(ctypes.byref(c), ctypes.byref(t)))
    return t


# The tensors of the calls below are checked and passed on by a small extension (csrc/calls.cpp): a call
# of a few microseconds on the GPU should not wait for its checks.  Where the extension answers
# _NOT_TAKEN it called nothing, and the checks after it name the mistake.
_bf16, _f32, _i32, _i64, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
_NOT_TAKEN = 1
_calls = None


def _native():
    """The extension (fails loudly if it has not been built)."""
    global _calls
    if _calls is None:
        lib()
        if not calls_current():
            raise PkvError(f"{CALLS_PATH} is missing, or was built for another torch or Python: build it with "
                           "paged_kv_cache_175_gb300._build.build_library()")
        _calls = importlib.import_module("._calls", __name__)
    return _calls


def _failed(name, status):
    if status == _NOT_TAKEN:
        raise PkvError(f"{name}: unsupported arguments")
    _check(name, status)


def _on_current(*ts):
    """All tensors (None is skipped) on the current CUDA device."""
    if not ts[0].is_cuda:
        raise PkvError("tensors must be CUDA tensors")
    d = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != d:             # -1 for a CPU tensor
            raise PkvError("tensors must be on the current CUDA device")


def _dense(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise PkvError("tensors must be contiguous")


def _typed(dtype, *ts):
    for t in ts:
        if t is not None and t.dtype != dtype:
            raise PkvError(f"expected {dtype}, got {t.dtype}")


def _shaped(what, t, *shape):
    if t is not None and tuple(t.shape) != shape:
        raise PkvError(f"{what} must have shape {shape}, got {tuple(t.shape)}")


def _dims(what, t, n):
    if t.dim() != n:
        raise PkvError(f"{what} must have {n} dimensions, got {t.dim()}")
    return t.shape


def _head_dense(t):
    """The heads of a token of [n_tok][heads][head_dim] are contiguous (tokens may be strided)."""
    _, h, d = t.shape
    if t.numel() and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d)):
        raise PkvError("the heads of a token must be contiguous")


def _table_type(table):
    if type(table) is not RopeTable:
        raise PkvError("the table must come from rope_table")


def _out_type(out_dtype):
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise PkvError("out_dtype must be bfloat16 or float32")
    return out_dtype


def rope_append(q, k, v, positions, slot_mapping, table: RopeTable, k_pool, v_pool, q_out=None, err=None, stream=None):
    """Rotate q and k [n_tok][heads][d] by positions (int32) and append k and v to the bf16 cache;
    returns the rotated q.  Tokens may be strided (parts of one fused projection); q_out may be q."""
    _table_type(table)
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    st = (_calls or _native()).rope_append(q, k, v, positions, slot_mapping, table, k_pool, v_pool, q_out, err,
                                           None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        n, n_h, d = _dims("q", q, 3)
        num_blocks, n_kv, bs, _ = _dims("k_pool", k_pool, 4)
        _on_current(q, k, v, positions, slot_mapping, k_pool, v_pool, q_out, err)
        _typed(_bf16, q, k, v, k_pool, v_pool, q_out)
        _typed(_i32, positions, err)
        _typed(_i64, slot_mapping)
        _shaped("k", k, n, n_kv, d)
        _shaped("v", v, n, n_kv, d)
        _shaped("positions", positions, n)
        _shaped("slot_mapping", slot_mapping, n)
        _shaped("k_pool", k_pool, num_blocks, n_kv, bs, d)
        _shaped("v_pool", v_pool, num_blocks, n_kv, bs, d)
        _shaped("q_out", q_out, n, n_h, d)
        _dense(positions, slot_mapping, k_pool, v_pool)
        for t in (q, k, v, q_out):
            _head_dense(t)
    if st:
        _failed("rope_append", st)
    return q_out


def rope_qk(q, k, positions, table: RopeTable, q_out=None, k_out=None, stream=None):
    """Rotate q and k [n_tok][heads][d] by positions (int32); returns (q_out, k_out), which may be
    given as q and k themselves."""
    _table_type(table)
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    if k_out is None:
        k_out = _empty(k.shape, k.dtype, k.device, stream)
    st = (_calls or _native()).rope_qk(q, k, positions, table, q_out, k_out,
                                       None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        n, n_h, d = _dims("q", q, 3)
        n_kv = _dims("k", k, 3)[1]
        _on_current(q, k, positions, q_out, k_out)
        _typed(_bf16, q, k, q_out, k_out)
        _typed(_i32, positions)
        _shaped("k", k, n, n_kv, d)
        _shaped("positions", positions, n)
        _shaped("q_out", q_out, n, n_h, d)
        _shaped("k_out", k_out, n, n_kv, d)
        _dense(positions)
        for t in (q, k, q_out, k_out):
            _head_dense(t)
    if st:
        _failed("rope_qk", st)
    return q_out, k_out


def q8_record_bytes(block_size, head_dim) -> int:
    """Bytes of one (block, kv head) record of the 8-bit cache (0 for an unsupported shape)."""
    return int(lib().pkv_q8_record_bytes(int(block_size), int(head_dim)))


@dataclass
class Q8CacheTensors:
    """8-bit paged cache: one record per (block, kv head) -- K codes, V codes in the order of pkv.h,
    K and V scale -- and the bf16 rows of each sequence's unfinished block."""
    records: torch.Tensor     # uint8 [num_blocks][n_kv][q8_record_bytes(bs, d)]
    k_tail: torch.Tensor      # bf16  [tail_rows][n_kv][bs][d]
    v_tail: torch.Tensor
    fmt: str = "e4m3"         # or "int8"

    @property
    def shape(self):
        _, n_kv, bs, d = self.k_tail.shape
        return self.records.shape[0], n_kv, bs, d

    @property
    def scales(self):         # fp32 [num_blocks][n_kv][2]: K, V (a view)
        _, _, bs, d = self.shape
        return self.records[:, :, 2 * bs * d:2 * bs * d + 8].view(torch.float32)

    def _codes(self, keys):
        nb, n_kv, bs, d = self.shape
        x = self.records[:, :, (0 if keys else bs * d):(bs * d if keys else 2 * bs * d)]
        # 16-token tile, group of 32 channels, lane (i, j), bytes (a, b, c, e) of pkv.h
        x = x.reshape(nb, n_kv, bs // 16, d // 32, 8, 4, 2, 2, 2, 2)
        order = (0, 1, 2, 7, 4, 3, 6, 8, 5, 9) if keys else (0, 1, 2, 8, 5, 9, 3, 6, 7, 4)
        return x.permute(order).reshape(nb, n_kv, bs, d).view(torch.float8_e4m3fn if self.fmt == "e4m3" else torch.int8)

    @property
    def k_codes(self):        # [num_blocks][n_kv][bs][d], token by token (a copy)
        return self._codes(True)

    @property
    def v_codes(self):
        return self._codes(False)


def alloc_q8_cache(num_blocks, n_kv, block_size, head_dim, tail_rows, fmt="e4m3", device="cuda") -> Q8CacheTensors:
    rec = q8_record_bytes(block_size, head_dim)
    if rec == 0 or fmt not in Q8_FORMATS:
        raise ValueError(f"8-bit cache: unsupported block_size {block_size} / head_dim {head_dim} / format {fmt}")
    tail = lambda: torch.zeros(tail_rows, n_kv, block_size, head_dim, dtype=torch.bfloat16, device=device)
    return Q8CacheTensors(torch.zeros(num_blocks, n_kv, rec, dtype=torch.uint8, device=device), tail(), tail(), fmt)


def _q8_refuse(cache):
    nb, n_kv, bs, d = cache.shape
    _typed(_u8, cache.records)
    _typed(_bf16, cache.k_tail, cache.v_tail)
    _dense(cache.records, cache.k_tail, cache.v_tail)
    _shaped("v_tail", cache.v_tail, *cache.k_tail.shape)
    _shaped("records", cache.records, nb, n_kv, 2 * bs * d + 16)


def _q8_format(cache):
    if cache.fmt not in Q8_FORMATS:
        raise PkvError(f"format must be one of {Q8_FORMATS}")
    return 0 if cache.fmt == "e4m3" else 1


def kv_quant_append_q8(k, v, slot_mapping, tail_seq, cache: Q8CacheTensors, err=None, stream=None):
    """Quantize-on-append of k, v [n_tok][n_kv][d] (tokens may be strided) into the 8-bit cache."""
    fmt = _q8_format(cache)
    st = (_calls or _native()).kv_quant_append_q8(k, v, slot_mapping, tail_seq, cache.records, cache.k_tail, cache.v_tail, fmt,
                                                  err, None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        n = _dims("k", k, 3)[0]
        _, n_kv, bs, d = _dims("k_tail", cache.k_tail, 4)
        _on_current(k, v, slot_mapping, tail_seq, cache.records, cache.k_tail, cache.v_tail, err)
        _typed(_bf16, k, v)
        _typed(_i64, slot_mapping)
        _typed(_i32, tail_seq, err)
        _shaped("k", k, n, n_kv, d)
        _shaped("v", v, n, n_kv, d)
        _shaped("slot_mapping", slot_mapping, n)
        _shaped("tail_seq", tail_seq, n)
        _dense(slot_mapping, tail_seq)
        _q8_refuse(cache)
        for t in (k, v):
            _head_dense(t)
    if st:
        _failed("kv_quant_append_q8", st)


def q8_workspace_bytes(batch, n_h, n_kv, head_dim, block_size, fmt="e4m3") -> int:
    """Bytes of workspace paged_decode_attn_q8 needs for this shape on the current device."""
    n = lib().pkv_q8_workspace_bytes(batch, n_h, n_kv, head_dim, block_size, Q8_FORMATS.index(fmt))
    if n == 0:
        raise PkvError("q8_workspace_bytes: invalid shape or no device")
    return n


def paged_decode_attn_q8(q, cache: Q8CacheTensors, block_tables, context_lens, scale, window=0, out=None,
                         out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """Decode attention over the 8-bit cache (the last `window` tokens of each context; 0: all).  A bfloat16
    output of groups of over four query heads takes the softmax weights rounded to fp16 once (2^-11); a float32
    output takes 22 bits of them."""
    fmt = _q8_format(cache)
    if out is None:
        out = _empty(q.shape, _out_type(out_dtype), q.device, stream)
    if workspace is None and q.is_cuda and q.shape[0]:
        _, n_kv, bs, d = _dims("k_tail", cache.k_tail, 4)
        B, n_h, _ = _dims("q", q, 3)
        workspace = _scratch(lib().pkv_q8_workspace_bytes(B, n_h, n_kv, d, bs, fmt), q.device, stream)
    st = (_calls or _native()).paged_decode_attn_q8(q, cache.records, cache.k_tail, cache.v_tail, fmt, block_tables,
                                                    context_lens, scale, int(window), out, workspace, err,
                                                    None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        d = _dims("k_tail", cache.k_tail, 4)[3]
        B, n_h, _ = _dims("q", q, 3)
        _dims("block_tables", block_tables, 2)
        _on_current(q, cache.records, cache.k_tail, cache.v_tail, block_tables, context_lens, out, workspace, err)
        _typed(_bf16, q)
        _typed(_i32, block_tables, context_lens, err)
        _out_type(out.dtype)
        _shaped("q", q, B, n_h, d)
        _shaped("block_tables", block_tables, B, block_tables.shape[1])
        _shaped("context_lens", context_lens, B)
        _shaped("out", out, B, n_h, d)
        _dense(q, block_tables, context_lens, out, workspace)
        _q8_refuse(cache)
    if st:
        _failed("paged_decode_attn_q8", st)
    return out


def mass_workspace_bytes(batch, n_h, n_kv, head_dim, block_size, max_blocks) -> int:
    """Bytes of workspace paged_decode_attn_mass needs for this shape on the current device."""
    n = lib().pkv_mass_workspace_bytes(batch, n_h, n_kv, head_dim, block_size, max_blocks)
    if n == 0:
        raise PkvError("mass_workspace_bytes: invalid shape or no device")
    return n


def paged_decode_attn_mass(q, k_pool, v_pool, block_tables, context_lens, scale, mass, out=None,
                           out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """paged_decode_attn that also adds each cached token's attention weight, summed over the query
    heads of its group, to mass (fp32 [B][n_kv][at least max_blocks * block_size]).  The softmax weights
    reach the output with all their bits (a bfloat16 output of groups of over eight heads: 16 of them)."""
    if out is None:
        out = _empty(q.shape, _out_type(out_dtype), q.device, stream)
    if workspace is None and q.is_cuda and q.shape[0]:
        B, n_h, d = _dims("q", q, 3)
        _, n_kv, bs, _ = _dims("k_pool", k_pool, 4)
        mb = _dims("block_tables", block_tables, 2)[1]
        workspace = _scratch(lib().pkv_mass_workspace_bytes(B, n_h, n_kv, d, bs, mb), q.device, stream)
    st = (_calls or _native()).paged_decode_attn_mass(q, k_pool, v_pool, block_tables, context_lens, scale, mass, out, workspace,
                                                      err, None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        B, n_h, d = _dims("q", q, 3)
        nb, n_kv, bs, _ = _dims("k_pool", k_pool, 4)
        mb = _dims("block_tables", block_tables, 2)[1]
        T = _dims("mass", mass, 3)[2]
        _on_current(q, k_pool, v_pool, block_tables, context_lens, mass, out, workspace, err)
        _typed(_bf16, q, k_pool, v_pool)
        _typed(_i32, block_tables, context_lens, err)
        _typed(_f32, mass)
        _out_type(out.dtype)
        _shaped("k_pool", k_pool, nb, n_kv, bs, d)
        _shaped("v_pool", v_pool, nb, n_kv, bs, d)
        _shaped("block_tables", block_tables, B, mb)
        _shaped("context_lens", context_lens, B)
        _shaped("mass", mass, B, n_kv, T)
        _shaped("out", out, B, n_h, d)
        _dense(q, k_pool, v_pool, block_tables, context_lens, mass, out, workspace)
    if st:
        _failed("paged_decode_attn_mass", st)
    return out


@dataclass
class EvictState:
    """What kv_evict keeps of each sequence (pkv.h): accounts, recorded positions, counts."""
    mass: torch.Tensor        # fp32  [B][n_kv][T]
    positions: torch.Tensor   # int32 [B][n_kv][T]
    kept: torch.Tensor        # int32 [B]
    dropped: torch.Tensor     # int32 [B]

    def reset(self, s):
        """Make row s ready for a new sequence."""
        self.mass[s].zero_()
        self.kept[s] = 0
        self.dropped[s] = 0


def alloc_evict_state(batch, n_kv, max_tokens, device="cuda") -> EvictState:
    """State for sequences of up to max_tokens rows (a multiple of the block size)."""
    z = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device=device)
    return EvictState(z(batch, n_kv, max_tokens, dtype=torch.float32), z(batch, n_kv, max_tokens), z(batch), z(batch))


def evict_workspace_bytes(batch, n_kv, block_size, max_blocks) -> int:
    n = lib().pkv_evict_workspace_bytes(batch, n_kv, block_size, max_blocks)
    if n == 0:
        raise PkvError("evict_workspace_bytes: invalid shape")
    return n


def kv_evict(k_pool, v_pool, block_tables, context_lens, keep, recent, state: EvictState, out: EvictState | None = None,
             new_lens=None, workspace=None, err=None, stream=None):
    """Cut each sequence of the bf16 cache to keep[s] rows (int32 [B]): those of its last `recent`
    tokens and those with the largest accounts.  With a BlockManager, `keep` comes from its cut_to, which goes
    first and knows whose rows may move.  Updates `state` in place, or writes the new state to
    `out`; returns the new context lengths (a tensor of its own)."""
    dst = state if out is None else out
    if new_lens is None:
        new_lens = _empty(context_lens.shape, _i32, context_lens.device, stream)
    if workspace is None and k_pool.is_cuda and block_tables.shape[0]:
        B, mb = _dims("block_tables", block_tables, 2)
        _, n_kv, bs, _ = _dims("k_pool", k_pool, 4)
        workspace = _scratch(lib().pkv_evict_workspace_bytes(B, n_kv, bs, mb), k_pool.device, stream)
    st = (_calls or _native()).kv_evict(k_pool, v_pool, block_tables, context_lens, keep, int(recent), state.mass,
                                        state.positions, state.kept, state.dropped, dst.mass, dst.positions, dst.kept,
                                        dst.dropped, new_lens, workspace, err,
                                        None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        nb, n_kv, bs, d = _dims("k_pool", k_pool, 4)
        B, mb = _dims("block_tables", block_tables, 2)
        T = _dims("mass", state.mass, 3)[2]
        _on_current(k_pool, v_pool, block_tables, context_lens, keep, state.mass, state.positions, state.kept,
                    state.dropped, dst.mass, dst.positions, dst.kept, dst.dropped, new_lens, workspace, err)
        _typed(_bf16, k_pool, v_pool)
        _typed(_i32, block_tables, context_lens, keep, state.positions, state.kept, state.dropped, dst.positions,
               dst.kept, dst.dropped, new_lens, err)
        _typed(_f32, state.mass, dst.mass)
        _shaped("v_pool", v_pool, nb, n_kv, bs, d)
        for es in (state, dst):
            _shaped("mass", es.mass, B, n_kv, T)
            _shaped("positions", es.positions, B, n_kv, T)
            _shaped("kept", es.kept, B)
            _shaped("dropped", es.dropped, B)
        _shaped("context_lens", context_lens, B)
        _shaped("keep", keep, B)
        _shaped("new_lens", new_lens, B)
        _dense(k_pool, v_pool, block_tables, context_lens, keep, state.mass, state.positions, state.kept, state.dropped,
               dst.mass, dst.positions, dst.kept, dst.dropped, new_lens, workspace)
    if st:
        _failed("kv_evict", st)
    return new_lens


# ---------------------------------------------------------------------------------------------
# Drafted tokens (several per sequence and step) and the latent cache (pkv.h).
def _step_refuse(q, block_tables, context_lens, q_start, tree_mask, out, workspace, err, w, v):
    T, n_h, _ = _dims("q", q, 3)
    B, _ = _dims("block_tables", block_tables, 2)
    _on_current(q, block_tables, context_lens, q_start, tree_mask, out, workspace, err)
    _typed(_bf16, q)
    _typed(_i32, block_tables, context_lens, err)
    _out_type(out.dtype)
    _shaped("q", q, T, n_h, w)
    _shaped("context_lens", context_lens, B)
    _shaped("out", out, T, n_h, v)
    if q_start is not None:
        _typed(_i32, q_start)
        _shaped("q_start", q_start, B + 1)
    elif B and T % B:
        raise PkvError(f"without q_start the {T} tokens must be a multiple of the {B} sequences")
    if tree_mask is not None:
        _typed(_i64, tree_mask)
        _shaped("tree_mask", tree_mask, T, _dims("tree_mask", tree_mask, 2)[1])
    _dense(q, block_tables, context_lens, q_start, tree_mask, out, workspace)


def tree_workspace_bytes(batch, n_tok, n_h, n_kv, head_dim, block_size) -> int:
    """Bytes of workspace paged_tree_attn needs for this shape on the current device."""
    n = lib().pkv_tree_workspace_bytes(batch, n_tok, n_h, n_kv, head_dim, block_size)
    if n == 0:
        raise PkvError("tree_workspace_bytes: invalid shape or no device")
    return n


def paged_tree_attn(q, k_pool, v_pool, block_tables, context_lens, scale, q_start=None, tree_mask=None, out=None,
                    out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """Attention of several (drafted) tokens per sequence, q [n_tok][n_h][d], over a paged bf16 cache that holds
    their rows already, as each sequence's last ones (context_lens counts them).  q_start (int32 [B + 1]): each
    sequence's first token; None: n_tok / B tokens each.  tree_mask (int64 [n_tok][words]): bit j of a token's
    words says whether it attends to token j of its sequence; None: to the earlier ones and itself."""
    if out is None:
        out = _empty(q.shape, _out_type(out_dtype), q.device, stream)
    if workspace is None and q.is_cuda and q.shape[0]:
        T, n_h, d = _dims("q", q, 3)
        _, n_kv, bs, _ = _dims("k_pool", k_pool, 4)
        workspace = _scratch(lib().pkv_tree_workspace_bytes(block_tables.shape[0], T, n_h, n_kv, d, bs), q.device, stream)
    st = (_calls or _native()).paged_tree_attn(q, k_pool, v_pool, block_tables, context_lens, scale, q_start, tree_mask, out,
                                               workspace, err, None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        nb, n_kv, bs, d = _dims("k_pool", k_pool, 4)
        _on_current(q, k_pool, v_pool)
        _typed(_bf16, k_pool, v_pool)
        _shaped("v_pool", v_pool, nb, n_kv, bs, d)
        _dense(k_pool, v_pool)
        _step_refuse(q, block_tables, context_lens, q_start, tree_mask, out, workspace, err, d, d)
    if st:
        _failed("paged_tree_attn", st)
    return out


def latent_workspace_bytes(batch, n_tok, n_h, latent, rope, block_size) -> int:
    """Bytes of workspace paged_latent_attn needs for this shape on the current device."""
    n = lib().pkv_latent_workspace_bytes(batch, n_tok, n_h, latent, rope, block_size)
    if n == 0:
        raise PkvError("latent_workspace_bytes: invalid shape or no device")
    return n


def paged_latent_attn(q, cache, latent, block_tables, context_lens, scale, q_start=None, tree_mask=None, out=None,
                      out_dtype=torch.bfloat16, workspace=None, err=None, stream=None):
    """Attention over the latent cache [num_blocks][block_size][latent + rope] with absorbed queries
    q [n_tok][n_h][latent + rope]; returns [n_tok][n_h][latent], the weighted sums of the latent parts.  One token
    per sequence, or several as for paged_tree_attn."""
    latent = int(latent)
    if out is None:
        out = _empty((*q.shape[:2], latent), _out_type(out_dtype), q.device, stream)
    if workspace is None and q.is_cuda and q.shape[0]:
        T, n_h, w = _dims("q", q, 3)
        bs = _dims("cache", cache, 3)[1]
        workspace = _scratch(lib().pkv_latent_workspace_bytes(block_tables.shape[0], T, n_h, latent, w - latent, bs), q.device, stream)
    st = (_calls or _native()).paged_latent_attn(q, cache, latent, block_tables, context_lens, scale, q_start, tree_mask, out,
                                                 workspace, err, None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        w = _dims("cache", cache, 3)[2]
        _on_current(q, cache)
        _typed(_bf16, cache)
        _dense(cache)
        _step_refuse(q, block_tables, context_lens, q_start, tree_mask, out, workspace, err, w, latent)
    if st:
        _failed("paged_latent_attn", st)
    return out


def _last_dense(t):
    if t.numel() and t.stride(-1) != 1:
        raise PkvError("the last dimension must be contiguous")


def latent_append(kv, q, positions, slot_mapping, table: RopeTable, cache, q_out=None, weight=None, eps=1e-6, err=None,
                  stream=None):
    """Append a step's vectors kv [n_tok][latent + rope] to the latent cache: the latent part normalised by its root
    mean square and scaled by weight (bf16 [latent]; None: as it is), the key part rotated by positions.  Rotates the
    position part of the queries, q [n_tok][n_h][rope], too, into q_out (a part of the absorbed queries, say; q
    itself is allowed), and returns it.  Tokens and heads may be strided.  table: of rope_table with rotary_dim = rope."""
    _table_type(table)
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    st = (_calls or _native()).latent_append(kv, q, positions, slot_mapping, table, cache, q_out, weight, eps, err,
                                             None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        n, n_h, rope = _dims("q", q, 3)
        w = _dims("cache", cache, 3)[2]
        _on_current(kv, q, positions, slot_mapping, cache, q_out, weight, err)
        _typed(_bf16, kv, q, cache, q_out, weight)
        _typed(_i32, positions, err)
        _typed(_i64, slot_mapping)
        _shaped("kv", kv, n, w)
        _shaped("positions", positions, n)
        _shaped("slot_mapping", slot_mapping, n)
        _shaped("q_out", q_out, n, n_h, rope)
        _shaped("weight", weight, w - rope)
        _dense(positions, slot_mapping, cache, weight)
        for t in (kv, q, q_out):
            _last_dense(t)
    if st:
        _failed("latent_append", st)
    return q_out


def kv_tree_accept(caches, block_tables, context_lens, q_start, path, n_accept, n_tok=None, new_lens=None, err=None,
                   stream=None):
    """Keep the accepted path of each sequence's drafted tokens, in every cache of the list (the K and V pools of all
    layers, or their latent caches; one shape): row base + path[s][i] becomes row base + i for i < n_accept[s], base
    being the rows in front of the drafted ones.  path (int32 [B][P]) ascends.  q_start as for the attention (None:
    n_tok / B tokens each); n_tok, which may be left out beside it, is what its entries must not exceed.  Returns the new
    context lengths, base + n_accept (a tensor of its own)."""
    caches = list(caches)
    if new_lens is None:
        new_lens = _empty(context_lens.shape, _i32, context_lens.device, stream)
    if q_start is None and n_tok is None:
        raise PkvError("without q_start the number of tokens must be given")
    n = 0x7fffffff if n_tok is None else int(n_tok)              # with q_start: what its entries are checked against
    st = (_calls or _native()).kv_tree_accept(caches, block_tables, context_lens, q_start, path, n_accept, new_lens, n, err,
                                              None if stream is None else stream.cuda_stream)
    if st == _NOT_TAKEN:
        B, _ = _dims("block_tables", block_tables, 2)
        P = _dims("path", path, 2)[1]
        if not caches or caches[0].dim() not in (3, 4):
            raise PkvError("caches must be tensors [num_blocks][heads][block_size][d] or [num_blocks][block_size][width]")
        _on_current(block_tables, context_lens, q_start, path, n_accept, new_lens, err, *caches)
        _typed(_bf16, *caches)
        _typed(_i32, block_tables, context_lens, q_start, path, n_accept, new_lens, err)
        for c in caches:
            _shaped("each cache", c, *caches[0].shape)
        _shaped("context_lens", context_lens, B)
        _shaped("n_accept", n_accept, B)
        _shaped("new_lens", new_lens, B)
        _shaped("q_start", q_start, B + 1)
        _shaped("path", path, B, P)
        _dense(block_tables, context_lens, q_start, path, n_accept, new_lens, *caches)
    if st:
        _failed("kv_tree_accept", st)
    return new_lens


# ---------------------------------------------------------------------------------------------
# Block manager (host, include/pkv_bm.h) and the GPU copies it records.
COPY_OFFLOAD, COPY_ONLOAD = 0, 1
BM_COUNTS = ("free", "active", "cached", "host", "reused_tokens", "evictions", "offloads", "onloads", "drops")


class _TokenRange(ctypes.Structure):
    _fields_ = [("start", ctypes.c_int32), ("end", ctypes.c_int32), ("priority", ctypes.c_int32)]


class BlockManager:
    """Physical block ids for a paged cache: cross-request reuse, priority-LRU eviction
    with retention ranges, host offload.  Host bookkeeping only; see include/pkv_bm.h."""

    def __init__(self, num_blocks, block_size, host_blocks=0, offload_min_priority=35, default_priority=35):
        import numpy as np
        self._np = np
        self.num_blocks, self.block_size, self.host_blocks = num_blocks, block_size, host_blocks
        self._h = lib().pkv_bm_create(num_blocks, block_size, host_blocks, offload_min_priority, default_priority)
        if not self._h:
            raise PkvError("pkv_bm_create: invalid argument")

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.pkv_bm_destroy(h)

    def _a(self, x, dtype):
        return self._np.ascontiguousarray(x, dtype=dtype)

    def add_sequence(self, seq_id, tokens, ranges=()):
        """Returns (block table as a list, number of reused prompt tokens)."""
        np = self._np
        toks = self._a(tokens, np.int32)
        rr = (_TokenRange * max(1, len(ranges)))(*[_TokenRange(int(a), int(b), int(c)) for a, b, c in ranges])
        cap = -(-len(toks) // self.block_size)
        table = np.empty(max(cap, 1), dtype=np.int32)
        r = lib().pkv_bm_add_sequence(self._h, int(seq_id), toks.ctypes.data, len(toks), rr, len(ranges),
                                      table.ctypes.data, cap)
        if r < 0:
            _check("bm_add_sequence", r)
        return table[:cap].tolist(), r

    def append_tokens(self, seq_ids, tokens):
        """One decode step: the cache slot of each sequence's new token (int64 array)."""
        np = self._np
        ids, toks = self._a(seq_ids, np.int64), self._a(tokens, np.int32)
        slots = np.empty(len(ids), dtype=np.int64)
        done = ctypes.c_int(0)
        r = lib().pkv_bm_append_tokens(self._h, ids.ctypes.data, toks.ctypes.data, len(ids), slots.ctypes.data,
                                       ctypes.byref(done))
        if r < 0:
            msg = lib().pkv_status_str(r).decode()
            raise PkvError(f"bm_append_tokens: {msg} after {done.value} of {len(ids)} sequences")
        return slots

    def append_drafts(self, seq_ids, counts):
        """Rows for counts[i] drafted tokens behind each sequence: their cache slots (int64, one sequence after another).
        No draft is reused by another request; until accept_drafts, tables() counts them in the context lengths and
        the sequences take no other call but release.  All sequences get their rows, or none."""
        np = self._np
        ids, counts = [int(s) for s in seq_ids], [int(n) for n in counts]
        if len(ids) != len(counts) or any(not 0 <= n <= 0x7fffffff for n in counts):
            raise PkvError("append_drafts: a number of drafts for each sequence")
        if any(n > self.num_blocks * self.block_size for n in counts):
            raise PkvError("append_drafts: more drafts than rows")
        slots, at = np.empty(sum(counts), dtype=np.int64), 0
        for i, (s, n) in enumerate(zip(ids, counts)):
            r = lib().pkv_bm_append_drafts(self._h, s, n, slots[at:].ctypes.data)
            if r < 0:
                for back in ids[:i]:
                    lib().pkv_bm_accept_drafts(self._h, back, None, 0)
                _check(f"bm_append_drafts of sequence {s}", r)
            at += n
        return slots

    def accept_drafts(self, seq_ids, tokens):
        """tokens[i], the accepted path's in its order, become the next ones of sequence i; the other drafts' rows are given
        back.  After kv_tree_accept has been launched with the tables and lengths from before, ahead of the manager's next call.
        Stops at the first sequence that refuses (more tokens than drafts, or unknown)."""
        np = self._np
        ids, tokens = [int(s) for s in seq_ids], [self._a(t, np.int32) for t in tokens]
        if len(ids) != len(tokens) or len(set(ids)) != len(ids):
            raise PkvError("accept_drafts: distinct sequences with a list of tokens each")
        for s, t in zip(ids, tokens):
            r = lib().pkv_bm_accept_drafts(self._h, s, t.ctypes.data, len(t))
            if r < 0:
                _check(f"bm_accept_drafts of sequence {s}", r)

    def release(self, seq_id):
        _check("bm_release", lib().pkv_bm_release(self._h, int(seq_id)))

    def slide_window(self, seq_id, window):
        r = lib().pkv_bm_slide_window(self._h, int(seq_id), int(window))
        if r < 0:
            _check("bm_slide_window", r)
        return r

    def evict(self, seq_id, keep):
        """Cut a sequence to its first `keep` cache rows; returns the blocks left.  Called before kv_evict, with
        the table from before it: where this refuses (a block that stays is shared), the rows must not move."""
        r = lib().pkv_bm_evict(self._h, int(seq_id), int(keep))
        if r < 0:
            _check("bm_evict", r)
        return r

    def cut_to(self, seq_ids, lens, budget):
        """Cut sequences of context lengths `lens` (from tables()) to at most `budget` rows; returns `keep` for
        kv_evict, which follows before the manager's next call, with the tables and lengths from before this one.
        Sequences no longer than the budget, or whose blocks may not be rewritten (one that stays is shared with
        another sequence, or some were released by slide_window), keep all their rows."""
        ids, lens, budget = [int(s) for s in seq_ids], [int(n) for n in lens], int(budget)
        if budget < 1 or len(lens) != len(ids) or len(set(ids)) != len(ids):
            raise PkvError("cut_to: a budget of at least one row, and distinct sequences with a length each")
        keep = list(lens)
        for i, s in enumerate(ids):
            if lens[i] <= budget:
                continue
            r = lib().pkv_bm_evict(self._h, s, budget)
            if r >= 0:
                keep[i] = budget
            elif r != -1:                                      # anything but a refusal
                _check("bm_evict", r)
        return keep

    def tables(self, seq_ids, max_blocks):
        """(block tables int32 [n][max_blocks], context lengths int32 [n]) for an attention call."""
        np = self._np
        ids = self._a(seq_ids, np.int64)
        t = np.empty((len(ids), max_blocks), dtype=np.int32)
        c = np.empty(len(ids), dtype=np.int32)
        _check("bm_tables", lib().pkv_bm_tables(self._h, ids.ctypes.data, len(ids), t.ctypes.data, max_blocks,
                                                c.ctypes.data))
        return t, c

    def take_copies(self):
        """Copies recorded since the last call: int32 [n][3] rows (kind, src, dst)."""
        np = self._np
        n = lib().pkv_bm_pending_copies(self._h)
        out = np.empty((max(n, 1), 3), dtype=np.int32)
        r = lib().pkv_bm_take_copies(self._h, out.ctypes.data, n)
        if r < 0:
            _check("bm_take_copies", r)
        return out[:r]

    def counts(self):
        out = (ctypes.c_int64 * len(BM_COUNTS))()
        lib().pkv_bm_counts(self._h, out)
        return dict(zip(BM_COUNTS, list(out)))


def copy_blocks(copies, k_pool, v_pool, k_host, v_host, stream=None):
    """Apply recorded copies (int32 [n][3] rows kind, src, dst) between the device pools and
    host pools in page-locked memory ([host_blocks][...] tensors of the same block shape)."""
    import numpy as np
    _cuda(k_pool, v_pool)
    for t in (k_host, v_host):
        if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
            raise PkvError("host pools must be contiguous page-locked CPU tensors")
    assert k_pool.shape[1:] == k_host.shape[1:] and k_pool.dtype == k_host.dtype
    c = np.ascontiguousarray(copies, dtype=np.int32).reshape(-1, 3)
    block_bytes = k_pool[0].numel() * k_pool.element_size()
    _check("copy_blocks", lib().pkv_copy_blocks(c.ctypes.data, len(c), _ptr(k_pool), _ptr(v_pool), k_pool.shape[0],
                                                _ptr(k_host), _ptr(v_host), k_host.shape[0], block_bytes,
                                                _stream(stream)))


# ---------------------------------------------------------------------------------------------
# CacheBlend's model-free steps (pkv.h): KV deviation, top-ratio selection, fuse.
def kv_deviation(k_pool, v_pool, slots, k_new, v_new, out=None, err=None, stream=None):
    """Per-token L2 distance between the cached K/V at slots and the recomputed rows (fp32 [n])."""
    _cuda(k_pool, v_pool, slots, k_new, v_new, out, err)
    assert k_pool.dtype == v_pool.dtype == k_new.dtype == v_new.dtype == torch.bfloat16
    assert slots.dtype == torch.int64
    num_blocks, n_kv, bs, d = k_pool.shape
    n = slots.numel()
    assert k_new.shape == v_new.shape == (n, n_kv, d)
    dev = _empty((n,), torch.float32, k_pool.device, stream) if out is None else out
    assert dev.dtype == torch.float32 and dev.numel() == n
    _check("kv_deviation", lib().pkv_kv_deviation(_ptr(k_pool), _ptr(v_pool), _ptr(slots), _ptr(k_new), _ptr(v_new),
                                                  n, num_blocks, bs, n_kv, d, _ptr(dev), _ptr(err), _stream(stream)))
    return dev


def select_top(dev, seg_offsets, counts, out=None, stream=None):
    """Per segment, the counts[s] largest deviations as ascending global indices (int32).
    seg_offsets / counts: host sequences (they size the output), or device int32 tensors
    together with a device `out` of the right size (no host work, e.g. inside a graph)."""
    import numpy as np
    _cuda(dev, out)
    assert dev.dtype == torch.float32
    if out is None:
        offs = np.ascontiguousarray(seg_offsets, dtype=np.int32)
        cnt = np.ascontiguousarray(counts, dtype=np.int32)
        assert len(offs) == len(cnt) + 1
        total = int(np.minimum(np.maximum(cnt, 0), np.maximum(np.diff(offs), 0)).sum())
        out = _empty((max(total, 1),), torch.int32, dev.device, stream)[:total]
        with torch.cuda.stream(stream):                        # None: the current stream
            seg_offsets = torch.as_tensor(offs, device=dev.device)
            counts = torch.as_tensor(cnt, device=dev.device)
    _cuda(seg_offsets, counts)
    assert seg_offsets.dtype == counts.dtype == out.dtype == torch.int32
    _check("select_top", lib().pkv_select_top(_ptr(dev), _ptr(seg_offsets), _ptr(counts), counts.numel(), _ptr(out),
                                              _stream(stream)))
    return out


def kv_fuse(k_new, v_new, row_slots, rows, k_pool, v_pool, err=None, stream=None):
    """pools[row_slots[rows[j]]] = k_new / v_new[rows[j]]: the recomputed rows of the selected tokens."""
    _cuda(k_new, v_new, rows, row_slots, k_pool, v_pool, err)
    assert rows.dtype == torch.int32 and row_slots.dtype == torch.int64 and row_slots.numel() == k_new.shape[0]
    num_blocks, n_kv, bs, d = k_pool.shape
    _check("kv_fuse", lib().pkv_kv_fuse(_ptr(k_new), _ptr(v_new), _ptr(row_slots), k_new.shape[0], _ptr(rows),
                                        rows.numel(), _ptr(k_pool), _ptr(v_pool), num_blocks, bs, n_kv, d, _ptr(err),
                                        _stream(stream)))


def recompute_ratio(load_time, full_recompute_time):
    return lib().pkv_recompute_ratio(float(load_time), float(full_recompute_time))


def select_count(ratio, n):
    return lib().pkv_select_count(float(ratio), int(n))


def selftest_wait(arrive, limit_us, err, stream=None):
    """Run the bounded-wait self-test; err (device int32) gets DEV_TIMEOUT if the wait ran out."""
    _cuda(err)
    _check("selftest_wait", lib().pkv_selftest_wait(1 if arrive else 0, int(limit_us), _ptr(err), _stream(stream)))


# ---------------------------------------------------------------------------------------------
# HBM ceiling probes (pkv.h): the read-only stream and the copy the roofline is measured against.
def probe_read(buf, sink=None, stream=None):
    """Stream every byte of the CUDA tensor `buf` once (16-byte loads)."""
    _cuda(buf, sink)
    _check("probe_read", lib().pkv_probe_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                              _stream(stream)))


def probe_copy(src, dst, stream=None):
    """Copy the CUDA tensor `src` into `dst` (same byte size; 16-byte loads and stores)."""
    _cuda(src, dst)
    n = src.numel() * src.element_size()
    assert dst.numel() * dst.element_size() == n
    _check("probe_copy", lib().pkv_probe_copy(_ptr(src), _ptr(dst), n, _stream(stream)))
