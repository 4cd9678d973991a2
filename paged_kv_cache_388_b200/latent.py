"""User-facing wrapper of the latent cache: one layer's paged cache that holds
one vector a token, shared by every head.

A token's row is ``latent_dim`` values, from which the keys and values of all
heads are linear maps, and ``rope_dim`` values that carry the position and
enter the logits only.  ``PagedLatentCache.write`` stores new rows,
``PagedLatentCache.attend`` attends in the absorbed form (queries brought into
the latent space, outputs left in it: single tokens and a few drafted ones),
``latent_prefill`` in the expanded form (keys and values of every head
multiplied out: prompts and chunks of prompts).  Block tables, slots and the
error word are those of ``PagedKVCache``.

Workspaces are taken from torch's allocator call by call, so calls on several
streams and several captured graphs never share one.
"""
from __future__ import annotations

import torch

from . import _lib


class PagedLatentCache:
    def __init__(self, num_blocks, latent_dim, rope_dim, block_size, dtype=torch.bfloat16,
                 device="cuda", latent_cache=None):
        shape = (num_blocks, block_size, latent_dim + rope_dim)
        if latent_cache is None:
            latent_cache = torch.empty(shape, dtype=dtype, device=device)
        if tuple(latent_cache.shape) != shape:
            raise ValueError(f"latent_cache must be {shape}, got {tuple(latent_cache.shape)}")
        self.latent_cache = latent_cache
        self.num_blocks, self.block_size = num_blocks, block_size
        self.latent_dim, self.rope_dim = latent_dim, rope_dim
        self.dtype, self.device = latent_cache.dtype, latent_cache.device
        self._ws_bytes = {}  # by batch sizes

    def write(self, latent, rope, slot_mapping):
        """Store rows latent [T, latent_dim] | rope [T, rope_dim] in their slots
        (negative slots are skipped)."""
        if latent.shape[-1] != self.latent_dim:
            raise ValueError(f"latent must be [num_tokens, {self.latent_dim}]")
        _lib.pa_latent_write(latent, rope, self.latent_cache, slot_mapping)

    def attend(self, q, block_tables, context_lens, scale, out=None, lse=None,
               query_start_loc=None, max_query_len=1, max_context_len=0):
        """Absorbed attention: q [Tq, H, latent_dim + rope_dim] over each
        sequence's cached rows; returns out [Tq, H, latent_dim].  ``lse``
        (float32 [Tq, H]) receives the logarithm of the softmax sums, by which
        partial results over disjoint keys are merged."""
        if out is None:
            out = q.new_empty((*q.shape[:-1], self.latent_dim))
        elif out.shape[-1] != self.latent_dim:
            raise ValueError(f"out must be [tokens, heads, {self.latent_dim}]")
        rows = 1 if query_start_loc is None else min(max_query_len, q.shape[0])
        sizes = (block_tables.shape[0], rows, q.shape[1], self.latent_dim)
        need = self._ws_bytes.get(sizes)
        if need is None:
            need = self._ws_bytes[sizes] = _lib.pa_latent_decode_workspace_size(*sizes)
        ws = q.new_empty(need, dtype=torch.uint8)
        _lib.pa_latent_decode(out, lse, q, self.latent_cache, block_tables, context_lens, scale,
                              query_start_loc=query_start_loc, max_query_len=max_query_len,
                              max_context_len=max_context_len, workspace=ws)
        return out


def latent_prefill(q, k, k_rope, v, query_start_loc, context_start_loc, scale, max_query_len,
                   out=None, lse=None, causal=True):
    """Expanded attention of a ragged batch: q [Tq, H, Dn + Dr], k [Tk, H, Dn],
    k_rope [Tk, Dr] (shared by the heads), v [Tk, H, Dv].  Row t of a sequence
    with Q rows and L keys sees keys 0 .. L-Q+t, or all L with causal=False.
    Returns out [Tq, H, Dv]; rows past the last sequence are left unwritten."""
    if out is None:
        out = q.new_empty((*q.shape[:-1], v.shape[-1]))
    need = _lib.pa_latent_prefill_workspace_size(query_start_loc.shape[0] - 1, q.shape[0], k.shape[0],
                                                 q.shape[1], v.shape[-1])
    ws = q.new_empty(need, dtype=torch.uint8) if need else None
    _lib.pa_latent_prefill(out, lse, q, k, k_rope, v, query_start_loc, context_start_loc, scale,
                           max_query_len, causal=causal, workspace=ws)
    return out
