"""Block tables, lengths and reference counts held on the device.

``DeviceBlockTables`` is the host allocator's bookkeeping (``BlockAllocator``)
in device arrays, for loops that must not wait for the host, a captured decode
loop among them: ``step`` releases, forks and grows all rows in one call and
hands out the new tokens' slots, copying the blocks that a shared row writes
into; ``compact`` moves the used blocks to the front of the pool, so that the
pool's tail can be given back.  Calls on the same tables, captured ones among
them, must follow one another (one stream, or streams that wait), since they
update the tables.  Their workspaces are taken from torch's allocator call by
call, on the stream of the call.

``step`` takes tables of up to 4096 rows, ``compact`` any number.
"""
from __future__ import annotations

import torch

from . import _lib


class DeviceBlockTables:
    def __init__(self, num_seqs, max_blocks_per_seq, num_blocks, block_size, device="cuda",
                 block_tables=None, context_lens=None, ref_counts=None):
        """Empty tables of ``num_seqs`` rows over a pool of ``num_blocks``, or
        the given int32 arrays, which are then updated in place."""
        def own(t, shape, name):
            if t is None:
                return torch.zeros(shape, dtype=torch.int32, device=device)
            if tuple(t.shape) != shape or t.dtype != torch.int32:
                raise ValueError(f"{name} must be int32 {shape}, got {t.dtype} {tuple(t.shape)}")
            return t

        if block_size <= 0 or num_seqs <= 0 or max_blocks_per_seq <= 0 or num_blocks <= 0:
            raise ValueError("sizes must be positive")
        self.num_seqs, self.max_blocks_per_seq = num_seqs, max_blocks_per_seq
        self.num_blocks, self.block_size = num_blocks, block_size
        self.block_tables = own(block_tables, (num_seqs, max_blocks_per_seq), "block_tables")
        self.context_lens = own(context_lens, (num_seqs,), "context_lens")
        self.ref_counts = own(ref_counts, (num_blocks,), "ref_counts")
        self.device = self.block_tables.device
        self._ws_bytes = _lib.pa_table_workspace_size(num_seqs, max_blocks_per_seq, num_blocks)

    @classmethod
    def from_allocator(cls, allocator, sids, max_blocks_per_seq, device="cuda"):
        """The host allocator's sequences ``sids`` as rows 0, 1, ...; sequences
        left out keep no claim on their blocks here."""
        tables = torch.from_numpy(allocator.block_tables_array(sids, max_blocks_per_seq))
        refs = torch.zeros(allocator.num_blocks, dtype=torch.int32)
        for sid in sids:
            refs[torch.tensor(allocator.block_table(sid), dtype=torch.int64)] += 1
        lens = torch.from_numpy(allocator.context_lens_array(sids))
        return cls(len(sids), max_blocks_per_seq, allocator.num_blocks, allocator.block_size,
                   block_tables=tables.to(device), context_lens=lens.to(device),
                   ref_counts=refs.to(device))

    def step(self, append, max_new_tokens, release=None, fork_src=None, pools=()):
        """One scheduling step: rows with release != 0 give up their blocks,
        rows with fork_src >= 0 come to hold that row's, then every row grows by
        append tokens (all int32 [num_seqs]).  Returns slot_mapping int64
        [max_new_tokens] (-1 past the last token and for rows that did not
        grow), query_start_loc int32 [num_seqs + 1] and the copy-on-write pairs
        int64 [num_seqs, 2]; the copies are done in all ``pools`` ([num_blocks,
        ...] tensors).  When the pool runs out the row and all later growing
        ones stay as they are (PA_DEVERR_POOL in the device error word)."""
        t = self.block_tables
        sizes = _lib._table_shapes(t, self.context_lens, self.ref_counts)
        n = sizes[0]
        slots = t.new_empty(max_new_tokens, dtype=torch.int64)
        qsl = t.new_empty(n + 1)
        pairs = t.new_empty((n, 2), dtype=torch.int64)
        _lib._table_step(sizes, t, self.context_lens, self.ref_counts, append, self.block_size,
                         slots, qsl, pairs, release, fork_src, pools, t.new_empty(self._ws_bytes, dtype=torch.uint8),
                         None)
        return slots, qsl, pairs

    def compact(self, pools=()):
        """Move the used blocks to ids [0, live) in the tables and in all
        ``pools``.  Returns live (int32 [1]) and the moves (src, dst), int64
        [max(1, num_blocks // 2), 2] filled up with (-1, -1)."""
        t = self.block_tables
        sizes = _lib._table_shapes(t, self.context_lens, self.ref_counts)
        live = t.new_empty(1)
        moves = t.new_empty((max(1, sizes[2] // 2), 2), dtype=torch.int64)
        _lib._table_compact(sizes, t, self.context_lens, self.ref_counts, self.block_size, live,
                            moves, pools, t.new_empty(self._ws_bytes, dtype=torch.uint8), None)
        return live, moves
