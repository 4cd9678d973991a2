"""The device tables hold no memory of their own beside the arrays that a caller
sees: a workspace belongs to one call and to its stream."""
import random
import weakref

import pytest
import torch

import tables_model as model
from paged_kv_cache_388_b200 import _lib
from paged_kv_cache_388_b200.tables import DeviceBlockTables


def test_a_workspace_lives_as_long_as_its_call(monkeypatch):
    seen = []

    def take(*args):
        ws = next(a for a in reversed(args) if torch.is_tensor(a) and a.dtype == torch.uint8)
        assert ws.numel() >= _lib.pa_table_workspace_size(3, 4, 20)
        seen.append(weakref.ref(ws))

    monkeypatch.setattr(_lib, "_table_shapes", lambda t, n, r: (*t.shape, r.shape[0], 0))
    monkeypatch.setattr(_lib, "_table_step", take)
    monkeypatch.setattr(_lib, "_table_compact", take)
    tab = DeviceBlockTables(3, 4, 20, 16, device="cpu")
    tab.step(torch.zeros(3, dtype=torch.int32), 2)
    tab.compact()
    assert len(seen) == 2 and all(ws() is None for ws in seen)
    mine = {tab.block_tables.data_ptr(), tab.context_lens.data_ptr(), tab.ref_counts.data_ptr()}
    assert {x.data_ptr() for x in vars(tab).values() if torch.is_tensor(x)} == mine


@pytest.mark.gpu
def test_tables_dropped_while_their_step_still_runs():
    """Stepped on a stream of their own behind other work; then the object goes, and its memory's like is written on
    another stream.  (The arrays are the caller's, who keeps them until the end.)"""
    rows, width, nb, bs = 200, 20, 3000, 16
    r = random.Random(0)
    append = [r.randint(0, 40) for _ in range(rows)]
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    arrays = i32(rows, width), i32(rows), i32(nb)
    dev = DeviceBlockTables(rows, width, nb, bs, block_tables=arrays[0], context_lens=arrays[1], ref_counts=arrays[2])
    need = _lib.pa_table_workspace_size(rows, width, nb)
    add = torch.tensor(append, dtype=torch.int32, device="cuda")
    side, work = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            work = work @ work
        slots, qsl, _ = dev.step(add, sum(append))
        dev.compact()
    del dev
    junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    tables, lens, refs = [[0] * width for _ in range(rows)], [0] * rows, [0] * nb
    want, starts, _, _ = model.step(tables, lens, refs, append, bs, sum(append))
    model.compact(tables, lens, refs, bs)
    assert slots.tolist() == want and qsl.tolist() == starts
    assert [a.tolist() for a in arrays] == [tables, lens, refs] and _lib.pa_get_device_error() == 0 and len(junk) == 8


@pytest.mark.gpu
def test_more_rows_than_a_step_takes_can_be_compacted():
    rows = 5000
    tables = torch.arange(rows, dtype=torch.int32).flip(0)[:, None].contiguous() * 2
    dev = DeviceBlockTables(rows, 1, 2 * rows, 16, block_tables=tables.cuda(),
                            context_lens=torch.ones(rows, dtype=torch.int32).cuda(),
                            ref_counts=torch.tensor([1, 0], dtype=torch.int32).repeat(rows).cuda())
    with pytest.raises(_lib.PAError, match="UNSUPPORTED"):
        dev.step(torch.ones(rows, dtype=torch.int32).cuda(), rows)
    live, _ = dev.compact()
    assert live.tolist() == [rows] and sorted(dev.block_tables.flatten().tolist()) == list(range(rows))
    assert _lib.pa_get_device_error() == 0
