"""The error word of the device tables' steps, bit for bit, through random steps
on which the pool runs out, rows outgrow their tables, sources lie outside the
rows and the slots are too few."""
import random

import pytest
import torch

import tables_model as model

pytestmark = pytest.mark.gpu


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _expected(lib, tables, lens, refs, append, bs, max_new, release, fork):
    """The model's step, and the bits its calls for."""
    n, cap = len(tables), len(tables[0]) * bs
    was = list(lens)
    slots, starts, pairs, _ = model.step(tables, lens, refs, append, bs, max_new, release, fork)
    code = 0
    for i, add in enumerate(append):
        now = was[i]
        if fork is not None and 0 <= fork[i] < n:
            now = was[fork[i]]
        elif release is not None and release[i]:
            now = 0
        if add < 0 or now + add > cap:
            code |= lib.PA_DEVERR_CONTEXT_LEN
        elif add > 0 and lens[i] != now + add:
            code |= lib.PA_DEVERR_POOL
        if fork is not None and fork[i] >= n:
            code |= lib.PA_DEVERR_TABLE
    if sum(max(a, 0) for a in append) > max_new:
        code |= lib.PA_DEVERR_SLOT
    return slots, starts, pairs, code


@pytest.mark.parametrize("rows,width,nb,bs,fill,seed,reached", [
    (5, 8, 14, 4, 9, 2, "pool table context slot"), (33, 20, 250, 16, 90, 3, "pool table context slot"),
    (300, 30, 1900, 16, 100, 4, "pool table context slot"), (1000, 6, 2100, 32, 60, 5, "pool table context slot"),
    (64, 40, 1025, 16, 300, 7, "pool table context slot"), (40, 50, 4000, 16, 20, 9, "none")])
def test_the_error_word_of_every_step(rows, width, nb, bs, fill, seed, reached):
    from paged_kv_cache_388_b200 import _lib
    from paged_kv_cache_388_b200.tables import DeviceBlockTables
    r = random.Random(seed)
    tables, lens, refs = [[0] * width for _ in range(rows)], [0] * rows, [0] * nb
    dev = DeviceBlockTables(rows, width, nb, bs)
    seen = set()
    odd = "none" not in reached
    for k in range(24):
        fork = [r.randrange(rows) if r.random() < 0.05 else -1 for _ in range(rows)] if k % 2 else None
        release = [int(r.random() < 0.1) for _ in range(rows)] if k % 3 else None
        append = [r.choice([0, 1, 1, r.randint(0, fill)]) for _ in range(rows)]
        if odd and fork and k % 4 == 1:
            fork[r.randrange(rows)] = rows + r.randrange(3)
        if odd and k % 5 == 4:
            append[r.randrange(rows)] = -1
        if odd and k % 7 == 6:
            append[r.randrange(rows)] = width * bs + 1
        new = sum(max(a, 0) for a in append)
        max_new = max(0, new + (r.choice([-1, 0, 5]) if odd else 3))
        slots, qsl, pairs = dev.step(_i32(append), max_new, release=_i32(release), fork_src=_i32(fork))
        want_slots, starts, want_pairs, want = _expected(_lib, tables, lens, refs, append, bs, max_new, release, fork)
        code = _lib.pa_get_device_error()
        assert code == want, (k, hex(code), hex(want))
        seen.add(code)
        assert dev.context_lens.tolist() == lens and dev.ref_counts.tolist() == refs
        for t, w, n in zip(dev.block_tables.tolist(), tables, lens):
            assert t[: -(-n // bs)] == w[: -(-n // bs)]
        assert slots.tolist() == want_slots and qsl.tolist() == starts
        assert [tuple(p) for p in pairs.tolist()] == want_pairs
    bits = {"pool": _lib.PA_DEVERR_POOL, "table": _lib.PA_DEVERR_TABLE, "context": _lib.PA_DEVERR_CONTEXT_LEN,
            "slot": _lib.PA_DEVERR_SLOT, "none": 0}
    for name in reached.split():
        assert any(c & bits[name] for c in seen) if bits[name] else seen == {0}, name
    assert 0 in seen


def test_no_error_from_two_tables_on_two_streams():
    from paged_kv_cache_388_b200 import _lib
    from paged_kv_cache_388_b200.tables import DeviceBlockTables
    assert _lib.pa_get_device_error() == 0
    r = random.Random(1)
    both = []
    for rows, width, nb in ((300, 20, 9000), (40, 30, 70000)):
        both.append(([[0] * width for _ in range(rows)], [0] * rows, [0] * nb, DeviceBlockTables(rows, width, nb, 16),
                     torch.cuda.Stream()))
    for _ in range(4):
        todo = [[r.randint(0, 20) for _ in t[1]] for t in both]
        dev = [_i32(a) for a in todo]
        torch.cuda.synchronize()
        for a, d, (_, _, _, tab, st) in zip(todo, dev, both):
            with torch.cuda.stream(st):
                tab.step(d, sum(a))
                tab.compact()
        torch.cuda.synchronize()
        assert _lib.pa_get_device_error() == 0
        for a, (tables, lens, refs, tab, _) in zip(todo, both):
            model.step(tables, lens, refs, a, 16, 0)
            model.compact(tables, lens, refs, 16)
            assert tab.context_lens.tolist() == lens and tab.ref_counts.tolist() == refs
