"""Block tables on the device against the sequential restatement: every result
is a whole number and has to be equal."""
import random

import pytest
import torch

import tables_model as model
from paged_kv_cache_388_b200.allocator import BlockAllocator


def _state(r, rows, width, nb, bs, fill):
    """Tables after some random steps of the model."""
    tables, lens, refs = [[r.randrange(nb) for _ in range(width)] for _ in range(rows)], [0] * rows, [0] * nb
    for _ in range(3):
        fork = [r.randrange(rows) if r.random() < 0.2 else -1 for _ in range(rows)]
        release = [int(r.random() < 0.1) for _ in range(rows)]
        append = [r.randint(0, fill) for _ in range(rows)]
        model.step(tables, lens, refs, append, bs, 0, release, fork)
    return tables, lens, refs


def test_the_model_agrees_with_the_host_allocator():
    """Grown token by token and forked, the model's rows hold the lengths and share the blocks that the allocator's do."""
    r = random.Random(0)
    al = BlockAllocator(64, 4)
    sids = [al.new_sequence(0) for _ in range(3)]
    tables, lens, refs = [[0] * 16 for _ in range(3)], [0] * 3, [0] * 64
    for i in range(40):
        fork = [-1] * 3
        if i == 17:
            al.free(sids[2])
            sids[2], fork[2] = al.fork(sids[0]), 0
        who = r.randrange(3)
        append = [int(x == who) for x in range(3)]
        slots, _, pairs, out = model.step(tables, lens, refs, append, 4, 1, None, fork)
        slot, cow = al.append_slot(sids[who])
        assert not out and (cow is None) == (pairs[who] == (-1, -1)) and slot % 4 == slots[0] % 4
        assert lens == [al.context_len(s) for s in sids]
        assert sorted(c for c in refs if c) == sorted(al.refcount(b) for b in range(64) if al.refcount(b))
    assert any(c > 1 for c in refs)


gpu = pytest.mark.gpu


def _device(tables, lens, refs, bs):
    from paged_kv_cache_388_b200.tables import DeviceBlockTables
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return DeviceBlockTables(len(tables), len(tables[0]), len(refs), bs, block_tables=t(tables), context_lens=t(lens),
                             ref_counts=t(refs))


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _pools(nb, n, seed):
    g = torch.Generator().manual_seed(seed)
    # blocks of 16 bytes up to several KB, of different types
    shapes = [(nb, 8), (nb, 3, 200, 8), (nb, 16, 4)]
    return [torch.randint(0, 1000, shapes[i % 3], generator=g).to([torch.bfloat16, torch.uint8, torch.float32][i % 3])
            for i in range(n)]


@gpu
@pytest.mark.parametrize("rows,width,nb,bs,fill,seed", [
    (1, 1, 1, 16, 1, 0), (1, 9, 12, 16, 40, 1), (5, 8, 64, 4, 9, 2), (33, 20, 700, 16, 90, 3), (300, 30, 5000, 16, 100, 4),
    (1000, 6, 3000, 32, 60, 5), (2500, 3, 7000, 2, 2, 6), (64, 40, 1025, 16, 300, 7), (4096, 2, 9000, 16, 9, 8)])
def test_steps_equal_the_model(rows, width, nb, bs, fill, seed):
    from paged_kv_cache_388_b200 import _lib
    r = random.Random(seed)
    tables, lens, refs = _state(r, rows, width, nb, bs, fill)
    dev = _device(tables, lens, refs, bs)
    pools = _pools(nb, 4 if rows < 500 else 1, seed)
    dpools = [p.cuda() for p in pools]
    seen = set()
    for k in range(6):
        fork = [r.randrange(rows) if r.random() < 0.1 else -1 for _ in range(rows)] if k % 2 else None
        release = [int(r.random() < 0.15) for _ in range(rows)] if k % 3 else None
        if k == 4:  # every row to row 0's blocks, all write into its last one
            fork = [0] * rows
        append = [r.choice([0, 1, 1, r.randint(0, fill)]) for _ in range(rows)]
        max_new = max(0, sum(append) + r.choice([0, 5]))
        slots, qsl, pairs = dev.step(_i32(append), max_new, release=_i32(release), fork_src=_i32(fork), pools=dpools)
        before = list(lens)
        want_slots, starts, want_pairs, out = model.step(tables, lens, refs, append, bs, max_new, release, fork)
        code = _lib.pa_get_device_error()
        assert bool(code & _lib.PA_DEVERR_POOL) == (out and any(a > 0 for a in append)) or not out
        seen |= {out}
        assert dev.context_lens.tolist() == lens and dev.ref_counts.tolist() == refs, (k, before)
        assert dev.block_tables.tolist() == tables
        assert slots.tolist() == want_slots and qsl.tolist() == starts
        assert [tuple(p) for p in pairs.tolist()] == want_pairs
        for p, d in zip(pools, dpools):
            for s, t in want_pairs:
                if s >= 0:
                    p[t] = p[s]
            assert torch.equal(d.cpu(), p)


@gpu
@pytest.mark.parametrize("rows,width,nb,bs,fill,seed", [
    (1, 1, 1, 16, 1, 0), (1, 9, 12, 16, 40, 1), (7, 8, 64, 4, 9, 2), (50, 20, 1025, 16, 90, 3), (300, 30, 9000, 16, 100, 4),
    (20, 300, 6000, 32, 4000, 5)])
def test_compaction_equals_the_model(rows, width, nb, bs, fill, seed):
    from paged_kv_cache_388_b200 import _lib
    r = random.Random(seed)
    tables, lens, refs = _state(r, rows, width, nb, bs, fill)
    model.step(tables, lens, refs, [0] * rows, bs, 0, [int(r.random() < 0.4) for _ in range(rows)])
    dev = _device(tables, lens, refs, bs)
    pools = _pools(nb, 3, seed)
    dpools = [p.cuda() for p in pools]
    live, moves = dev.compact(pools=dpools)
    want_live, want_moves = model.compact(tables, lens, refs, bs)
    assert _lib.pa_get_device_error() == 0
    assert live.tolist() == [want_live] and dev.ref_counts.tolist() == refs and dev.block_tables.tolist() == tables
    want_moves = (want_moves + [(-1, -1)] * nb)[: max(1, nb // 2)]
    assert [tuple(p) for p in moves.tolist()] == want_moves
    for p, d in zip(pools, dpools):
        for s, t in want_moves:
            if s >= 0:
                p[t] = p[s]
        assert torch.equal(d.cpu(), p)
    # once more: nothing is left to move
    live, moves = dev.compact(pools=dpools)
    assert live.tolist() == [want_live] and torch.all(moves == -1) and dev.block_tables.tolist() == tables


@gpu
def test_compaction_of_an_empty_and_of_a_full_pool():
    dev = _device([[0, 0]], [0], [0] * 2000, 16)
    live, moves = dev.compact()
    assert live.tolist() == [0] and torch.all(moves == -1)
    dev = _device([list(range(1024))], [1024 * 16], [1] * 1024, 16)
    live, moves = dev.compact(pools=[torch.zeros(1024, 16, device="cuda")])
    assert live.tolist() == [1024] and torch.all(moves == -1) and dev.block_tables.tolist() == [list(range(1024))]


@gpu
def test_bad_items_are_skipped_and_reported():
    from paged_kv_cache_388_b200 import _lib
    tables = [[0, 1], [2, 999], [3, 4]]
    dev = _device(tables, [20, 20, 20], [1] * 5 + [0] * 27, 16)
    # negative growth, growth past the table, and a fork from a row that is not there
    slots, qsl, pairs = dev.step(_i32([-1, 13, 0]), 16, fork_src=_i32([-1, -1, 3]))
    assert _lib.pa_get_device_error() == _lib.PA_DEVERR_CONTEXT_LEN | _lib.PA_DEVERR_TABLE
    assert dev.context_lens.tolist() == [20] * 3 and torch.all(slots == -1) and qsl.tolist() == [0, 0, 13, 13]
    # a block id outside the pool in a row that is given up
    dev.step(_i32([0, 0, 0]), 0, release=_i32([0, 1, 0]))
    assert _lib.pa_get_device_error() == _lib.PA_DEVERR_BLOCK_ID
    assert dev.ref_counts.tolist() == [1, 1, 0, 1, 1] + [0] * 27 and dev.context_lens.tolist() == [20, 0, 20]
    # more tokens than announced
    slots, qsl, _ = dev.step(_i32([2, 3, 2]), 4)
    assert _lib.pa_get_device_error() == _lib.PA_DEVERR_SLOT
    assert qsl.tolist() == [0, 2, 5, 7] and slots.tolist() == [20, 21, 32, 33]
    # a length that the table cannot hold counts as none
    dev.context_lens[0] = 33
    dev.step(_i32([0, 0, 0]), 0)
    assert _lib.pa_get_device_error() == _lib.PA_DEVERR_CONTEXT_LEN
    assert dev.context_lens.tolist() == [0, 3, 22]
    # held ids outside the pool stay where they are
    dev.block_tables[2, 0] = -7
    dev.compact()
    assert _lib.pa_get_device_error() == _lib.PA_DEVERR_BLOCK_ID and dev.block_tables[2, 0] == -7


@gpu
def test_rows_permuted_by_forks():
    tables = [[5], [6], [7]]
    dev = _device(tables, [16, 3, 9], [0] * 5 + [1] * 3, 16)
    dev.step(_i32([0, 0, 0]), 0, release=_i32([1, 1, 1]), fork_src=_i32([2, 0, 1]))
    assert dev.block_tables.tolist() == [[7], [5], [6]] and dev.context_lens.tolist() == [9, 16, 3]
    assert dev.ref_counts.tolist() == [0] * 5 + [1] * 3


@gpu
def test_a_captured_step_runs_on_by_itself():
    """A captured step replayed: rows grow block by block without the host, on a stream of its own."""
    from paged_kv_cache_388_b200 import _lib
    tables, lens, refs = [[0] * 8 for _ in range(3)], [0] * 3, [0] * 40
    dev = _device(tables, lens, refs, 4)
    pool = torch.arange(40 * 8, dtype=torch.float32).view(40, 8).cuda()
    append = _i32([1, 2, 1])
    fork = _i32([-1, -1, -1])
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        dev.step(append, 4, fork_src=fork, pools=[pool])
    st.synchronize()
    model.step(tables, lens, refs, [1, 2, 1], 4, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slots, qsl, pairs = dev.step(append, 4, fork_src=fork, pools=[pool])
    for k in range(10):
        f = [-1, -1, 0] if k == 5 else [-1] * 3
        fork.copy_(_i32(f))
        g.replay()
        want = model.step(tables, lens, refs, [1, 2, 1], 4, 4, None, f)
        assert slots.tolist() == want[0] and [tuple(p) for p in pairs.tolist()] == want[2]
        assert dev.block_tables.tolist() == tables and dev.ref_counts.tolist() == refs
    assert _lib.pa_get_device_error() == 0


@gpu
def test_seventy_pools_follow():
    """More pools than a launch takes: K and V of 35 layers."""
    from paged_kv_cache_388_b200 import _lib
    tables, lens, refs = [[5, 0], [5, 0], [9, 8]], [10, 10, 20], [0] * 40
    for b, c in ((5, 2), (9, 1), (8, 1)):
        refs[b] = c
    dev = _device(tables, lens, refs, 16)
    pools = [torch.randint(0, 255, (40, 16 + 16 * (i % 5)), dtype=torch.uint8) for i in range(70)]
    dpools = [p.cuda() for p in pools]
    _, _, pairs = dev.step(_i32([1, 1, 0]), 2, pools=dpools)
    want = model.step(tables, lens, refs, [1, 1, 0], 16, 2)[2]
    assert [tuple(p) for p in pairs.tolist()] == want and want[0] == (5, 0)
    _, moves = dev.compact(pools=dpools)
    for s, t in want + model.compact(tables, lens, refs, 16)[1]:
        if s >= 0:
            for p in pools:
                p[t] = p[s]
    assert dev.block_tables.tolist() == tables and dev.ref_counts.tolist() == refs
    for p, d in zip(pools, dpools):
        assert torch.equal(d.cpu(), p)
    assert _lib.pa_get_device_error() == 0


@gpu
def test_two_tables_at_once():
    """Steps and compactions of two tables on two streams, each against its own model."""
    from paged_kv_cache_388_b200 import _lib
    r = random.Random(3)
    both = []
    for rows, width, nb in ((300, 20, 9000), (40, 30, 70000)):
        tables, lens, refs = _state(r, rows, width, nb, 16, 60)
        both.append([tables, lens, refs, _device(tables, lens, refs, 16), torch.cuda.Stream(),
                     torch.zeros(nb, 1024, dtype=torch.uint8, device="cuda")])
    torch.cuda.synchronize()
    for _ in range(4):
        todo = []
        for t in both:
            append = [r.randint(0, 20) for _ in t[1]]
            release = [int(r.random() < 0.2) for _ in t[1]]
            todo.append((append, release, _i32(append), _i32(release)))
        torch.cuda.synchronize()
        for (append, release, da, dr), (_, _, _, dev, st, pool) in zip(todo, both):
            with torch.cuda.stream(st):
                dev.step(da, sum(append), release=dr, pools=[pool])
                dev.compact(pools=[pool])
        torch.cuda.synchronize()
        for (append, release, _, _), (tables, lens, refs, dev, _, _) in zip(todo, both):
            model.step(tables, lens, refs, append, 16, 0, release)
            model.compact(tables, lens, refs, 16)
            assert dev.block_tables.tolist() == tables and dev.ref_counts.tolist() == refs
            assert dev.context_lens.tolist() == lens
    _lib.pa_get_device_error()


@gpu
def test_from_the_host_allocator():
    from paged_kv_cache_388_b200.tables import DeviceBlockTables
    al = BlockAllocator(50, 16, free_order=reversed(range(50)))
    a, b = al.new_sequence(40), al.new_sequence(5)
    c = al.fork(a)
    dev = DeviceBlockTables.from_allocator(al, [a, b, c], 6)
    assert dev.context_lens.tolist() == [40, 5, 40]
    assert dev.ref_counts.tolist() == [al.refcount(x) for x in range(50)]
    slots, _, pairs = dev.step(_i32([1, 0, 1]), 2)
    last = al.block_table(a)[-1]
    assert pairs.tolist() == [[last, 0], [-1, -1], [-1, -1]] and slots.tolist() == [8, last * 16 + 8]


@gpu
def test_pools_of_the_kv_cache_follow():
    """Compaction under PagedKVCache: the attention output stays the same bit for bit."""
    from paged_kv_cache_388_b200.session import PagedKVCache
    g = torch.Generator().manual_seed(0)
    cache = PagedKVCache(64, 2, 128, 16)
    for t in (cache.k_cache, cache.v_cache):
        t.copy_(torch.randn(t.shape, generator=g))
    perm = torch.randperm(64, generator=g)[:12].tolist()
    refs = [int(b in perm) for b in range(64)]
    dev = _device([perm[:6], perm[6:]], [90, 81], refs, 16)
    q = torch.randn(2, 8, 128, generator=g).to(torch.bfloat16).cuda()
    want = cache.attend(q, dev.block_tables, dev.context_lens, 0.1)
    live, _ = dev.compact(pools=[cache.k_cache, cache.v_cache])
    assert live.tolist() == [12] and int(dev.block_tables.max()) < 12
    assert torch.equal(cache.attend(q, dev.block_tables, dev.context_lens, 0.1), want)
