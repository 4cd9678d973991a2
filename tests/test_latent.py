"""The latent cache on the GPU: byte-exact writes, absorbed and expanded
attention against plain 64-bit restatements, at the sizes and masks where they
can go wrong."""
import math

import pytest
import torch

from latent_ref import attend, bounds

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_388_b200 import _lib
    assert torch.cuda.is_available()
    return _lib


def _randn(g, *shape):
    return torch.randn(*shape, generator=g)


def _paged(lens, bs, width, dtype, seed, extra_blocks=5, fill=None):
    """A cache [NB, bs, width] with every slot finite, or `fill` in the slots no sequence holds, and tables."""
    g = torch.Generator().manual_seed(seed)
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks) + extra_blocks
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(1, max(blocks)) + 2), 2 ** 30, dtype=torch.int32)
    cache = _randn(g, nb, bs, width).to(dtype)
    held = torch.zeros(nb, bs, dtype=torch.bool)
    at = 0
    for i, (n, b) in enumerate(zip(lens, blocks)):
        tables[i, :b] = perm[at:at + b]
        at += b
        for j in range(b):
            held[tables[i, j], : min(bs, n - j * bs)] = True
    if fill is not None:
        cache[~held] = fill
    return cache, tables


def _rows(cache, tables, i, n, bs):
    b = -(-n // bs)
    return cache[tables[i, :b].long()].reshape(-1, cache.shape[2])[:n].double()


# ---- writes ------------------------------------------------------------------------


@pytest.mark.parametrize("tokens,latent,bs,dtype", [(1, 512, 16, "bf16"), (7, 256, 32, "f16"), (300, 512, 64, "bf16"),
                                                    (5003, 256, 16, "bf16")])
def test_write_is_exact_and_skips_padding(lib, tokens, latent, bs, dtype):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    g = torch.Generator().manual_seed(tokens)
    nb = tokens // bs + 3
    both = _randn(g, tokens, latent + 64 + 8).to(DT[dtype])  # rows 8 values longer than used
    slots = torch.randperm(nb * bs, generator=g)[:tokens]
    slots[::3] = -1
    before = _randn(g, nb, bs, latent + 64).to(DT[dtype])
    want = before.clone().view(-1, latent + 64)
    want[slots[slots >= 0]] = both[slots >= 0, : latent + 64]
    both = both.cuda()
    user = PagedLatentCache(nb, latent, 64, bs, latent_cache=before.cuda())
    user.write(both[:, :latent], both[:, latent:latent + 64], slots.cuda())
    assert lib.pa_get_device_error() == 0
    assert torch.equal(user.latent_cache.cpu().view(torch.int16), want.view(nb, bs, -1).view(torch.int16))


def test_write_past_the_pool_is_reported_and_skipped(lib):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    user = PagedLatentCache(4, 256, 64, 16, latent_cache=torch.zeros(4, 16, 320, dtype=torch.bfloat16, device="cuda"))
    user.write(torch.ones(2, 256, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 64, dtype=torch.bfloat16, device="cuda"),
               torch.tensor([64, 3], device="cuda"))
    assert lib.pa_get_device_error() == lib.PA_DEVERR_SLOT
    got = user.latent_cache.cpu().view(64, 320).float().sum(1)
    assert got[3] == 320 and got.sum() == 320


# ---- absorbed form -----------------------------------------------------------------


def _check_decode(lib, lens, heads, latent, bs, dtype, rows=None, scale=0.07, spread=1.0, seed=0, fill=float("nan"),
                  pad_rows=0, max_context_len=0):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    dt = DT[dtype]
    cache, tables = _paged(lens, bs, latent + 64, dt, seed, fill=fill)
    g = torch.Generator().manual_seed(seed + 1)
    counts = rows or [1] * len(lens)
    tq = sum(counts) + pad_rows
    q = (_randn(g, tq, heads, latent + 64) * spread).to(dt)
    qsl = None
    if rows is not None:
        qsl = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32).cuda()
    user = PagedLatentCache(cache.shape[0], latent, 64, bs, latent_cache=cache.cuda())
    out = torch.full((tq, heads, latent), 7.0, dtype=dt, device="cuda")
    lse = torch.full((tq, heads), 7.0, device="cuda")
    got = user.attend(q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale, out=out, lse=lse,
                      query_start_loc=qsl, max_query_len=max(counts), max_context_len=max_context_len)
    assert got is out and lib.pa_get_device_error() == 0
    out, lse, at = out.cpu().double(), lse.cpu().double(), 0
    for i, (n, c) in enumerate(zip(lens, counts)):
        k = _rows(cache, tables, i, n, bs)
        limit = (torch.arange(c) + n - c + 1).clamp(min=0)
        ref, ref_lse, absolute, size = attend(q[at:at + c].double(), k[:, None], k[:, None, :latent], limit, scale)
        b_out, b_lse = bounds(ref, ref_lse, absolute, size, n, latent + 64, dt)
        blank = limit <= 0
        assert torch.all(out[at:at + c][blank] == 0) and torch.all(lse[at:at + c][blank] == -math.inf)
        far = (out[at:at + c] - ref).abs() - b_out
        assert torch.all(far[~blank] <= 0), (i, n, c, far.max())
        far = (lse[at:at + c] - ref_lse).abs() - b_lse
        assert torch.all(far[~blank] <= 0), (i, n, c, far[~blank].max())
        at += c
    assert torch.all(out[at:] == 7) and torch.all(lse[at:] == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("latent", [512, 256])
@pytest.mark.parametrize("bs", [16, 32, 64])
def test_decode_lengths_around_the_tiles(lib, bs, latent, dtype):
    _check_decode(lib, [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 0, 1000], 16, latent, bs, dtype)


@pytest.mark.parametrize("heads", [1, 2, 5, 8, 16, 17, 24, 32, 40, 64, 65, 96, 128, 144])
@pytest.mark.parametrize("latent", [512, 256])
def test_decode_head_counts(lib, heads, latent):
    _check_decode(lib, [1, 70, 333, 0, 129], heads, latent, 16, "bf16", seed=heads)


def test_decode_one_long_sequence_is_split(lib):
    _check_decode(lib, [20011], 16, 512, 16, "bf16")
    _check_decode(lib, [9000], 128, 512, 64, "f16")
    _check_decode(lib, [15000], 33, 256, 32, "bf16")


def test_decode_many_sequences(lib):
    r = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 700, (400,), generator=r).tolist()
    _check_decode(lib, lens, 16, 512, 16, "bf16")
    _check_decode(lib, lens[:200], 3, 256, 64, "f16")


@pytest.mark.parametrize("heads,rows", [(16, 4), (32, 4), (128, 3), (5, 7), (40, 2), (1, 33)])
@pytest.mark.parametrize("latent", [512, 256])
def test_decode_rows_of_drafted_tokens(lib, heads, rows, latent):
    # sequences with fewer keys than rows leave rows without any
    r = torch.Generator().manual_seed(heads)
    counts = torch.randint(1, rows + 1, (7,), generator=r).tolist()
    lens = [c + x for c, x in zip(counts, [0, 1, 62, 64, 300, 1000, -1])]
    counts[2], lens[2] = 0, 50  # a sequence without rows in this step
    _check_decode(lib, lens, heads, latent, 32, "bf16", rows=counts, pad_rows=3, fill=0.5)


def test_decode_rows_past_the_last_sequence_are_left(lib):
    _check_decode(lib, [40, 3], 16, 512, 16, "f16", rows=[1, 1], pad_rows=5)


def test_decode_large_logits_and_growing_maximum(lib):
    # logits of +-300 make the running maximum move between tiles
    _check_decode(lib, [1500, 700], 16, 512, 16, "bf16", scale=0.5, spread=25.0)
    _check_decode(lib, [1500, 700], 64, 256, 16, "f16", scale=0.5, spread=25.0)
    # zero scale: every key weighs the same
    _check_decode(lib, [1500, 70], 16, 512, 16, "f16", scale=0.0)


def test_decode_rising_logits_rescale_every_tile(lib):
    # key j's logit grows along the sequence, so each tile has a new maximum
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    n, heads, latent = 1000, 20, 512
    g = torch.Generator().manual_seed(3)
    cache = _randn(g, 64, 16, 576) * 0.01
    cache[..., 0] = (torch.arange(1024) / 4.0).view(64, 16)
    cache = cache.to(torch.bfloat16)
    q = _randn(g, 1, heads, 576) * 0.01
    q[..., 0] = 1.0
    q = q.to(torch.bfloat16)
    tables = torch.arange(64, dtype=torch.int32)[None]
    user = PagedLatentCache(64, latent, 64, 16, latent_cache=cache.cuda())
    lse = torch.empty(1, heads, device="cuda")
    out = user.attend(q.cuda(), tables.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 1.0, lse=lse)
    k = cache.view(-1, 576)[:n].double()
    ref, ref_lse, absolute, size = attend(q.double(), k[:, None], k[:, None, :latent], torch.tensor([n]), 1.0)
    b_out, b_lse = bounds(ref, ref_lse, absolute, size, n, 576, torch.bfloat16)
    assert torch.all((out.cpu().double() - ref).abs() <= b_out)
    assert torch.all((lse.cpu().double() - ref_lse).abs() <= b_lse)


def test_decode_bad_lengths_and_blocks_are_zeroed_and_reported(lib):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    cache, tables = _paged([100, 100, 100, 100], 16, 576, torch.bfloat16, 0)
    tables[1, 3] = cache.shape[0]
    tables[2, 0] = -1
    user = PagedLatentCache(cache.shape[0], 512, 64, 16, latent_cache=cache.cuda())
    g = torch.Generator().manual_seed(0)
    q = _randn(g, 4, 16, 576).to(torch.bfloat16)
    for lens, bits, good in (([100] * 4, lib.PA_DEVERR_BLOCK_ID, [0, 3]),
                             ([100, 0, 0, 10 ** 6], lib.PA_DEVERR_CONTEXT_LEN, [0]),
                             ([100, 40, 0, -5], lib.PA_DEVERR_CONTEXT_LEN, [0, 1])):
        lse = torch.zeros(4, 16, device="cuda")
        out = user.attend(q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.1, lse=lse)
        assert lib.pa_get_device_error() == bits
        for i in range(4):
            if i in good:
                k = _rows(cache, tables, i, lens[i], 16)
                ref, _, absolute, size = attend(q[i:i + 1].double(), k[:, None], k[:, None, :512], torch.tensor([lens[i]]), 0.1)
                b, _ = bounds(ref, _, absolute, size, lens[i], 576, torch.bfloat16)
                assert torch.all((out[i:i + 1].cpu().double() - ref).abs() <= b)
            else:
                assert torch.all(out[i] == 0) and torch.all(lse[i] == -math.inf), i


def test_decode_more_rows_than_announced(lib):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    cache, tables = _paged([100, 100], 16, 320, torch.bfloat16, 0)
    user = PagedLatentCache(cache.shape[0], 256, 64, 16, latent_cache=cache.cuda())
    q = torch.ones(6, 16, 320, dtype=torch.bfloat16, device="cuda")
    qsl = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    out = user.attend(q, tables.cuda(), torch.tensor([100, 100], dtype=torch.int32).cuda(), 0.1, query_start_loc=qsl,
                      max_query_len=2)
    assert lib.pa_get_device_error() == lib.PA_DEVERR_QUERY_LEN
    assert torch.all(out[:4] == 0) and torch.all(out[4:].abs().sum(-1) > 0)


def test_a_cache_beyond_32_bit_offsets(lib):
    """Rows written and read where the byte offset passes 2^32 (a pool of 5 GB)."""
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    bs, nb, n = 64, 70000, 500
    user = PagedLatentCache(nb, 512, 64, bs)
    assert user.latent_cache.numel() * 2 > 5 * 10 ** 9
    g = torch.Generator().manual_seed(1)
    rows = _randn(g, n, 576).to(torch.bfloat16)
    ids = torch.arange(nb - 8, nb, dtype=torch.int32).flip(0)  # the last blocks
    pos = torch.arange(n)
    slots = ids[pos // bs].long() * bs + pos % bs
    user.write(rows[:, :512].cuda(), rows[:, 512:].cuda(), slots.cuda())
    q = _randn(g, 1, 16, 576).to(torch.bfloat16)
    out = user.attend(q.cuda(), ids[None].contiguous().cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 0.05)
    k = rows.double()
    ref, lse, absolute, size = attend(q.double(), k[:, None], k[:, None, :512], torch.tensor([n]), 0.05)
    assert torch.all((out.cpu().double() - ref).abs() <= bounds(ref, lse, absolute, size, n, 576, torch.bfloat16)[0])
    assert lib.pa_get_device_error() == 0


@pytest.mark.parametrize("latent_dim, tokens", [(512, 29826200), (256, 53687200)])
def test_write_of_more_vectors_than_31_bits(lib, latent_dim, tokens):
    """More than 2^31 16-byte vectors in one call: one row for all tokens, nearly all of them padding."""
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    row = latent_dim + 64
    assert tokens * (row // 8) > 2 ** 31
    user = PagedLatentCache(4, latent_dim, 64, 16)
    user.latent_cache.fill_(-1.0)
    one = _randn(torch.Generator().manual_seed(4), 1, row).to(torch.bfloat16).cuda()
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    slots[0], slots[tokens // 2 + 1], slots[tokens - 1] = 3, 17, 63
    user.write(one[:, :latent_dim].expand(tokens, -1), one[:, latent_dim:].expand(tokens, -1), slots)
    want = torch.full((64, row), -1.0, dtype=torch.bfloat16, device="cuda")
    want[[3, 17, 63]] = one
    assert torch.equal(user.latent_cache.view(64, row), want)
    assert lib.pa_get_device_error() == 0


def test_decode_on_two_streams_and_captured(lib):
    """Two captured graphs and an eager call, replayed on different streams at once, each with its own result."""
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    g = torch.Generator().manual_seed(9)
    calls = []
    for seed, lens, heads in ((1, [3000, 10, 777], 16), (2, [6000], 128)):
        cache, tables = _paged(lens, 16, 576, torch.bfloat16, seed)
        user = PagedLatentCache(cache.shape[0], 512, 64, 16, latent_cache=cache.cuda())
        args = (_randn(g, len(lens), heads, 576).to(torch.bfloat16).cuda(), tables.cuda(),
                torch.tensor(lens, dtype=torch.int32).cuda(), 0.05)
        want = user.attend(*args).clone()
        again = user.attend(*args)
        assert torch.equal(want, again)  # the same call gives the same bits
        calls.append((user, args, want))
    graphs = []
    for user, args, want in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = user.attend(*args)
        graphs.append((gr, out, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (gr, out, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for gr, out, want in graphs:
        assert torch.equal(out, want)
    assert lib.pa_get_device_error() == 0


# ---- expanded form -----------------------------------------------------------------


def _check_prefill(lib, qs, ks, heads, dn, dtype, causal=True, side_by_side=True, scale=None, spread=1.0, seed=0, pad_rows=0):
    from paged_kv_cache_388_b200.latent import latent_prefill
    dt = DT[dtype]
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(qs) + pad_rows, sum(ks)
    q = (_randn(g, tq, heads, dn + 64) * spread).to(dt)
    if side_by_side:
        kv = _randn(g, tk, heads, 2 * dn).to(dt).cuda()
        k, v = kv[:, :, :dn], kv[:, :, dn:]
        kr = _randn(g, tk, 576).to(dt).cuda()[:, 512:]  # the rope part of cache rows
    else:
        k, v, kr = (_randn(g, *s).to(dt).cuda() for s in ((tk, heads, dn), (tk, heads, dn), (tk, 64)))
    scale = 1.0 / math.sqrt(dn + 64) if scale is None else scale
    start = lambda n: torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda()  # noqa: E731
    out = torch.full((tq, heads, dn), 7.0, dtype=dt, device="cuda")
    lse = torch.full((tq, heads), 7.0, device="cuda")
    latent_prefill(q.cuda(), k, kr, v, start(qs), start(ks), scale, max_query_len=max(1, max(qs)), out=out, lse=lse, causal=causal)
    assert lib.pa_get_device_error() == 0
    out, lse = out.cpu().double(), lse.cpu().double()
    k, v, kr = k.cpu().double(), v.cpu().double(), kr.cpu().double()
    a = b = 0
    for i, (n, m) in enumerate(zip(qs, ks)):
        key = torch.cat([k[b:b + m], kr[b:b + m, None].expand(m, heads, 64)], 2)
        limit = (torch.arange(n) + m - n + 1).clamp(min=0) if causal else torch.full((n,), m)
        ref, ref_lse, absolute, size = attend(q[a:a + n].double(), key, v[b:b + m], limit, scale)
        b_out, b_lse = bounds(ref, ref_lse, absolute, size, m, dn + 64, dt)
        blank = limit <= 0
        assert torch.all(out[a:a + n][blank] == 0) and torch.all(lse[a:a + n][blank] == -math.inf)
        far = (out[a:a + n] - ref).abs() - b_out
        assert torch.all(far[~blank] <= 0), (i, n, m, far.max())
        far = (lse[a:a + n] - ref_lse).abs() - b_lse
        assert torch.all(far[~blank] <= 0), (i, n, m, far[~blank].max())
        a, b = a + n, b + m
    assert torch.all(out[a:] == 7) and torch.all(lse[a:] == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dn", [128, 64])
def test_prefill_ragged_prompts(lib, dn, dtype):
    qs = [1, 2, 127, 128, 129, 0, 255, 256, 257, 300, 64]
    _check_prefill(lib, qs, qs, 3, dn, dtype)


@pytest.mark.parametrize("dn", [128, 64])
def test_prefill_over_a_prefix(lib, dn):
    _check_prefill(lib, [100, 1, 256, 33], [1000, 513, 257, 33], 4, dn, "bf16", side_by_side=False)


@pytest.mark.parametrize("dn", [128, 64])
def test_prefill_rows_without_keys(lib, dn):
    # more rows than keys: the leading rows see nothing; and a sequence without any key
    _check_prefill(lib, [300, 2], [0, 0], 2, dn, "f16")
    _check_prefill(lib, [200, 5, 3, 130], [150, 0, 1, 2], 2, dn, "bf16", pad_rows=4)


@pytest.mark.parametrize("dn", [128, 64])
def test_prefill_not_causal(lib, dn):
    _check_prefill(lib, [200, 5, 3, 64], [150, 0, 700, 128], 2, dn, "f16", causal=False, pad_rows=2)


@pytest.mark.parametrize("qs,ks,heads,causal", [
    ([100], [5000], 4, True),  # a few rows over a long prefix: their keys are split over the machine
    ([1], [9001], 1, True), ([130, 1, 17], [1500, 1, 3000], 2, True), ([300], [700], 3, True), ([257], [4096], 1, False),
    ([700, 0, 5], [1100, 0, 0], 1, True), ([1500], [1100], 1, True), ([40, 900], [3000, 130], 5, True)])
@pytest.mark.parametrize("dn", [128, 64])
def test_prefill_split_over_the_keys(lib, dn, qs, ks, heads, causal):
    _check_prefill(lib, qs, ks, heads, dn, "bf16", causal=causal, seed=heads, pad_rows=3)


def test_workspaces_may_hold_anything(lib):
    """Bytes that read as NaN in the workspace, and one byte too few."""
    g = torch.Generator().manual_seed(2)
    cache, tables = _paged([3000, 70, 1], 16, 576, torch.bfloat16, 0)
    args = (_randn(g, 3, 16, 576).to(torch.bfloat16).cuda(), cache.cuda(), tables.cuda(),
            torch.tensor([3000, 70, 1], dtype=torch.int32).cuda(), 0.05)
    need = lib.pa_latent_decode_workspace_size(3, 1, 16, 512)
    outs = []
    for fill in (0, 255):
        outs.append(torch.empty(3, 16, 512, dtype=torch.bfloat16, device="cuda"))
        lib.pa_latent_decode(outs[-1], None, *args, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
    assert torch.equal(*outs)
    with pytest.raises(lib.PAError, match="WORKSPACE"):
        lib.pa_latent_decode(outs[0], None, *args, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    q = _randn(g, 90, 2, 192).to(torch.bfloat16).cuda()
    kv = _randn(g, 4000, 2, 256).to(torch.bfloat16).cuda()
    kr = _randn(g, 4000, 64).to(torch.bfloat16).cuda()
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    need = lib.pa_latent_prefill_workspace_size(1, 90, 4000, 2, 128)
    assert need > 0 and lib.pa_latent_prefill_workspace_size(8, 20000, 20000, 16, 128) == 0
    outs = []
    for fill in (0, 255):
        outs.append(torch.empty(90, 2, 128, dtype=torch.bfloat16, device="cuda"))
        lib.pa_latent_prefill(outs[-1], None, q, kv[..., :128], kr, kv[..., 128:], t(0, 90), t(0, 4000), 0.05, 90,
                              workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
    assert torch.equal(*outs)
    with pytest.raises(lib.PAError, match="WORKSPACE"):
        lib.pa_latent_prefill(outs[0], None, q, kv[..., :128], kr, kv[..., 128:], t(0, 90), t(0, 4000), 0.05, 90)
    assert lib.pa_get_device_error() == 0


def test_prefill_one_head_one_token(lib):
    _check_prefill(lib, [1], [1], 1, 128, "bf16")
    _check_prefill(lib, [1], [1], 1, 64, "f16", side_by_side=False)


def test_prefill_many_heads_and_sequences(lib):
    g = torch.Generator().manual_seed(1)
    qs = torch.randint(1, 90, (40,), generator=g).tolist()
    _check_prefill(lib, qs, [x + y for x, y in zip(qs, torch.randint(0, 200, (40,), generator=g).tolist())], 24, 128, "bf16")


def test_prefill_large_logits(lib):
    _check_prefill(lib, [300, 40], [600, 40], 2, 128, "bf16", scale=0.5, spread=25.0)
    _check_prefill(lib, [300, 40], [600, 40], 2, 64, "f16", scale=0.0)


def test_prefill_strides(lib):
    """Heads before tokens, and token rows whose distance is no multiple of a head's."""
    from paged_kv_cache_388_b200.latent import latent_prefill
    g = torch.Generator().manual_seed(6)
    n, heads = 150, 3
    q = _randn(g, n, heads, 192).to(torch.bfloat16).cuda()
    k, v = (_randn(g, n, heads, 128).to(torch.bfloat16).cuda() for _ in range(2))
    kr = _randn(g, n, 64).to(torch.bfloat16).cuda()
    sl = torch.tensor([0, n], dtype=torch.int32).cuda()
    want = latent_prefill(q, k, kr, v, sl, sl, 0.07, max_query_len=n)
    turned = k.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros(n, heads * 128 + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :heads * 128] = v.reshape(n, -1)
    padded = wide.as_strided((n, heads, 128), (heads * 128 + 8, 128, 1))
    assert torch.equal(latent_prefill(q, turned, kr, padded, sl, sl, 0.07, max_query_len=n), want)
    assert lib.pa_get_device_error() == 0


def test_prefill_infinities_behind_the_last_key(lib):
    """Tokens of k, v and k_rope past a sequence's keys may hold anything."""
    from paged_kv_cache_388_b200.latent import latent_prefill
    g = torch.Generator().manual_seed(4)
    q = _randn(g, 70, 2, 192).to(torch.bfloat16).cuda()
    kv = _randn(g, 400, 2, 256).to(torch.bfloat16).cuda()
    kr = _randn(g, 400, 64).to(torch.bfloat16).cuda()
    sl = torch.tensor([0, 70], dtype=torch.int32).cuda()
    args = dict(max_query_len=70)
    want = latent_prefill(q, kv[:70, :, :128], kr[:70], kv[:70, :, 128:], sl, sl, 0.07, **args)
    kv[70:], kr[70:] = float("nan"), float("inf")
    got = latent_prefill(q, kv[..., :128], kr, kv[..., 128:], sl, sl, 0.07, **args)
    assert torch.equal(got, want) and torch.isfinite(got).all()


def test_prefill_on_two_streams_and_captured(lib):
    """A split and a whole call captured, replayed on different streams at once."""
    from paged_kv_cache_388_b200.latent import latent_prefill
    g = torch.Generator().manual_seed(8)
    graphs = []
    for n, keys, heads in ((90, 6000, 2), (600, 600, 40)):
        q = _randn(g, n, heads, 192).to(torch.bfloat16).cuda()
        kv = _randn(g, keys, heads, 256).to(torch.bfloat16).cuda()
        kr = _randn(g, keys, 64).to(torch.bfloat16).cuda()
        qsl, ksl = (torch.tensor([0, x], dtype=torch.int32).cuda() for x in (n, keys))
        args = (q, kv[..., :128], kr, kv[..., 128:], qsl, ksl, 0.05)
        want = latent_prefill(*args, max_query_len=n)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = latent_prefill(*args, max_query_len=n)
        graphs.append((gr, out, want, args))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (gr, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for gr, out, want, _ in graphs:
        assert torch.equal(out, want)
    assert lib.pa_get_device_error() == 0


def test_prefill_bad_offsets_are_reported(lib):
    from paged_kv_cache_388_b200.latent import latent_prefill
    q = torch.ones(6, 2, 192, dtype=torch.bfloat16, device="cuda")
    kv = torch.ones(8, 2, 256, dtype=torch.bfloat16, device="cuda")
    kr = torch.ones(8, 64, dtype=torch.bfloat16, device="cuda")
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for qsl, ksl, rows, zero, left in (((0, 4, 6), (0, 4, 8), 3, slice(0, 4), None),  # more rows than announced
                                       ((0, 4, 6), (0, 4, 9), 4, None, slice(4, 6)),
                                       ((0, 4, 7), (0, 4, 8), 4, None, slice(4, 6)),
                                       ((0, 4, 3), (0, 4, 8), 4, None, slice(4, 6))):
        out = torch.full((6, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        latent_prefill(q, kv[..., :128], kr, kv[..., 128:], t(*qsl), t(*ksl), 0.1, max_query_len=rows, out=out)
        assert lib.pa_get_device_error() == lib.PA_DEVERR_QUERY_LEN
        want = torch.ones_like(out)
        if zero:
            want[zero] = 0
        if left:
            want[left] = 7
        assert torch.allclose(out, want)


# ---- as they are used together -----------------------------------------------------


def test_a_prompt_then_steps_through_the_device_tables(lib):
    """Prompts are admitted, attended in the expanded form and written; then decode steps with a fork and a release, all
    bookkeeping on the device, each step's absorbed attention against the rows that were written."""
    from paged_kv_cache_388_b200.latent import PagedLatentCache, latent_prefill
    from paged_kv_cache_388_b200.tables import DeviceBlockTables
    g = torch.Generator().manual_seed(11)
    heads, r, bs = 4, 256, 16
    dn, scale = 64, 0.09
    up_k, up_v = (_randn(g, r, heads, dn) / 16 for _ in range(2))
    tab = DeviceBlockTables(3, 40, 100, bs)
    cache = PagedLatentCache(100, r, 64, bs)
    rows = {0: [], 1: [], 2: []}  # every sequence's cache rows, on the host
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def grow(counts, release=None, fork=None):
        slots, qsl, _ = tab.step(i32(*counts), sum(counts), release=release, fork_src=fork, pools=[cache.latent_cache])
        new = _randn(g, sum(counts), r + 64).to(torch.bfloat16)
        cache.write(new[:, :r].cuda(), new[:, r:].cuda(), slots)
        for i, part in enumerate(new.split(counts)):
            rows[i] += list(part)
        return qsl

    prompt = [50, 7, 0]
    qsl = grow(prompt)
    # expanded: keys and values of the prompts' rows
    c = torch.stack(rows[0] + rows[1]).cuda()
    k = torch.einsum("td,dhn->thn", c[:, :r].float(), up_k.cuda()).to(torch.bfloat16)
    v = torch.einsum("td,dhn->thn", c[:, :r].float(), up_v.cuda()).to(torch.bfloat16)
    q = _randn(g, 57, heads, dn + 64).to(torch.bfloat16)
    out = latent_prefill(q.cuda(), k, c[:, r:], v, qsl, qsl, scale, max_query_len=50).cpu().double()
    at = 0
    for n in prompt[:2]:
        key = torch.cat([k[at:at + n].cpu().double(), c[at:at + n, None, r:].cpu().double().expand(n, heads, 64)], 2)
        ref, l, a, s = attend(q[at:at + n].double(), key, v[at:at + n].cpu().double(), torch.arange(n) + 1, scale)
        assert torch.all((out[at:at + n] - ref).abs() <= bounds(ref, l, a, s, n, dn + 64, torch.bfloat16)[0])
        at += n
    for step in range(20):
        release = fork = None
        if step == 3:
            fork, rows[2] = i32(-1, -1, 0), list(rows[0])
        if step == 12:
            release, rows[1] = i32(0, 1, 0), []
        grow([1, 1, 1], release, fork)
        q = _randn(g, 3, heads, r + 64).to(torch.bfloat16)
        lse = torch.empty(3, heads, device="cuda")
        out = cache.attend(q.cuda(), tab.block_tables, tab.context_lens, scale, lse=lse, max_context_len=200).cpu().double()
        if step == 15:
            tab.compact(pools=[cache.latent_cache])
        for i in range(3):
            k = torch.stack(rows[i]).double()
            ref, l, a, s = attend(q[i:i + 1].double(), k[:, None], k[:, None, :r], torch.tensor([len(rows[i])]), scale)
            b_out, b_lse = bounds(ref, l, a, s, len(rows[i]), r + 64, torch.bfloat16)
            assert torch.all((out[i:i + 1] - ref).abs() <= b_out), (step, i)
            assert torch.all((lse[i:i + 1].cpu().double() - l).abs() <= b_lse), (step, i)
    assert lib.pa_get_device_error() == 0
    assert int((tab.ref_counts > 0).sum()) == len({int(b) for i in range(3) for b in
                                                   tab.block_tables[i, : -(-len(rows[i]) // bs)].cpu()})
