"""Absorbed attention of batches whose sequences differ much in rows, or whose
announced maximum is far above any."""
import math

import pytest
import torch

from latent_ref import attend, bounds
from test_latent import _check_decode, _paged, _rows, lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,latent,dtype", [(3, 512, "bf16"), (16, 256, "f16"), (64, 512, "bf16")])
@pytest.mark.parametrize("rows", [[70] + [1] * 60, [1] * 60 + [70], [0, 0, 1] * 20 + [40, 0, 3] + [0, 2] * 15])
def test_many_rows_among_single_ones(lib, rows, heads, latent, dtype):  # noqa: F811
    lens = [max(0, 37 * (i % 31) + c - 1 + (i % 3)) for i, c in enumerate(rows)]
    _check_decode(lib, lens, heads, latent, 16, dtype, rows=rows, pad_rows=40, fill=0.5)


def _batch(n, heads, pad, seed=0):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, 900, (n,), generator=g).tolist()
    cache, tables = _paged(lens, 16, 320, torch.bfloat16, seed)
    user = PagedLatentCache(cache.shape[0], 256, 64, 16, latent_cache=cache.cuda())
    q = torch.randn(n + pad, heads, 320, generator=g).to(torch.bfloat16)
    return user, cache, q, tables, lens


def test_a_loose_maximum_gives_the_same_and_costs_little(lib):  # noqa: F811
    """Single rows announced as up to 4096: within the bounds, rows behind the last sequence left, and not many times the
    time of the call that announces them as they are (CTAs counted by the maximum made it 80 times)."""
    n, heads, pad = 256, 16, 3840
    user, cache, q, tables, lens = _batch(n, heads, pad)
    start = torch.arange(n + 1, dtype=torch.int32).cuda()
    dq, dt, dl = q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    out = torch.full((n + pad, heads, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + pad, heads), 7.0, device="cuda")

    def call(most):
        return user.attend(dq, dt, dl, 0.06, out=out, lse=lse, query_start_loc=start, max_query_len=most)

    def time(most):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        took = []
        for _ in range(7):
            torch.cuda.synchronize()
            a.record()
            call(most)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        return sorted(took)[3]

    call(4096)
    assert lib.pa_get_device_error() == 0
    assert torch.all(out[n:] == 7) and torch.all(lse[n:] == 7)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    for i in range(0, n, 5):
        k = _rows(cache, tables, i, lens[i], 16)
        ref, ref_lse, absolute, size = attend(q[i:i + 1].double(), k[:, None], k[:, None, :256], torch.tensor([lens[i]]), 0.06)
        b_out, b_lse = bounds(ref, ref_lse, absolute, size, lens[i], 320, torch.bfloat16)
        assert torch.all((got[i:i + 1] - ref).abs() <= b_out) and torch.all((got_lse[i:i + 1] - ref_lse).abs() <= b_lse)
    loose, exact = time(4096), time(1)
    assert loose < 8 * exact, (loose, exact)


def test_more_rows_than_announced_among_many(lib):  # noqa: F811
    n, heads = 80, 8
    user, cache, q, tables, lens = _batch(n, heads, 200, seed=2)
    start = torch.cat([torch.arange(n), torch.tensor([n + 199])]).to(torch.int32).cuda()  # the last one has 200
    out = torch.full((n + 200, heads, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 200, heads), 7.0, device="cuda")
    user.attend(q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.06, out=out, lse=lse,
                query_start_loc=start, max_query_len=150)
    assert lib.pa_get_device_error() == lib.PA_DEVERR_QUERY_LEN
    assert torch.all(out[n - 1:n + 199] == 0) and torch.all(lse[n - 1:n + 199] == -math.inf)
    assert torch.all(out[n + 199:] == 7) and torch.all(out[: n - 1].abs().sum(-1) > 0)


@pytest.mark.parametrize("pad", [0, 300])
def test_row_offsets_out_of_range_are_skipped(lib, pad):  # noqa: F811
    """The sequence whose offsets leave the tensor is left as it was, all others are as ever; offsets that go back are
    reported, and nothing outside is touched."""
    n, heads = 60, 8
    user, cache, q, tables, lens = _batch(n, heads, pad, seed=1)
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    good = torch.arange(n + 1, dtype=torch.int32)
    most = max(1, pad)
    want = user.attend(q.cuda(), tables.cuda(), dl, 0.06, query_start_loc=good.cuda(), max_query_len=most)[:n]
    assert lib.pa_get_device_error() == 0
    bad = good.clone()
    bad[-1] = n + pad + 1
    room = torch.full((n + pad + 8, heads, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    out = user.attend(q.cuda(), tables.cuda(), dl, 0.06, out=room[:n + pad], query_start_loc=bad.cuda(), max_query_len=most)
    assert lib.pa_get_device_error() == lib.PA_DEVERR_QUERY_LEN
    # the line of tiles is cut elsewhere without it: half a step of the result and of each weight
    assert torch.all((out[:n - 1].float() - want[:n - 1].float()).abs() <= 2.0 ** -6 * want.float().abs().amax())
    assert torch.all(room[n - 1:] == 7)
    bad = good.clone()
    bad[30] = 2
    user.attend(q.cuda(), tables.cuda(), dl, 0.06, out=room[:n + pad], query_start_loc=bad.cuda(), max_query_len=most)
    assert lib.pa_get_device_error() == lib.PA_DEVERR_QUERY_LEN
    assert torch.all(room[n + pad:] == 7)
