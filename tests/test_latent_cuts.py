"""The latent cache's attention where a sequence's keys are cut over the machine
and joined: every key counts, none twice.

With scale 0 all visible keys weigh the same, and key j's value is 1 in column
j mod R alone, so out * keys is the number of keys seen per column and exp(lse)
the number of keys: one key lost or taken twice changes a column by one part in
its count (at most 160 here: 0.6 %, beside a rounding of the result of 0.4 % at
most) and lse by one part in the keys (2^-15 at least, beside 2^-18)."""
import math

import pytest
import torch

from latent_ref import HALF_STEP

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_388_b200 import _lib
    assert torch.cuda.is_available()
    return _lib


def _one_hot(n, width, cols, dtype):
    x = torch.zeros(n, width, dtype=dtype)
    x[torch.arange(n), torch.arange(n) % cols] = 1.0
    return x


def _check(out, lse, limit, cols, dtype):
    """out [T, H, cols], lse [T, H]: row t sees the first limit[t] keys."""
    limit = limit.clamp(min=0)
    count = (limit[:, None] + cols - 1 - torch.arange(cols)[None]).div(cols, rounding_mode="floor")  # keys per column
    want = (count.double() / limit.clamp(min=1)[:, None])[:, None]
    # the result's rounding, and in fp32 the exponential's, the inverse's and the product's
    far = (out.double().cpu() - want).abs()
    assert torch.all(far <= want * (HALF_STEP[dtype] + 2.0 ** -21)), far.max()
    some = limit > 0
    assert torch.all(lse.cpu()[~some] == -math.inf)
    # fp32: the logarithm of a sum below 2^32 is off by 2^-19 in base 2, the rest by half of that
    assert torch.all((lse.double().cpu()[some] - torch.log(limit[some].double())[:, None]).abs() <= 2.0 ** -18)
    # the bounds tell one key more or less
    big = int(limit.max())
    if big:
        assert 1.0 / (big // cols + 1) > 1.5 * HALF_STEP[dtype] and 1.0 / big > 2.0 ** -18


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,heads,latent,rows", [
    ([20011], 16, 512, None), ([20011], 128, 512, None), ([15000], 33, 256, None),  # one sequence, all workers on it
    ([9001, 1, 0, 37, 30000, 64, 2000], 16, 512, None), ([9001, 1, 0, 37, 30000, 64, 2000], 100, 512, None),
    ([31 * i for i in range(200)], 16, 512, None), ([17 * i for i in range(300)], 64, 256, None),
    ([20011], 40, 512, [4]), ([9001, 2, 0, 37, 30000, 64, 2000], 48, 512, [3, 4, 0, 1, 5, 2, 7]),  # rows differ
    ([15000, 3, 7777], 32, 256, [4, 2, 3]), ([129 * i for i in range(90)], 24, 256, [i % 5 for i in range(90)])])
def test_decode_counts_every_key_once(lib, lens, heads, latent, rows, dtype):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    dt, bs = DT[dtype], 16
    g = torch.Generator().manual_seed(len(lens) + heads)
    blocks = [-(-n // bs) for n in lens]
    nb = -(-max(lens) // bs)
    # all sequences' rows are the same keys, in one pool in disorder
    perm = torch.randperm(nb, generator=g)
    cache = torch.zeros(nb, bs, latent + 64, dtype=dt)
    cache[perm] = _one_hot(nb * bs, latent + 64, latent, dt).view(nb, bs, -1)
    tables = torch.full((len(lens), nb), 2 ** 30, dtype=torch.int32)
    for i, b in enumerate(blocks):
        tables[i, :b] = perm[:b]
    counts = rows or [1] * len(lens)
    q = torch.randn(sum(counts), heads, latent + 64, generator=g).to(dt).cuda()
    qsl = None
    if rows is not None:
        qsl = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32).cuda()
    user = PagedLatentCache(nb, latent, 64, bs, latent_cache=cache.cuda())
    lse = torch.empty(sum(counts), heads, device="cuda")
    out = user.attend(q, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.0, lse=lse, query_start_loc=qsl,
                      max_query_len=max(counts))
    assert lib.pa_get_device_error() == 0
    limit = torch.cat([torch.arange(c) + n - c + 1 for n, c in zip(lens, counts)])
    _check(out, lse, limit, latent, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("qs,ks,heads,dn,causal", [
    ([100], [20000], 4, 128, True), ([1], [9001], 1, 64, True), ([300, 1], [8001, 2000], 2, 64, True),
    ([257], [10000], 1, 128, False), ([40, 900], [3000, 130], 5, 128, True),  # keys cut over the machine
    ([700, 300], [3000, 4001], 40, 128, True)])  # an item a CTA
def test_prefill_counts_every_key_once(lib, qs, ks, heads, dn, causal, dtype):
    from paged_kv_cache_388_b200.latent import latent_prefill
    dt = DT[dtype]
    g = torch.Generator().manual_seed(heads)
    q = torch.randn(sum(qs), heads, dn + 64, generator=g).to(dt).cuda()
    v = torch.cat([_one_hot(n, dn, dn, dt) for n in ks])[:, None].expand(-1, heads, -1).contiguous().cuda()
    k = torch.randn(sum(ks), 1, dn, generator=g).to(dt).expand(-1, heads, -1).contiguous().cuda()
    kr = torch.randn(sum(ks), 64, generator=g).to(dt).cuda()
    start = lambda n: torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda()  # noqa: E731
    lse = torch.empty(sum(qs), heads, device="cuda")
    out = latent_prefill(q, k, kr, v, start(qs), start(ks), 0.0, max_query_len=max(qs), lse=lse, causal=causal)
    assert lib.pa_get_device_error() == 0
    limit = torch.cat([torch.arange(n) + m - n + 1 if causal else torch.full((n,), m) for n, m in zip(qs, ks)])
    _check(out, lse, limit, dn, dt)


def test_what_is_cut(lib):
    """Keys are cut, and a workspace asked for, where few rows meet many keys."""
    need = lib.pa_latent_prefill_workspace_size
    assert need(1, 1, 1024, 16, 128) > 0 and need(1, 200, 2048, 16, 64) > 0 and need(2, 1024, 16384, 16, 128) > 0
    assert need(1, 1, 1023, 16, 128) == 0 and need(1, 200, 2047, 16, 128) == 0 and need(2, 1024, 1024, 16, 128) == 0
    assert need(1, 1, 1 << 20, 148, 128) == 0  # items enough for every SM
