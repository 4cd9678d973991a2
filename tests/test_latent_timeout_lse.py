"""Rows of the latent cache's attention that a timed-out wait left as zeros carry
an lse of -infinity, so that a merge by lse gives them no weight
(libpa_waittest.so: a 50 ms limit and one copy of CTA 0 announced but never made)."""
import math

import pytest
import torch

from test_latent_wait_timeout import waittest  # noqa: F401

pytestmark = pytest.mark.gpu


def _compare(waittest, call):  # noqa: F811
    from paged_kv_cache_388_b200 import _lib
    want, want_lse = call()
    assert _lib.pa_get_device_error() == 0
    waittest(True)
    out, lse = call()
    code = _lib.pa_get_device_error()
    waittest(False)
    assert code & _lib.PA_DEVERR_TIMEOUT, hex(code)
    zero = (out == 0).all(-1)
    assert bool(zero.any()) and not bool((want == 0).all(-1).any())
    assert torch.all(lse[zero] == -math.inf)
    assert torch.equal(lse[~zero], want_lse[~zero]) and torch.equal(out[~zero], want[~zero])


# an item a CTA, of rows that see up to a thousand keys: CTA 0 loses its fourth tile; cut over the keys
@pytest.mark.parametrize("rows,keys,heads,dn", [(900, 900, 60, 128), (600, 1400, 60, 64), (300, 60000, 3, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(waittest, rows, keys, heads, dn, causal):  # noqa: F811
    from paged_kv_cache_388_b200.latent import latent_prefill
    g = torch.Generator().manual_seed(0)
    q = torch.randn(rows, heads, dn + 64, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(keys, heads, 2 * dn, generator=g).to(torch.bfloat16).cuda()
    kr = torch.randn(keys, 64, generator=g).to(torch.bfloat16).cuda()
    start = [torch.tensor([0, n], dtype=torch.int32).cuda() for n in (rows, keys)]

    def call():
        lse = torch.empty(rows, heads, device="cuda")
        out = latent_prefill(q, kv[..., :dn], kr, kv[..., dn:], *start, 0.07, max_query_len=rows, lse=lse, causal=causal)
        return out, lse

    _compare(waittest, call)


@pytest.mark.parametrize("heads,latent", [(16, 512), (40, 256)])
def test_decode(waittest, heads, latent):  # noqa: F811
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(300, 1500, (90,), generator=g).tolist()
    blocks = [-(-n // 16) for n in lens]
    tables = torch.zeros(len(lens), max(blocks), dtype=torch.int32)
    for i, part in enumerate(torch.randperm(sum(blocks), generator=g).to(torch.int32).split(blocks)):
        tables[i, : len(part)] = part
    cache = torch.randn(sum(blocks), 16, latent + 64, generator=g).to(torch.bfloat16).cuda()
    user = PagedLatentCache(sum(blocks), latent, 64, 16, latent_cache=cache)
    args = (torch.randn(len(lens), heads, latent + 64, generator=g).to(torch.bfloat16).cuda(), tables.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), 0.05)

    def call():
        lse = torch.empty(len(lens), heads, device="cuda")
        return user.attend(*args, lse=lse), lse

    _compare(waittest, call)
