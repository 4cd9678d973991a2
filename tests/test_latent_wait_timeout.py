"""A wait of the latent cache's attention kernels that runs out ends in
PA_DEVERR_TIMEOUT, not a hang (libpa_waittest.so: a 50 ms limit and one copy of
CTA 0 announced but never made).  Outputs of the unwound CTA are zeros, all others
equal the normal library's, and the device keeps working."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def waittest(monkeypatch):
    """The binding over the test build."""
    from paged_kv_cache_388_b200 import _lib, build
    lib = ctypes.CDLL(build.WAITTEST_LIB)
    for name in ("pa_latent_decode", "pa_latent_prefill", "pa_get_device_error", "pa_status_string",
                 "pa_latent_decode_workspace_size", "pa_latent_prefill_workspace_size"):
        f, g = getattr(lib, name), getattr(_lib._lib, name)
        f.restype, f.argtypes = g.restype, g.argtypes

    normal = _lib._lib
    yield lambda on: monkeypatch.setattr(_lib, "_lib", lib if on else normal)


def _compare(waittest, call):
    from paged_kv_cache_388_b200 import _lib
    want, lse = call()
    assert _lib.pa_get_device_error() == 0
    waittest(True)
    got, got_lse = call()
    code = _lib.pa_get_device_error()
    waittest(False)
    assert code & _lib.PA_DEVERR_TIMEOUT, hex(code)
    assert not torch.isnan(got).any()
    same, zero = (got == want).all(-1), (got == 0).all(-1)
    assert bool((same | zero).all()) and bool(zero.any()) and bool(same.any())
    assert torch.equal(got_lse[same & ~zero], lse[same & ~zero])
    again, _ = call()
    assert torch.equal(again, want) and _lib.pa_get_device_error() == 0


@pytest.mark.parametrize("heads,latent", [(16, 512), (128, 512), (40, 256)])
def test_decode(waittest, heads, latent):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(300, 1500, (90,), generator=g).tolist()
    blocks = [-(-n // 16) for n in lens]
    tables = torch.zeros(len(lens), max(blocks), dtype=torch.int32)
    ids = torch.randperm(sum(blocks), generator=g).to(torch.int32)
    for i, part in enumerate(ids.split(blocks)):
        tables[i, : len(part)] = part
    cache = torch.randn(sum(blocks), 16, latent + 64, generator=g).to(torch.bfloat16).cuda()
    user = PagedLatentCache(sum(blocks), latent, 64, 16, latent_cache=cache)
    args = (torch.randn(len(lens), heads, latent + 64, generator=g).to(torch.bfloat16).cuda(), tables.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), 0.05)

    def call():
        lse = torch.empty(len(lens), heads, device="cuda")
        return user.attend(*args, lse=lse), lse

    _compare(waittest, call)


# an item a CTA; split over the keys, long enough for CTA 0 to have a fourth tile
@pytest.mark.parametrize("rows,keys,heads", [(700, 700, 60), (300, 60000, 3)])
def test_prefill(waittest, rows, keys, heads):
    from paged_kv_cache_388_b200.latent import latent_prefill
    g = torch.Generator().manual_seed(0)
    q = torch.randn(rows, heads, 192, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(keys, heads, 256, generator=g).to(torch.bfloat16).cuda()
    kr = torch.randn(keys, 64, generator=g).to(torch.bfloat16).cuda()
    start = [torch.tensor([0, n], dtype=torch.int32).cuda() for n in (rows, keys)]

    def call():
        lse = torch.empty(rows, heads, device="cuda")
        out = latent_prefill(q, kv[..., :128], kr, kv[..., 128:], *start, 0.07, max_query_len=rows, lse=lse)
        return out, lse

    _compare(waittest, call)
