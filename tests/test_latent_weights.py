"""The latent cache's attention with many weak keys beside one strong one: each
weak weight is far below the strong one's, all of them together are not."""
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


def _weak(n, gap, dtype):
    """out and lse of one key of logit 0 and value 0 and n - 1 keys of logit -gap and value 1, and how far a kernel may be
    from them: weights and result are each rounded once to the type; the exponential and the sums over n keys run in fp32
    (an argument below 2^5 is off by 2^-19, the exponential and each sum by 2^-22 and n 2^-24); an f16 weight that is
    subnormal is off by 2^-25 where the largest is at least 2^7."""
    total = 1.0 + (n - 1) * math.exp(-gap)
    out = (total - 1.0) / total
    rel = 2.0 * HALF_STEP[dtype] + 2.0 ** -18 + 2.0 * n * 2.0 ** -24
    small = n * 2.0 ** -32 if dtype == torch.float16 else 0.0
    return out, math.log(total), rel * out + small, 2.0 ** -18 + 2.0 * n * 2.0 ** -24


GAPS = [17.34375, 14.0, 10.5]  # exact in both types (bf16: 17.375); below, at and above f16's least normal weight


def _rounded(gap, dtype):
    return float(torch.tensor(gap).to(dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("heads,latent,rows", [(16, 512, 1), (3, 256, 1), (40, 256, 1), (128, 512, 1), (24, 512, 3)])
def test_decode_weak_keys_beside_a_strong_one(lib, heads, latent, rows, gap, dtype):
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    dt, n, bs, seqs = DT[dtype], 16384, 64, 160  # more sequences than SMs: most are not cut
    gap = _rounded(gap, dt)
    cache = torch.zeros(n, latent + 64, dtype=dt)
    cache[1:, :latent] = 1.0
    cache[1:, latent] = -gap
    user = PagedLatentCache(n // bs, latent, 64, bs, latent_cache=cache.view(n // bs, bs, -1).cuda())
    q = torch.zeros(seqs * rows, heads, latent + 64, dtype=dt)
    q[..., latent] = 1.0
    tables = torch.arange(n // bs, dtype=torch.int32).expand(seqs, -1).contiguous().cuda()
    lse = torch.empty(seqs * rows, heads, device="cuda")
    qsl = torch.arange(0, seqs * rows + 1, rows, dtype=torch.int32).cuda() if rows > 1 else None
    out = user.attend(q.cuda(), tables, torch.full((seqs,), n, dtype=torch.int32).cuda(), 1.0, lse=lse, query_start_loc=qsl,
                      max_query_len=rows)
    assert lib.pa_get_device_error() == 0
    for t in range(rows):
        want, want_lse, far, far_lse = _weak(n - rows + 1 + t, gap, dt)
        assert float((out[t::rows].double() - want).abs().max()) <= far, t
        assert float((lse[t::rows].double() - want_lse).abs().max()) <= far_lse, t


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("heads,dn,n,rows", [(160, 128, 6000, 1), (40, 64, 6000, 1025), (2, 64, 60000, 100)])
def test_prefill_weak_keys_beside_a_strong_one(lib, heads, dn, n, rows, gap, dtype):
    from paged_kv_cache_388_b200.latent import latent_prefill
    dt = DT[dtype]
    gap = _rounded(gap, dt)
    q = torch.zeros(rows, heads, dn + 64, dtype=dt, device="cuda")
    q[..., dn] = 1.0
    k = torch.zeros(n, heads, dn, dtype=dt, device="cuda")
    v = torch.ones(n, heads, dn, dtype=dt, device="cuda")
    v[0] = 0.0
    kr = torch.zeros(n, 64, dtype=dt, device="cuda")
    kr[1:, 0] = -gap
    start = [torch.tensor([0, x], dtype=torch.int32).cuda() for x in (rows, n)]
    lse = torch.empty(rows, heads, device="cuda")
    out = latent_prefill(q, k, kr, v, *start, 1.0, max_query_len=rows, lse=lse)
    assert lib.pa_get_device_error() == 0
    for t in {0, rows // 2, rows - 1}:
        want, want_lse, far, far_lse = _weak(n - rows + 1 + t, gap, dt)
        assert float((out[t].double() - want).abs().max()) <= far, t
        assert float((lse[t].double() - want_lse).abs().max()) <= far_lse, t


@pytest.mark.parametrize("latent", [512, 256])
def test_decode_large_f16_logits_stay_finite(lib, latent):
    """Logits near 2^25, where the reference is known to a few units only: the largest weights saturate, nothing is
    infinite.  All keys alike, so that every weighted mean is 1."""
    from paged_kv_cache_388_b200.latent import PagedLatentCache
    cache = torch.ones(40, 16, latent + 64, dtype=torch.float16)
    cache[..., latent:] = torch.linspace(20000.0, 24000.0, 640).view(40, 16, 1)
    user = PagedLatentCache(40, latent, 64, 16, latent_cache=cache.cuda())
    q = torch.full((1, 16, latent + 64), 25.0, dtype=torch.float16, device="cuda")
    out = user.attend(q, torch.arange(40, dtype=torch.int32)[None].cuda(), torch.tensor([640], dtype=torch.int32).cuda(), 1.0)
    assert torch.isfinite(out).all()
