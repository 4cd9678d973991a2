"""Expanded attention of batches whose sequences differ much in rows, or whose
announced maximum is far above any: one long prompt among many short ones."""
import math

import pytest
import torch

from test_latent import _check_prefill, lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dn,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("qs", [
    [2000] + [1] * 200, [1] * 200 + [2000], [0, 0] + [3, 0, 1] * 50 + [1537] + [0, 2] * 50 + [0],
    # offsets before, on and after multiples of 256
    [255, 1, 256, 0, 0, 257, 255, 1700, 1, 1, 254, 512, 0, 511, 3] + [0] * 150, [1300, 1300] + [85] * 120])
def test_one_long_prompt_among_short_ones(lib, qs, dn, dtype):  # noqa: F811
    _check_prefill(lib, qs, qs, 2, dn, dtype, pad_rows=300)


def test_prefixes_and_rows_without_keys(lib):  # noqa: F811
    qs = [1, 0, 900, 2] + [1, 5] * 60
    ks = [0, 3, 1000, 2] + [300, 0] * 60
    _check_prefill(lib, qs, ks, 3, 64, "bf16", pad_rows=1)
    _check_prefill(lib, qs, ks, 3, 64, "bf16", causal=False)


def _ones(tq, heads):
    q = torch.ones(tq, heads, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.arange(1, tq + 1, device="cuda").float().remainder(64).add(1)[:, None, None].expand(tq, heads, 64)
    return q, torch.ones_like(q[..., :64]), torch.ones(tq, 64, dtype=torch.bfloat16, device="cuda"), v.to(torch.bfloat16).contiguous()


def test_a_loose_maximum_changes_nothing(lib):  # noqa: F811
    from paged_kv_cache_388_b200.latent import latent_prefill
    g = torch.Generator().manual_seed(0)
    counts = [5, 0, 300, 1] * 40
    start = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32).cuda()
    q = torch.randn(sum(counts), 4, 192, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(sum(counts), 4, 256, generator=g).to(torch.bfloat16).cuda()
    kr = torch.randn(sum(counts), 64, generator=g).to(torch.bfloat16).cuda()
    call = lambda most: latent_prefill(q, kv[..., :128], kr, kv[..., 128:], start, start, 0.07, max_query_len=most)  # noqa: E731
    want = call(300)
    assert torch.equal(call(sum(counts)), want) and torch.equal(call(10 ** 9), want)
    assert lib.pa_get_device_error() == 0


@pytest.mark.parametrize("bad", ["rows", "keys", "end", "back"])
def test_bad_sequences_among_many(lib, bad):  # noqa: F811
    """More rows than announced: zeros.  Keys or rows outside the tensors: that sequence alone is skipped.  Row offsets that
    go back: reported, and nothing outside the tensors is touched."""
    from paged_kv_cache_388_b200.latent import latent_prefill
    counts = [1, 2, 1500, 700] + [1] * 150 + [40]
    tq, heads = sum(counts), 2
    q, k, kr, v = _ones(tq, heads)
    start = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    qsl, ksl, most, hit, value = start.clone(), start.clone(), 1500, None, 7.0
    if bad == "rows":
        most, hit, value = 1030, 2, 0.0
    elif bad == "keys":
        ksl[-1], hit = tq + 1, len(counts) - 1
    elif bad == "end":
        qsl[-1], hit = tq + 9, len(counts) - 1
    else:
        qsl[60], hit = 0, 0
    room = torch.full((tq + 64, heads, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq, heads), 7.0, device="cuda")
    out = latent_prefill(q, k, kr, v, qsl.cuda(), ksl.cuda(), 0.1, max_query_len=most, out=room[:tq], lse=lse)
    assert lib.pa_get_device_error() == lib.PA_DEVERR_QUERY_LEN
    assert torch.all(room[tq:] == 7)
    if bad == "back":
        assert torch.isfinite(out).all()
        return
    a, b = int(start[hit]), int(start[hit + 1])
    assert torch.all(out[a:b] == value)
    assert torch.all(lse[a:b] == (-math.inf if value == 0.0 else 7.0))
    for i, (x, y) in enumerate(zip(start.tolist(), start.tolist()[1:])):
        if i != hit:  # keys alike: the mean of the values so far, rounded once, weights exact
            want = v[x:y].double().cumsum(0) / torch.arange(1, y - x + 1, device="cuda")[:, None, None]
            assert torch.all((out[x:y].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want), i


def test_more_sequences_and_rows_than_a_grid_of_all_pairs_holds(lib):  # noqa: F811
    """Half a million sequences of two rows under an announced maximum of all rows: 2^31 pairs of a sequence and a place."""
    from paged_kv_cache_388_b200.latent import latent_prefill
    seqs = 2 ** 19
    tq = 2 * seqs + 600
    assert -(-tq // 256) * (seqs + 1) >= 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, kr, v = rand(tq, 1, 128), rand(tq, 1, 64), rand(tq, 64), rand(tq, 1, 64)
    start = torch.cat([torch.arange(0, 2 * seqs + 1, 2), torch.tensor([tq])]).to(torch.int32).cuda()
    out = latent_prefill(q, k, kr, v, start, start, 0.1, max_query_len=tq)
    assert lib.pa_get_device_error() == 0
    n = 2 * seqs
    key = torch.cat([k[:, 0], kr], 1).double()
    s = 0.1 * (q[1:n:2, 0].double()[:, None] * key[:n].view(seqs, 2, 128)).sum(-1)
    w = torch.softmax(s, -1)[..., None]
    both = v[:n, 0].double().view(seqs, 2, 64)
    assert torch.equal(out[0:n:2, 0], v[0:n:2, 0])
    want, absolute = (w * both).sum(1), (w * both.abs()).sum(1)
    # a rounding of each weight, one of the result, and logits of 128 fp32 terms
    far = 2.0 ** -8 * absolute + 2.0 ** -8 * (want.abs() + 2.0 ** -8 * absolute) + 2.0 ** -12 * absolute
    assert torch.all((out[1:n:2, 0].double() - want).abs() <= far)
    s = 0.1 * q[n:, 0].double() @ key[n:].T
    w = torch.softmax(s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(1), -math.inf), -1)
    want, absolute = w @ v[n:, 0].double(), w @ v[n:, 0].double().abs()
    far = 2.0 ** -8 * absolute + 2.0 ** -8 * (want.abs() + 2.0 ** -8 * absolute) + 2.0 ** -12 * absolute
    assert torch.all((out[n:, 0].double() - want).abs() <= far)
