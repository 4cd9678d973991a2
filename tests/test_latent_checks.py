"""Refusals of the latent cache's and the device tables' entry points (no GPU):
the binding refuses tensors that disagree, the library's host checks the rest."""
import ctypes

import pytest
import torch

from paged_kv_cache_388_b200 import _lib
from paged_kv_cache_388_b200.latent import PagedLatentCache, latent_prefill
from paged_kv_cache_388_b200.tables import DeviceBlockTables

BF = torch.bfloat16
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_write_shapes():
    cache = z(4, 16, 576)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="one row per token"):
        _lib.pa_latent_write(z(3, 512), z(2, 64), cache, slots)
    with pytest.raises(ValueError, match="576 values"):
        _lib.pa_latent_write(z(3, 256), z(3, 64), cache, slots)
    with pytest.raises(ValueError, match="one slot per token"):
        _lib.pa_latent_write(z(3, 512), z(3, 64), cache, slots[:2])
    with pytest.raises(ValueError, match="num_blocks, block_size"):
        _lib.pa_latent_write(z(3, 512), z(3, 64), z(64, 576), slots)
    with pytest.raises(ValueError, match="CUDA tensor"):
        _lib.pa_latent_write(z(3, 512), z(3, 64), cache, slots)
    with pytest.raises(ValueError, match="num_tokens, 512"):
        PagedLatentCache(4, 512, 64, 16, latent_cache=cache).write(z(3, 500), z(3, 76), slots)
    with pytest.raises(ValueError, match="latent_cache must be"):
        PagedLatentCache(5, 512, 64, 16, latent_cache=cache)


def test_decode_shapes():
    cache, q, out, t, n = z(4, 16, 576), z(2, 8, 576), z(2, 8, 512), i32(2, 3), i32(2)
    with pytest.raises(ValueError, match="match the cache"):
        _lib.pa_latent_decode(out, None, z(2, 8, 512), cache, t, n, 0.1)
    with pytest.raises(ValueError, match="out must be"):
        _lib.pa_latent_decode(z(2, 7, 512), None, q, cache, t, n, 0.1)
    with pytest.raises(ValueError, match="out must be"):
        _lib.pa_latent_decode(q, None, q, cache, t, n, 0.1)
    with pytest.raises(ValueError, match="lse must be"):
        _lib.pa_latent_decode(out, z(2, 9), q, cache, t, n, 0.1)
    with pytest.raises(ValueError, match="number of sequences"):
        _lib.pa_latent_decode(out, None, q, cache, t, i32(3), 0.1)
    with pytest.raises(ValueError, match="one row per sequence"):
        _lib.pa_latent_decode(z(3, 8, 512), None, z(3, 8, 576), cache, t, n, 0.1)
    with pytest.raises(ValueError, match="num_seqs \\+ 1"):
        _lib.pa_latent_decode(out, None, q, cache, t, n, 0.1, query_start_loc=i32(2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        _lib.pa_latent_decode(out, None, q, cache, t, n, 0.1)
    with pytest.raises(ValueError, match="out must be"):
        PagedLatentCache(4, 512, 64, 16, latent_cache=cache).attend(q, t, n, 0.1, out=z(2, 8, 500))


def test_prefill_shapes():
    q, k, v, kr, s = z(5, 2, 192), z(9, 2, 128), z(9, 2, 128), z(9, 64), i32(3)
    for bad, match in (((z(5, 2, 190), k, kr, v, s, s), "nope_dim"), ((q, z(9, 3, 128), kr, v, s, s), "same tokens"),
                       ((q, k, kr, z(8, 2, 128), s, s), "same tokens"), ((q, k, z(8, 64), v, s, s), "same tokens"),
                       ((q, k, kr, v, s, i32(4)), "num_seqs \\+ 1"), ((q, k, kr, v, s, s), "CUDA tensor"),
                       ((q[0], k, kr, v, s, s), "tokens, heads, dim")):
        with pytest.raises(ValueError, match=match):
            latent_prefill(*bad, 0.1, max_query_len=3)
    with pytest.raises(ValueError, match="out must be"):
        latent_prefill(q, k, kr, v, s, s, 0.1, max_query_len=3, out=z(5, 2, 64))
    with pytest.raises(ValueError, match="lse must be"):
        latent_prefill(q, k, kr, v, s, s, 0.1, max_query_len=3, lse=z(5, 3))


def test_table_shapes():
    with pytest.raises(ValueError, match="positive"):
        DeviceBlockTables(0, 4, 4, 16, device="cpu")
    with pytest.raises(ValueError, match="context_lens must be int32"):
        DeviceBlockTables(2, 4, 4, 16, device="cpu", context_lens=i32(3))
    with pytest.raises(ValueError, match="ref_counts must be int32"):
        DeviceBlockTables(2, 4, 4, 16, device="cpu", ref_counts=torch.zeros(4, dtype=torch.int64))
    tab = DeviceBlockTables(2, 4, 4, 16, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        tab.step(i32(2), 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tab.compact()


# ---- the library's own checks: nothing is launched, so any non-null address will do ----

BUF = ctypes.create_string_buffer(1 << 12)
A = (ctypes.addressof(BUF) + 255) // 256 * 256


def _write(t=1, ls=512, rs=64, r=512, d=64, bs=16, nb=4, dt=2, latent=A):
    return _lib.library().pa_latent_write(latent, A, A, A, t, ls, rs, r, d, bs, nb, dt, None)


def _decode(out=A, q=A + 16, s=1, tq=1, mq=1, h=16, r=512, d=64, bs=16, nb=4, scale=0.1, mbps=4, dt=2, qsl=None):
    return _lib.library().pa_latent_decode(out, None, q, A, A, mbps, A, qsl, s, tq, mq, h, r, d, bs, nb, scale, 0, dt,
                                           None, 0, None)


def _prefill(out=A, q=A + 16, k=A, ks=256, kh=128, krs=64, s=1, tq=1, tk=1, mq=1, h=2, dn=128, dr=64, dv=128, scale=0.1, dt=2):
    return _lib.library().pa_latent_prefill(out, None, q, k, A, A, ks, kh, krs, 256, 128, A, A, s, tq, tk, mq, h, dn, dr, dv,
                                            scale, 1, dt, None, 0, None)


def test_library_refuses_write():
    assert _write(t=0) == 0
    assert _write(t=-1) == INVALID and _write(nb=0) == INVALID and _write(latent=A + 8) == INVALID
    assert _write(ls=516) == INVALID and _write(rs=-64) == INVALID and _write(latent=None) == INVALID
    assert _write(r=384) == UNSUPPORTED and _write(d=32) == UNSUPPORTED and _write(bs=48) == UNSUPPORTED
    assert _write(dt=0) == UNSUPPORTED and _write(dt=3) == UNSUPPORTED and _write(dt=-1) == UNSUPPORTED


def test_library_refuses_decode():
    assert _decode(s=0, tq=0) == 0
    for bad in (dict(scale=float("nan")), dict(scale=-1.0), dict(scale=float("inf")), dict(h=0), dict(nb=0), dict(mbps=0),
                dict(tq=2), dict(out=None), dict(q=A), dict(q=A + 8), dict(s=-1), dict(mq=0, qsl=A)):
        assert _decode(**bad) == INVALID, bad
    for bad in (dict(r=128), dict(d=128), dict(bs=8), dict(dt=0), dict(dt=3), dict(mbps=1 << 27), dict(nb=1 << 28)):
        assert _decode(**bad) == UNSUPPORTED, bad


def test_library_refuses_prefill():
    assert _prefill(s=0) == 0 and _prefill(tq=0) == 0
    for bad in (dict(scale=float("nan")), dict(scale=-1.0), dict(h=0), dict(mq=0), dict(out=None), dict(q=A), dict(k=A + 2),
                dict(ks=100), dict(kh=0), dict(krs=-64), dict(k=None)):
        assert _prefill(**bad) == INVALID, bad
    for bad in (dict(dn=96, dv=96), dict(dv=64), dict(dr=32), dict(dt=0), dict(tq=1 << 20, h=1 << 11)):
        assert _prefill(**bad) == UNSUPPORTED, bad


def test_library_refuses_tables():
    lib = _lib.library()

    def step(s=1, w=4, nb=4, bs=16, new=1, pool=A, size=16, n=1, ws=A, ws_bytes=1 << 20, refs=A):
        ptrs, sizes = (ctypes.c_void_p * 1)(pool), (ctypes.c_int64 * 1)(size)
        return lib.pa_table_step(A, w, A, refs, None, None, A, s, nb, bs, A, new, A, A, ptrs, sizes, n, ws, ws_bytes, None)

    def compact(s=1, w=4, nb=4, bs=16, ws_bytes=1 << 20, live=A, n=0):
        return lib.pa_table_compact(A, w, A, A, s, nb, bs, live, A, None, None, n, A, ws_bytes, None)

    for bad in (dict(s=0), dict(w=0), dict(nb=0), dict(bs=0), dict(new=-1), dict(pool=A + 8), dict(size=24), dict(size=0),
                dict(pool=None), dict(refs=None), dict(n=-1), dict(n=1025)):
        assert step(**bad) == INVALID, bad
    assert step(s=4097) == UNSUPPORTED and step(w=1 << 26) == UNSUPPORTED
    assert step(ws=None) == WORKSPACE and step(ws_bytes=100) == WORKSPACE and step(ws=A + 8) == WORKSPACE
    for bad in (dict(s=0), dict(live=None), dict(n=2)):
        assert compact(**bad) == INVALID, bad
    assert compact(ws_bytes=64) == WORKSPACE and compact(w=1 << 26) == UNSUPPORTED
    assert _lib.pa_table_workspace_size(0, 4, 4) == 0 and _lib.pa_table_workspace_size(3, 4, 4) > 0
