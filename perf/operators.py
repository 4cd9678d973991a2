"""Cases of the latent cache's operators and of the device block tables'.

A latent cache holds one vector a token, shared by every head: ``latent_dim``
values that stand for keys and values both, and ``rope_dim`` values that carry
the position and enter the logits only.  The operators: writing new tokens
into it, attention over it in the absorbed form (queries brought into the
latent space; the form for single tokens and a few drafted ones) and in the
expanded form (keys and values of every head multiplied out; the form for
prompts), and the block tables kept on the device: growing, forking and
releasing rows in one step, and compacting the pool.

``run`` computes each in elementary torch operations where ``own`` is false
and through the framework's classes where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _ceil(a, b):
    return -(-a // b)


# ---- the cases -------------------------------------------------------------------


def listed():
    return [
        # one decode step's new tokens, one per sequence of a 256-sequence batch
        {"name": "write_step", "op": "write", "tokens": 256, "latent": 512, "rope": 64, "bs": 16,
         "dtype": "bf16", "pad": 7},
        # the tokens of a prefill batch, both parts slices of one projection's rows
        {"name": "write_prompts", "op": "write", "tokens": 16411, "latent": 512, "rope": 64, "bs": 64,
         "dtype": "f16", "pad": 0},
        # one user's next token over a short context: latency
        {"name": "decode_one", "op": "decode", "seqs": 1, "heads": 16, "latent": 512, "rope": 64, "bs": 16,
         "dtype": "bf16", "min_len": 901, "max_len": 901, "rows": 1, "shape": 1},
        # a serving batch on one rank of a head-parallel group: 256 sequences, ragged contexts
        {"name": "decode_serving", "op": "decode", "seqs": 256, "heads": 16, "latent": 512, "rope": 64,
         "bs": 16, "dtype": "bf16", "min_len": 1, "max_len": 4096, "rows": 1, "shape": 2},
        # all heads of a layer on one GPU, long contexts
        {"name": "decode_all_heads", "op": "decode", "seqs": 64, "heads": 128, "latent": 512, "rope": 64,
         "bs": 64, "dtype": "bf16", "min_len": 2048, "max_len": 8192, "rows": 1, "shape": 3},
        # drafted tokens attended together with the current one, long contexts, the small latent
        {"name": "decode_drafts", "op": "decode", "seqs": 12, "heads": 32, "latent": 256, "rope": 64,
         "bs": 32, "dtype": "f16", "min_len": 37, "max_len": 32768, "rows": 4, "shape": 4},
        # a batch of whole prompts, from one token up
        {"name": "prefill_prompts", "op": "prefill", "seqs": 9, "heads": 16, "nope": 128, "v": 128,
         "dtype": "bf16", "min_q": 1, "max_q": 2048, "prefix": 0, "shape": 5},
        # a chunk of a long prompt over its cached prefix
        {"name": "prefill_chunk", "op": "prefill", "seqs": 2, "heads": 16, "nope": 128, "v": 128,
         "dtype": "bf16", "min_q": 2048, "max_q": 2048, "prefix": 14337, "shape": 6},
        # a decode step's bookkeeping: every row grows by one token, a few rows end or fork
        {"name": "tables_step", "op": "step", "rows": 256, "width": 256, "blocks": 32768, "bs": 16,
         "max_len": 4000, "fan": 4, "release": 16, "fork": 16, "new": 1, "elems": 9216, "shape": 7},
        # admission: a quarter of a large batch ends and new prompts come in, the pool is large
        {"name": "tables_admit", "op": "step", "rows": 1024, "width": 1024, "blocks": 262144, "bs": 32,
         "max_len": 12000, "fan": 8, "release": 4, "fork": 8, "new": 2048, "elems": 2048, "shape": 8},
        # a small pool after a few requests have ended
        {"name": "compact_small", "op": "compact", "rows": 16, "width": 64, "blocks": 640, "bs": 16,
         "max_len": 1000, "fan": 2, "release": 3, "elems": 9216, "pools": 2, "shape": 9},
        # a large pool, half of whose rows have ended, key and value pools of one layer
        {"name": "compact_large", "op": "compact", "rows": 512, "width": 512, "blocks": 65536, "bs": 16,
         "max_len": 4096, "fan": 1, "release": 2, "elems": 16384, "pools": 2, "shape": 10},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "decode", "decode", "decode", "prefill", "prefill", "step", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    shape = rng.randrange(1 << 30)
    if op == "write":
        return {"op": op, "tokens": spread(1, 16000), "latent": rng.choice([512, 512, 256]), "rope": 64,
                "bs": rng.choice([16, 32, 64]), "dtype": dtype, "pad": rng.choice([0, 3, 11])}
    if op == "decode":
        heads = rng.choice([1, 5, 8, 16, 16, 32, 40, 64, 128])
        rows = rng.choice([1, 1, 1, 2, 3, 5])
        # at most the work of the largest listed case: 64 sequences x 128 heads x 4352 keys on average
        most = 64 * 128 * 4000
        max_len = spread(1, 60000)
        seqs = max(1, min(spread(1, 300), most // max(1, heads * rows * max_len), 600000 // max_len))
        return {"op": op, "seqs": seqs, "heads": heads, "latent": rng.choice([512, 512, 256]), "rope": 64,
                "bs": rng.choice([16, 32, 64]), "dtype": dtype, "min_len": rng.choice([0, 1, max_len // 2]),
                "max_len": max_len, "rows": rows, "shape": shape}
    if op == "prefill":
        heads = rng.choice([1, 4, 16, 16, 24])
        max_q = spread(1, 2048)
        prefix = rng.choice([0, 0, spread(1, 12000)])
        # the scores of the plain form stay below those of the largest listed case
        seqs = max(1, min(spread(1, 16), 2 * 16 * 2048 * 16385 // (heads * max_q * (max_q + prefix))))
        small = rng.random() < 0.3
        return {"op": op, "seqs": seqs, "heads": heads, "nope": 64 if small else 128, "v": 64 if small else 128,
                "dtype": dtype, "min_q": rng.choice([0, 1, max_q]), "max_q": max_q, "prefix": prefix,
                "shape": shape}
    bs = rng.choice([16, 32, 64])
    rows = spread(1, 1000)
    max_len = spread(1, 10000)
    width = _ceil(max_len, bs) + rng.choice([1, 7, 60])
    blocks = max(64, int(rows * width * rng.uniform(1.0, 1.6)))
    if op == "step":
        # a row grows within its table
        new = rng.choice([1, 1, spread(1, bs * (width - _ceil(max_len, bs)))])
        return {"op": op, "rows": rows, "width": width, "blocks": min(blocks, 250000), "bs": bs, "max_len": max_len,
                "fan": rng.choice([1, 2, 5]), "release": rng.choice([2, 5, 30]), "fork": rng.choice([2, 7, 30]),
                "new": new, "elems": 1024, "shape": shape}
    blocks = min(blocks, 60000)
    return {"op": op, "rows": rows, "width": width, "blocks": blocks, "bs": bs, "max_len": max_len,
            "fan": rng.choice([1, 3]), "release": rng.choice([2, 3, 9]), "elems": rng.choice([512, 4608, 16384]),
            "pools": rng.choice([1, 2, 3]), "shape": shape}


# ---- lengths: they follow from the case, values and places from the seed ---------------


def _lens(case):
    """Context lengths and query rows of a decode batch."""
    r = random.Random(case["shape"])
    lens, rows = [], []
    for i in range(case["seqs"]):
        lo, hi = case["min_len"], case["max_len"]
        if lo * 8 < hi:  # most contexts are short, a few long
            n = int(min(hi, max(lo, round(math.exp(math.log(max(hi / 5, 1)) + 0.8 * r.gauss(0, 1))))))
        else:
            n = r.randint(lo, hi)
        if i == 0:
            n = hi
        q = 1 if case["rows"] == 1 else r.randint(1, case["rows"])
        lens.append(max(n, q) if n else 0)
        rows.append(q)
    return lens, rows


def _prompts(case):
    """Query rows and keys of a prefill batch."""
    r = random.Random(case["shape"])
    qs = [r.randint(case["min_q"], case["max_q"]) for _ in range(case["seqs"])]
    qs[0] = case["max_q"]
    return qs, [q + (r.randint(case["prefix"] // 2, case["prefix"]) if i else case["prefix"])
                for i, q in enumerate(qs)]


def _visible(q, k):
    """Pairs that a causal mask of q rows over k >= q keys leaves."""
    return q * (k - q) + q * (q + 1) // 2


def _table_rows(case):
    """Rows of the tables: lengths, and the row whose leading blocks each shares (itself for none)."""
    r = random.Random(case["shape"])
    n, fan = case["rows"], case["fan"]
    lens = [r.randint(0, case["max_len"]) for _ in range(n)]
    base = [i - i % fan for i in range(n)]
    shared = []
    for i in range(n):
        if base[i] == i:
            shared.append(0)
            continue
        # every other fork still holds all of its parent's blocks, the rest have grown past some of them
        whole = i % 2 == 1
        lens[i] = lens[base[i]] if whole else lens[i]
        shared.append(_ceil(lens[i], case["bs"]) if whole else min(lens[i], lens[base[i]]) // case["bs"])
    return lens, base, shared


def _fits(case):
    """The rows that the pool has room for (the others are empty), with their blocks."""
    lens, base, shared = _table_rows(case)
    left = int(case["blocks"] * 0.9)
    for i, n in enumerate(lens):
        if base[i] != i and lens[base[i]] == 0:
            lens[i], shared[i] = 0, 0
        need = _ceil(lens[i], case["bs"]) - shared[i]
        if need > left:
            lens[i], shared[i], need = 0, 0, 0
        left -= need
    return lens, base, shared


# ---- inputs -------------------------------------------------------------------------


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed * 2654435761 % (1 << 62))
    return {"write": _prepare_write, "decode": _prepare_decode, "prefill": _prepare_prefill,
            "step": _prepare_tables, "compact": _prepare_tables}[case["op"]](case, g, seed)


def _prepare_write(case, g, seed):
    t, r, d = case["tokens"], case["latent"], case["rope"]
    dtype = DTYPES[case["dtype"]]
    nb = _ceil(t, case["bs"]) * 5 // 4 + 1
    both = _normal(g, (t, r + d), dtype)  # one projection's output rows
    slots = torch.randperm(nb * case["bs"], generator=g, device=DEV)[:t]
    if case["pad"]:
        slots[:: case["pad"]] = -1  # padding tokens
    cache = torch.zeros((nb, case["bs"], r + d), dtype=dtype, device=DEV)
    st = {"op": "write", "latent": both[:, :r], "rope": both[:, r:], "slots": slots, "cache": cache}
    if own:
        from paged_kv_cache_388_b200.latent import PagedLatentCache
        st["user"] = PagedLatentCache(nb, r, d, case["bs"], latent_cache=cache)
    return st


def _prepare_decode(case, g, seed):
    lens, rows = _lens(case)
    r, d, bs, h = case["latent"], case["rope"], case["bs"], case["heads"]
    dtype = DTYPES[case["dtype"]]
    blocks = [_ceil(n, bs) for n in lens]
    width = max(1, max(blocks))
    nb = sum(blocks) * 5 // 4 + 1
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    n_blocks = torch.tensor(blocks, device=DEV)
    place = torch.arange(width, device=DEV)[None] < n_blocks[:, None]
    tables = torch.zeros((len(lens), width), dtype=torch.int32, device=DEV)
    tables[place] = perm[: sum(blocks)]
    cache = torch.empty((nb, bs, r + d), dtype=dtype, device=DEV)
    for i in range(0, nb, 8192):  # in slabs, for the sake of the 32-bit copy
        cache[i:i + 8192] = _normal(g, (min(8192, nb - i), bs, r + d), dtype)
    q = _normal(g, (sum(rows), h, r + d), dtype)
    qsl = None
    if case["rows"] > 1:
        qsl = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32, device=DEV)
    # queries of a trained layer spread the logits over a few units
    st = {"op": "decode", "q": q, "cache": cache, "tables": tables, "bs": bs, "latent": r,
          "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "qsl": qsl, "rows": case["rows"],
          "max_len": max(1, max(lens)), "scale": 1.0 / math.sqrt(192.0), "lse": case["rows"] > 1}
    if own:
        from paged_kv_cache_388_b200.latent import PagedLatentCache
        st["user"] = PagedLatentCache(nb, r, d, bs, latent_cache=cache)
    return st


def _prepare_prefill(case, g, seed):
    qs, ks = _prompts(case)
    h, dn, dv, dr = case["heads"], case["nope"], case["v"], 64
    dtype = DTYPES[case["dtype"]]
    tq, tk = sum(qs), sum(ks)
    kv = _normal(g, (tk, h, dn + dv), dtype)  # keys and values of a token side by side, as one projection leaves them
    return {"op": "prefill", "q": _normal(g, (tq, h, dn + dr), dtype), "k": kv[:, :, :dn], "v": kv[:, :, dn:],
            "k_rope": _normal(g, (tk, dr), dtype),
            "qsl": torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device=DEV),
            "ksl": torch.tensor([0] + list(np.cumsum(ks)), dtype=torch.int32, device=DEV),
            "max_q": max(1, max(qs)), "max_k": max(1, max(ks)), "scale": 1.0 / math.sqrt(dn + dr)}


def _prepare_tables(case, g, seed):
    lens, base, shared = _fits(case)
    n, w, nb, bs = case["rows"], case["width"], case["blocks"], case["bs"]
    perm = np.random.RandomState(seed % (1 << 32)).permutation(nb).astype(np.int32)
    tables = np.zeros((n, w), np.int32)
    at = 0
    for i in range(n):
        s, b = shared[i], _ceil(lens[i], bs)
        tables[i, :s] = tables[base[i], :s]
        tables[i, s:b] = perm[at:at + b - s]
        at += b - s
    lens = np.asarray(lens, np.int32)
    held = np.arange(w)[None] < -(-lens[:, None] // bs)
    r = random.Random(case["shape"] + 1)
    release = np.asarray([i % case["release"] == case["release"] - 1 for i in range(n)], np.int32)
    if case["op"] == "compact":  # the rows that have ended give up their blocks before
        held &= release[:, None] == 0
        lens = np.where(release, 0, lens).astype(np.int32)
    refs = np.bincount(tables[held], minlength=nb).astype(np.int32)
    st = {"op": case["op"], "bs": bs, "tables0": torch.from_numpy(tables).to(DEV),
          "lens0": torch.from_numpy(lens).to(DEV), "refs0": torch.from_numpy(refs).to(DEV),
          "tables": torch.zeros((n, w), dtype=torch.int32, device=DEV),
          "lens": torch.zeros(n, dtype=torch.int32, device=DEV),
          "refs": torch.zeros(nb, dtype=torch.int32, device=DEV)}
    pools = [torch.empty((nb, case["elems"]), dtype=torch.bfloat16, device=DEV) for _ in range(case.get("pools", 1))]
    for p in pools:
        for i in range(0, nb, 16384):
            p[i:i + 16384] = _normal(g, (min(16384, nb - i), case["elems"]), torch.bfloat16)
    st["pools"] = pools
    if case["op"] == "step":
        fork = np.full(n, -1, np.int32)
        for i in range(case["fork"] - 2, n, case["fork"]):
            if i >= 0:
                fork[i] = r.randrange(n)
        after = np.where(fork >= 0, lens[np.maximum(fork, 0)], np.where(release, 0, lens))
        append = np.asarray([min(case["new"] if case["new"] == 1 else r.randint(0, case["new"]), w * bs - int(a))
                             for a in after], np.int32)
        st |= {"release": torch.from_numpy(release).to(DEV), "fork": torch.from_numpy(fork).to(DEV),
               "append": torch.from_numpy(append).to(DEV), "max_new": int(append.sum()) + 5}
    if own:
        from paged_kv_cache_388_b200.tables import DeviceBlockTables
        st["user"] = DeviceBlockTables(n, w, nb, bs, block_tables=st["tables"], context_lens=st["lens"],
                                       ref_counts=st["refs"])
    return st


# ---- one pass ------------------------------------------------------------------------


def run(st):
    return {"write": _run_write, "decode": _run_decode, "prefill": _run_prefill, "step": _run_step,
            "compact": _run_compact}[st["op"]](st)


def _run_write(st):
    if own:
        st["user"].write(st["latent"], st["rope"], st["slots"])
        return st["cache"]
    keep = st["slots"] >= 0
    rows = torch.cat([st["latent"], st["rope"]], 1)
    st["cache"].view(-1, rows.shape[1])[st["slots"][keep]] = rows[keep]
    return st["cache"]


def _softmax_times(s, seen, values):
    """Softmax over the last axis where `seen`, times values; zeros and -inf where a row sees nothing."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = values(e) / torch.where(total > 0, total, 1.0)
    return o, (torch.log(total) + m).squeeze(-1)


def _run_decode(st):
    q, r = st["q"], st["latent"]
    if own:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV) if st["lse"] else None
        out = st["user"].attend(q, st["tables"], st["lens"], st["scale"], lse=lse, query_start_loc=st["qsl"],
                                max_query_len=st["rows"], max_context_len=st["max_len"])
        return {"out": out, "lse": lse} if st["lse"] else out
    n = st["lens"].shape[0]
    qsl = st["qsl"] if st["qsl"] is not None else torch.arange(n + 1, device=DEV, dtype=torch.int32)
    at = torch.arange(st["max_len"], device=DEV)
    slots = st["tables"][:, at // st["bs"]].long() * st["bs"] + at % st["bs"]
    c = st["cache"].view(-1, q.shape[2])[slots].float()  # [seqs, keys, latent + rope]
    c = c * (at[None] < st["lens"][:, None])[..., None]
    t = torch.arange(st["rows"], device=DEV)
    count = qsl[1:] - qsl[:-1]
    real = t[None] < count[:, None]
    row = (qsl[:-1, None] + t).clamp(max=q.shape[0] - 1)
    s = torch.einsum("sthd,skd->sthk", q[row].float(), c) * st["scale"]
    last = st["lens"][:, None] - count[:, None] + t
    seen = (at <= last[..., None])[:, :, None, :].expand_as(s)
    o, lse = _softmax_times(s, seen, lambda e: torch.einsum("sthk,skd->sthd", e, c[..., :r]))
    out = torch.zeros((*q.shape[:2], r), dtype=q.dtype, device=DEV)
    out[row[real]] = o[real].to(q.dtype)
    if not st["lse"]:
        return out
    all_lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    all_lse[row[real]] = lse[real]
    return {"out": out, "lse": all_lse}


def _run_prefill(st):
    q, k, v, kr = st["q"], st["k"], st["v"], st["k_rope"]
    qsl, ksl = st["qsl"], st["ksl"]
    if own:
        from paged_kv_cache_388_b200.latent import latent_prefill
        return latent_prefill(q, k, kr, v, qsl, ksl, st["scale"], max_query_len=st["max_q"])
    t, j = torch.arange(st["max_q"], device=DEV), torch.arange(st["max_k"], device=DEV)
    nq, nk = qsl[1:] - qsl[:-1], ksl[1:] - ksl[:-1]
    real = t[None] < nq[:, None]
    row = (qsl[:-1, None] + t).clamp(max=q.shape[0] - 1)
    key = (ksl[:-1, None] + j).clamp(max=k.shape[0] - 1)
    qf, dn = q[row].float(), k.shape[2]
    s = torch.einsum("sthd,skhd->shtk", qf[..., :dn], k[key].float())
    s += torch.einsum("sthd,skd->shtk", qf[..., dn:], kr[key].float())
    s *= st["scale"]
    seen = (j <= (nk - nq)[:, None, None] + t[:, None])[:, None].expand_as(s)
    o, _ = _softmax_times(s, seen, lambda e: torch.einsum("shtk,skhd->shtd", e, v[key].float()))
    out = torch.zeros((*q.shape[:2], v.shape[2]), dtype=q.dtype, device=DEV)
    out[row[real]] = o.transpose(1, 2)[real].to(q.dtype)
    return out


def _restore(st):
    """The tables as they stood before the step, so that a pass can be repeated (the pools keep:
    a copied block's source stays what it was)."""
    st["tables"].copy_(st["tables0"])
    st["lens"].copy_(st["lens0"])
    st["refs"].copy_(st["refs0"])


def _run_step(st):
    _restore(st)
    tables, lens, refs, bs = st["tables"], st["lens"], st["refs"], st["bs"]
    if own:
        slots, qsl, copies = st["user"].step(st["append"], st["max_new"], release=st["release"],
                                             fork_src=st["fork"], pools=st["pools"])
        return [tables, lens, refs, slots, qsl, copies, st["pools"]]
    n, w = tables.shape
    i, j = torch.arange(n, device=DEV), torch.arange(w, device=DEV)
    # blocks that rows give up, and that forks come to hold
    held = j < (-(-lens // bs))[:, None]
    forked = st["fork"] >= 0
    gone = (forked | (st["release"] != 0))[:, None] & held
    src = torch.where(forked, st["fork"].long(), i)
    taken = forked[:, None] & held[src]
    old = tables[src]
    refs.index_add_(0, torch.where(gone, tables, 0).flatten(), -gone.flatten().int())
    refs.index_add_(0, torch.where(taken, old, 0).flatten(), taken.flatten().int())
    tables.copy_(torch.where(taken, old, tables))
    now = torch.where(forked, lens[src], torch.where(st["release"] != 0, 0, lens)).long()
    # blocks that the new tokens need: a shared last block is copied by all of its writers but the last holder
    add = st["append"].long()
    blocks = -(-now // bs)
    last = tables[i, (blocks - 1).clamp(min=0)].long()
    shared = (add > 0) & (now % bs != 0) & (refs[last] > 1)
    before = ((last[:, None] == last[None]) & shared[:, None] & shared[None]).tril(-1).sum(1)
    cow = shared & (refs[last] - before > 1)
    more = -(-(now + add) // bs) - blocks
    need = more + cow
    end = need.cumsum(0)
    fits = end <= (refs == 0).sum()
    cow, more, add_now = cow & fits, torch.where(fits, more, 0), torch.where(fits, add, 0)
    free = torch.nonzero(refs == 0).squeeze(1)
    free = torch.cat([free, free.new_zeros(1)])
    first = (end - need).clamp(max=free.shape[0] - 1)
    refs.index_add_(0, last, -cow.int())
    grown = (j >= blocks[:, None]) & (j < (blocks + more)[:, None])
    fresh = free[(first[:, None] + cow[:, None] + j - blocks[:, None]).clamp(0, free.shape[0] - 1)].int()
    fresh = torch.where(grown, fresh, tables)
    fresh = torch.where(cow[:, None] & (j == blocks[:, None] - 1), free[first].int()[:, None], fresh)
    tables.copy_(fresh)
    total = (more + cow).sum()
    refs.masked_fill_((refs == 0) & ((refs == 0).cumsum(0) <= total), 1)
    lens.copy_(now + add_now)
    # slots of the new tokens, one after the other by rows
    qsl = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    qsl[1:] = add.cumsum(0)
    p = torch.arange(st["max_new"], device=DEV)
    of = (torch.searchsorted(qsl[1:].long(), p, right=True)).clamp(max=n - 1)
    pos = now[of] + p - qsl[of]
    slots = tables[of, (pos // bs).clamp(max=w - 1)].long() * bs + pos % bs
    slots = torch.where((p < qsl[-1]) & fits[of], slots, -1)
    copies = torch.where(cow[:, None], torch.stack([last, free[first]], 1), -1)
    for pool in st["pools"]:
        pool[copies[cow][:, 1]] = pool[copies[cow][:, 0]]
    return [tables, lens, refs, slots, qsl, copies, st["pools"]]


def _run_compact(st):
    _restore(st)
    tables, refs = st["tables"], st["refs"]
    if own:
        live, moves = st["user"].compact(pools=st["pools"])
        return [tables, refs, live, moves, st["pools"]]
    nb = refs.shape[0]
    ids = torch.arange(nb, device=DEV)
    used = refs > 0
    live = used.sum()
    source = ids[used & (ids >= live)]
    hole = ids[~used & (ids < live)]
    to = ids.clone()
    to[source] = hole
    held = torch.arange(tables.shape[1], device=DEV) < (-(-st["lens"] // st["bs"]))[:, None]
    tables.copy_(torch.where(held, to[tables].int(), tables))
    refs[hole] = refs[source]
    refs[source] = 0
    for pool in st["pools"]:
        pool[hole] = pool[source]
    moves = torch.full((max(1, nb // 2), 2), -1, dtype=torch.int64, device=DEV)
    moves[: source.shape[0], 0] = source
    moves[: source.shape[0], 1] = hole
    return [tables, refs, live.int().reshape(1), moves, st["pools"]]


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "write":
        kept = case["tokens"] - (_ceil(case["tokens"], case["pad"]) if case["pad"] else 0)
        return {"bytes": kept * 2 * (case["latent"] + case["rope"]) * 2 + 8 * case["tokens"], "flops": 0}
    if op == "decode":
        lens, rows = _lens(case)
        r, d, h = case["latent"], case["rope"], case["heads"]
        pairs = sum(_visible(q, n) for n, q in zip(lens, rows) if n)
        data = sum(lens) * (r + d) * 2 + sum(rows) * h * (2 * r + d) * 2
        data += 4 * sum(_ceil(n, case["bs"]) for n in lens) + 8 * len(lens)
        return {"bytes": data, "flops": 2 * pairs * h * (2 * r + d)}
    if op == "prefill":
        qs, ks = _prompts(case)
        h, dn, dv = case["heads"], case["nope"], case["v"]
        pairs = sum(_visible(q, k) for q, k in zip(qs, ks))
        return {"bytes": 2 * (sum(qs) * h * (dn + 64 + dv) + sum(ks) * (h * (dn + dv) + 64)),
                "flops": 2 * pairs * h * (dn + 64 + dv)}
    lens, base, shared = _fits(case)
    n, bs, nb = case["rows"], case["bs"], case["blocks"]
    if op == "step":
        # the counts once, the rows' entries that change, lengths, new slots
        return {"bytes": 4 * nb + 28 * n + 12 * n * max(1, case["new"] // 2), "flops": 0}
    kept = [0 if i % case["release"] == case["release"] - 1 else _ceil(x, bs) for i, x in enumerate(lens)]
    live = sum(kept)
    moved = live * max(0, nb - live) // nb  # used blocks beyond the live count, spread evenly
    return {"bytes": 8 * nb + 8 * live + 2 * moved * case["elems"] * 2 * case["pools"], "flops": 0}


# ---- the definitions in 64 bits -------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "decode":
        return _exact_decode(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(case, seed)
    return None  # bytes and whole numbers


def _attend64(q, k, v, limits, scale):
    """Rows q [t, h, d] over keys k [h or 1, n, d]; row t sees the first limits[t] keys."""
    n = k.shape[1]
    if n == 0:
        return (torch.zeros((*q.shape[:2], v.shape[2]), dtype=torch.float64, device=DEV),
                torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV))
    s = scale * torch.matmul(q.transpose(0, 1), k.transpose(1, 2))
    hidden = torch.arange(n, device=DEV)[None] >= limits[:, None]
    s[:, hidden] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.nan_to_num(torch.exp(s - lse[..., None]), nan=0.0)
    return torch.matmul(p, v).transpose(0, 1), lse.transpose(0, 1)


def _exact_decode(case, seed):
    st = _prepare_decode(case, torch.Generator(DEV).manual_seed(seed * 2654435761 % (1 << 62)), seed)
    lens, rows = _lens(case)
    outs, lses, at = [], [], 0
    for i, (n, q) in enumerate(zip(lens, rows)):
        c = st["cache"][st["tables"][i, : _ceil(n, case["bs"])].long()].reshape(-1, st["q"].shape[2])[:n].double()
        limits = torch.arange(n - q + 1, n + 1, device=DEV)
        o, lse = _attend64(st["q"][at:at + q].double(), c[None], c[None, :, : case["latent"]], limits, st["scale"])
        outs.append(o)
        lses.append(lse)
        at += q
    out = torch.cat(outs)
    return {"out": out, "lse": torch.cat(lses)} if st["lse"] else out


def _exact_prefill(case, seed):
    st = _prepare_prefill(case, torch.Generator(DEV).manual_seed(seed * 2654435761 % (1 << 62)), seed)
    qs, ks = _prompts(case)
    outs, a, b = [], 0, 0
    for q, n in zip(qs, ks):
        kr = st["k_rope"][b:b + n].double()
        heads = []
        for h in range(case["heads"]):
            k = torch.cat([st["k"][b:b + n, h].double(), kr], 1)
            o, _ = _attend64(st["q"][a:a + q, h:h + 1].double(), k[None], st["v"][b:b + n, h].double()[None],
                             torch.arange(n - q + 1, n + 1, device=DEV), st["scale"])
            heads.append(o)
        outs.append(torch.cat(heads, 1))
        a, b = a + q, b + n
    return torch.cat(outs)
