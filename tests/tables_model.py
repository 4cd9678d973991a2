"""A sequential restatement of the device block tables, one row and one block at
a time: what the GPU tests compare with."""


def step(tables, lens, refs, append, bs, max_new, release=None, fork=None):
    """Lists in, changed in place; returns slots, query_start_loc, copy pairs, whether the pool ran out."""
    n, width = len(tables), len(tables[0])
    blocks = lambda x: -(-x // bs)  # noqa: E731
    was = [(list(t), x) for t, x in zip(tables, lens)]
    for i in range(n):
        forked = fork is not None and 0 <= fork[i] < n
        if forked or (release is not None and release[i]):
            for b in was[i][0][: blocks(was[i][1])]:
                refs[b] -= 1
            lens[i] = 0
    for i in range(n):
        if fork is not None and 0 <= fork[i] < n:
            src, length = was[fork[i]]
            tables[i][: blocks(length)] = src[: blocks(length)]
            lens[i] = length
            for b in src[: blocks(length)]:
                refs[b] += 1
    slots, starts, pairs, out = [], [0], [], False
    for i in range(n):
        now, add = lens[i], append[i]
        starts.append(starts[-1] + max(add, 0))
        pair = (-1, -1)
        grows = 0 <= add and now + add <= width * bs
        need, copies = 0, False
        if grows and add:
            need = blocks(now + add) - blocks(now)
            copies = now % bs != 0 and refs[tables[i][blocks(now) - 1]] > 1
        free = [b for b, c in enumerate(refs) if c == 0]
        if out or need + copies > len(free):
            out, grows = True, False
        if grows:
            if copies:
                old, fresh = tables[i][blocks(now) - 1], free.pop(0)
                refs[old] -= 1
                refs[fresh] = 1
                tables[i][blocks(now) - 1] = fresh
                pair = (old, fresh)
            for k in range(need):
                fresh = free.pop(0)
                refs[fresh] = 1
                tables[i][blocks(now) + k] = fresh
            lens[i] = now + add
            slots += [tables[i][p // bs] * bs + p % bs for p in range(now, now + add)]
        else:
            slots += [-1] * max(add, 0)
        pairs.append(pair)
    slots = (slots + [-1] * max_new)[:max_new]
    return slots, starts, pairs, out


def compact(tables, lens, refs, bs):
    live = sum(c > 0 for c in refs)
    source = [b for b, c in enumerate(refs) if c > 0 and b >= live]
    hole = [b for b, c in enumerate(refs) if c <= 0 and b < live]
    to = dict(zip(source, hole))
    for t, n in zip(tables, lens):
        for j in range(-(-n // bs)):
            t[j] = to.get(t[j], t[j])
    for s, h in to.items():
        refs[h], refs[s] = refs[s], 0
    return live, list(to.items())
