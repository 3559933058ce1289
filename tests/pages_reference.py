"""Plain host implementations of the page operators and of the grouping rule
of attn_shared_plan, from their definitions in include/kvpaged.h (lists and
loops; no code of the library).  Test infrastructure."""
from __future__ import annotations


def ceil(a, b):
    return -(-a // b)


def _len(c, cap):
    return c if 0 <= c <= cap else 0


def fork(tables, lens, counts, parents, bs):
    """-> (tables, lens, counts, copies [(src, dst, tokens)], bad)."""
    width, nb = len(tables[0]) if tables else 0, len(counts)
    bad = False
    cap = width * bs
    counts = list(counts)
    pages = []
    for row, c in zip(tables, lens):
        n = _len(c, cap)
        bad |= n != c
        row = list(row[:ceil(n, bs)])
        for e in row:
            if 0 <= e < nb:
                counts[e] -= 1
            else:
                bad = True
        pages.append((n, [e if 0 <= e < nb else -1 for e in row]))
    new, kept, waiting = [], set(), []
    for r, p in enumerate(parents):
        if not -1 <= p < len(tables):
            bad, p = True, -1
        n, row = pages[p] if p >= 0 else (0, [])
        row = list(row)
        last_open = n % bs != 0
        for j, e in enumerate(row):
            if e < 0:
                continue
            if last_open and j == len(row) - 1:
                if e in kept:
                    waiting.append(r)
                    continue
                kept.add(e)
            counts[e] += 1
        new.append([n, row])
    free = [p for p in range(nb) if counts[p] == 0]
    copies = []
    for k, r in enumerate(waiting):
        n, row = new[r]
        if k < len(free):
            copies.append((row[-1], free[k], n % bs))
            row[-1] = free[k]
            counts[free[k]] = 1
        else:
            bad = True
            for e in row[:-1]:
                if e >= 0:
                    counts[e] -= 1
            new[r] = [0, []]
    out = [row + [-1] * (width - len(row)) for _, row in new]
    return out, [n for n, _ in new], counts, copies, bad


def extend(tables, lens, counts, new_tokens, bs, num_slots):
    """-> (tables, lens, counts, slots, bad)."""
    width, nb = len(tables[0]) if tables else 0, len(counts)
    cap = width * bs
    out_counts = list(counts)
    free = [p for p in range(nb) if counts[p] == 0]
    taken = 0
    out, out_lens, slots, bad = [], [], [], False
    for row, c, add in zip(tables, lens, new_tokens):
        n = _len(c, cap)
        ok = n == c
        if add < 0 or n + add > cap:
            ok, add = False, 0
        asked = add
        if ok and add > 0 and n % bs:
            e = row[ceil(n, bs) - 1]
            ok = 0 <= e < nb and counts[e] <= 1
        if not ok:
            bad, add = True, 0
        had, need = ceil(n, bs), ceil(n + add, bs) - ceil(n, bs)
        row = list(row[:had])
        if need and taken + need > len(free):
            bad = True
            slots += [-1] * asked
            taken += need  # later rows that need pages fail too
        elif add == 0:
            slots += [-1] * asked
        else:
            got = free[taken:taken + need]
            taken += need
            row += got
            for p in got:
                out_counts[p] = 1
            slots += [row[p // bs] * bs + p % bs for p in range(n, n + add)]
            n += add
        out.append(row + [-1] * (width - len(row)))
        out_lens.append(n)
    bad |= len(slots) > num_slots
    slots = (slots + [-1] * num_slots)[:num_slots]
    return out, out_lens, out_counts, slots, bad


def compact(tables, lens, counts, bs):
    """-> (tables, counts, places, moves [(src, dst)], bad)."""
    width, nb = len(tables[0]) if tables else 0, len(counts)
    live = [p for p in range(nb) if counts[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if counts[p] <= 0]
    moves = list(zip([p for p in live if p >= n], holes))
    places = [p if counts[p] > 0 else -1 for p in range(nb)]
    for s, d in moves:
        places[s] = d
    out_counts = [0] * nb
    for p in live:
        out_counts[places[p]] = counts[p]
    bad, out = False, []
    for row, c in zip(tables, lens):
        m = _len(c, width * bs)
        bad |= m != c
        new = [places[e] if 0 <= e < nb else -1 for e in row[:ceil(m, bs)]]
        bad |= any(e < 0 for e in new)
        out.append(new + [-1] * (width - len(new)))
    return out, out_counts, places, moves, bad


def shared_prefixes(tables, lens, bs, min_shared=128):
    """Keys that each sequence reads with its group."""
    n = len(tables)
    same = [0] * (n + 1)
    for b in range(1, n):
        most = (min(lens[b - 1], lens[b]) - 1) // bs if lens[b - 1] > 0 and lens[b] > 0 else 0
        while same[b] < most and tables[b][same[b]] == tables[b - 1][same[b]]:
            same[b] += 1
    joined = [b > 0 and same[b] > 0 and same[b] * bs >= min_shared and
              2 * same[b] >= max(same[b - 1], same[b + 1]) for b in range(n)]
    prefix = [0] * n
    b = 0
    while b < n:
        e = b + 1
        while e < n and joined[e]:
            e += 1
        if e - b > 1:
            prefix[b:e] = [min(same[b + 1:e]) * bs] * (e - b)
        b = e
    return prefix
