"""One step's page bookkeeping and the packing of a pool, one sequence and one page at a time on Python lists: the definition
of include/fox.h, for the tests. No code of the library."""


def pages_of(tokens, S):
    return -(-max(tokens, 0) // S)


def step(refs, lens, table, parent, add, S, prefix, out_rows):
    """-> (refs, lens, table rows {(b, entry): page}, copies, whether the pages or a row did not reach)."""
    refs, stride = list(refs), len(table[0]) if table else 0
    children = [0] * len(lens)
    for p in parent:
        if p >= 0:
            children[p] += 1
    own = [n - prefix if n else 0 for n in lens]
    for b, t in enumerate(table):
        for c in range(pages_of(own[b], S)):
            refs[t[c]] += children[b] - 1
    new_lens, rows, copies, short = [], {}, [], False
    wants, holders = [], {}
    for b, (p, n) in enumerate(zip(parent, add)):
        length = lens[p] if p >= 0 else 0
        have = length - prefix if length else 0
        held = table[p][: pages_of(have, S)] if p >= 0 else []
        fits = n > 0 and have + n <= stride * S
        short |= n > 0 and not fits
        copy = False
        if fits and have % S:
            last = held[-1]
            copy = refs[last] - holders.get(last, 0) > 1
            holders[last] = holders.get(last, 0) + 1
        wants.append((length, have, held, fits, copy, pages_of(have + n, S) - len(held) + copy if fits else 0))
    free = [i for i, r in enumerate(refs) if r <= 0]
    taken = 0
    for b, (length, have, held, fits, copy, need) in enumerate(wants):
        mine = free[taken : taken + need]
        taken += need
        served = fits and (need == 0 or taken <= len(free))
        short |= fits and not served
        copies.append((-1, -1))
        if not served:
            new_lens.append(length)
        else:
            new_lens.append((length or prefix) + add[b])
            for i in mine:
                refs[i] = 1
            held = list(held)
            if copy:
                copies[-1] = (held[-1], mine[0])
                refs[held[-1]] -= 1
                held[-1] = mine[0]
                mine = mine[1:]
            held += mine
        for c, page in enumerate(held):
            rows[b, c] = page
    assert len(new_lens) == out_rows
    return refs, new_lens, rows, copies, short


def compact(refs, lens, table, prefix_table, S, prefix, max_moves):
    """-> (refs, table rows {(b, entry): page}, prefix table, map, moves, used)."""
    refs = list(refs)
    used = sum(r > 0 for r in refs)
    source = [i for i in range(len(refs) - 1, used - 1, -1) if refs[i] > 0]
    free = [i for i in range(used) if refs[i] <= 0]
    assert len(source) == len(free)
    moves = list(zip(source, free))[:max_moves]
    new = list(range(len(refs)))
    for x, y in moves:
        new[x] = y
        refs[y], refs[x] = refs[x], 0
    rows = {(b, c): new[table[b][c]] for b, n in enumerate(lens) if n for c in range(pages_of(n - prefix, S))}
    top = max([i + 1 for i, r in enumerate(refs) if r > 0], default=0)
    return refs, rows, [new[x] for x in prefix_table], new, moves, (used, top)
