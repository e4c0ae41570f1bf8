"""The page operators in plain Python, on lists: for tests."""
BLOCK = 16


def pages_of(tokens, page):
    return -(-tokens // page)


def grow(refs, lens, table, counts, page):
    """Returns (ok, refs, lens, table)."""
    refs, lens, table, before = list(refs), list(lens), [list(r) for r in table], list(refs)
    free = [p for p, n in enumerate(refs) if n == 0]
    cols, upto, ok = len(table[0]), 0, []
    for s, n in enumerate(counts):
        old, new = lens[s], max(lens[s] + n, 0)
        have, want = pages_of(old, page), pages_of(new, page)
        good = True
        if n > 0:
            good = want <= cols and new < 2 ** 31
            if good:
                need = want - have
                if need and upto + need > len(free):
                    good = False
                else:
                    for i in range(need):
                        table[s][have + i] = free[upto + i]
                        refs[free[upto + i]] = 1
                upto += need
        elif n < 0:
            good = not (new % page and before[table[s][want - 1]] > 1)
            if good:
                for c in range(want, have):
                    refs[table[s][c]] -= 1
        if good:
            lens[s] = new
        ok.append(good)
    return ok, refs, lens, table


def fork(refs, lens, table, parents, page):
    """Returns (ok, refs, lens, table, copies): copies are (from page, to page, tokens)."""
    S, free = len(lens), [p for p, n in enumerate(refs) if n == 0]
    keeper = {}
    for s, p in enumerate(parents):
        if 0 <= p < S:
            keeper[p] = p if parents[p] == p else keeper.get(p, s)
    new_lens, new_table, ok, copies, taken = [], [list(r) for r in table], [], [], 0
    for s, p in enumerate(parents):
        good, n = True, 0
        if p >= S:
            good = False
        elif p >= 0:
            n = lens[p]
            row = list(table[p][:pages_of(n, page)])
            if n % page and keeper[p] != s:
                if taken < len(free):
                    copies.append((row[-1], free[taken], n % page))
                    row[-1] = free[taken]
                else:
                    good, n, row = False, 0, []
                taken += 1
            new_table[s][:len(row)] = row
        new_lens.append(n)
        ok.append(good)
    refs = list(refs)
    for s in range(S):
        for p in table[s][:pages_of(lens[s], page)]:
            refs[p] -= 1
        for p in new_table[s][:pages_of(new_lens[s], page)]:
            refs[p] += 1
    return ok, refs, new_lens, new_table, copies


def compact(refs, lens, table, page, room):
    """Returns (refs, lens, table, pages): pages[i] is the page that becomes page i."""
    used = [p for p, n in enumerate(refs) if n > 0]
    place = {p: i for i, p in enumerate(used)}
    out = [refs[p] for p in used[:room]] + [0] * (room - len(used))
    new_lens, new_table = [], []
    for n, row in zip(lens, table):
        to = [place[p] for p in row[:pages_of(n, page)]]
        fits = all(t < room for t in to)
        if not fits:
            for t in to:
                if t < room:
                    out[t] -= 1
        new_lens.append(n if fits else 0)
        new_table.append((to if fits else []) + [0] * (len(row) - (len(to) if fits else 0)))
    return out, new_lens, new_table, used[:room]
