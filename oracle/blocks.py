"""The states of a paged cache's blocks, one request and one block at a time.

TEST INFRASTRUCTURE ONLY, as the rest of the oracle.  A state is (rows, lens,
refs): each request's list of blocks, its number of tokens, and how many rows
hold each block.  ``contents`` are lists, one entry per block, copied with it.
"""
BLOCK = 128


def held(table, lens):
    """The rows' blocks, from a block table."""
    return [list(map(int, row[:-(-int(n) // BLOCK)])) for row, n in zip(table, lens)]


def fork(rows, lens, refs, parent, new_tokens, contents, max_blocks):
    """The state after the call, and whether blocks ran out; entries without a
    block are -1."""
    refs = list(refs)
    for row in rows:
        for b in row:
            refs[b] -= 1
    new_rows, new_lens, claimed, copies = [], [], set(), []
    for r, (p, more) in enumerate(zip(parent, new_tokens)):
        n = lens[p] if p >= 0 else 0
        row = [] if p < 0 else list(rows[p])
        if n % BLOCK:
            if p in claimed:
                copies.append((r, len(row) - 1, row[-1]))
                row[-1] = None
            claimed.add(p)
        n = min(n + more, max_blocks * BLOCK)
        row += [None] * (-(-n // BLOCK) - len(row))
        for b in row:
            if b is not None:
                refs[b] += 1
        new_rows.append(row)
        new_lens.append(n)
    free = [b for b, k in enumerate(refs) if k == 0]
    short = False
    for row in new_rows:
        for j, b in enumerate(row):
            if b is None and free:
                row[j] = free.pop(0)
                refs[row[j]] = 1
            elif b is None:
                row[j], short = -1, True
    before = [list(c) for c in contents]
    for r, j, b in copies:
        if new_rows[r][j] >= 0:
            for c, old in zip(contents, before):
                c[new_rows[r][j]] = old[b]
    return (new_rows, new_lens, refs), short


def compact(rows, refs, contents):
    """(rows, refs, new ids) with the blocks in use at the lowest ids."""
    live = [b for b, k in enumerate(refs) if k > 0]
    holes = [b for b in range(len(live)) if refs[b] <= 0]
    ids = [-1] * len(refs)
    for b in live:
        ids[b] = b if b < len(live) else holes.pop(0)
    new_refs = [0] * len(refs)
    before = [list(c) for c in contents]
    for b in live:
        new_refs[ids[b]] = refs[b]
        for c, old in zip(contents, before):
            c[ids[b]] = old[b]
    return [[ids[b] for b in row] for row in rows], new_refs, ids
