"""Reference for the operators on a pool of pages (test infrastructure only):
plain Python, one sequence and one page after another.  Tables are lists of rows."""


def pages_of(tokens, page_size):
    return -(-tokens // page_size)


def fork(refs, table, lengths, parent, page_size, columns):
    """(refs, table, lengths) with the children's rows."""
    refs, rows, out = list(refs), [], []
    for p in parent:
        length = lengths[p] if 0 <= p < len(table) else 0
        if length < 0 or length > min(len(table[0]) if table else 0, columns) * page_size:
            length = 0
        row = [-1] * columns
        for c in range(pages_of(length, page_size)):
            if 0 <= table[p][c] < len(refs):
                row[c] = table[p][c]
                refs[row[c]] += 1
        rows.append(row)
        out.append(length)
    return refs, rows, out


def resize(refs, table, before, after, page_size):
    """(refs, table, moves, missing)."""
    refs, table = list(refs), [list(row) for row in table]
    fine = [0 <= x <= len(row) * page_size and 0 <= y <= len(row) * page_size
            for row, x, y in zip(table, before, after)]
    for b, row in enumerate(table):
        if fine[b]:
            for c in range(pages_of(after[b], page_size), pages_of(before[b], page_size)):
                if 0 <= row[c] < len(refs):
                    refs[row[c]] -= 1
                row[c] = -1
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    shared = [r > 1 for r in refs]
    moves, missing, wanted = [], [], 0
    for b, row in enumerate(table):
        moves.append([-1, -1])
        if not fine[b]:
            missing.append(-1)
            continue
        held, want = pages_of(before[b], page_size), pages_of(after[b], page_size)
        again = after[b] > before[b] and before[b] % page_size != 0 and 0 <= row[held - 1] < len(refs) and \
            shared[row[held - 1]]
        columns = ([held - 1] if again else []) + list(range(held, want))
        first, wanted = wanted, wanted + len(columns)
        if wanted > len(free):
            missing.append(len(columns))
            continue
        missing.append(0)
        if again:
            moves[b] = [row[held - 1], free[first]]
            refs[row[held - 1]] -= 1
        for r, c in enumerate(columns):
            row[c] = free[first + r]
            refs[row[c]] = 1
    return refs, table, moves, missing


def compact(refs, table, lengths, page_size):
    """(refs, table, moves, used)."""
    used = [p for p in range(len(refs)) if refs[p] > 0]
    n = len(used)
    holes = [p for p in range(n) if refs[p] <= 0]
    movers = [p for p in used if p >= n]
    where = {p: p for p in used}
    where.update(zip(movers, holes))
    out = [0] * len(refs)
    for p in used:
        out[where[p]] = refs[p]
    rows = []
    for row, length in zip(table, lengths):
        held = pages_of(length, page_size) if 0 <= length <= len(row) * page_size else 0
        rows.append([where.get(p, -1) if c < held else -1 for c, p in enumerate(row)])
    moves = [[a, b] for a, b in zip(movers, holes)]
    return out, rows, moves + [[-1, -1]] * (len(refs) // 2 - len(moves)), n
