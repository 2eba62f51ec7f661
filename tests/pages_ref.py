"""Plain implementations of the calls on the cache's pages, with lists, for the tests."""


def entries(n, size):
    return -(-n // size)


def rows_of(table, lens, size, cap):
    """The used entries of each row."""
    return [list(t[: entries(min(max(x, 0), cap), size)]) for t, x in zip(table, lens)]


def fork(table, lens, sources, count, size):
    P, N = len(table[0]), len(count)
    cap = P * size
    count = list(count)
    out, out_lens = [], []
    for s in sources:
        ok = 0 <= s < len(table)
        n = min(max(lens[s], 0), cap) if ok else 0
        row = list(table[s][: entries(n, size)]) if ok else []
        for p in row:
            if 0 <= p < N:
                count[p] += 1
        out.append(row + [-1] * (P - len(row)))
        out_lens.append(n)
    return out, out_lens, count


def free(table, lens, release, count, size):
    count = list(count)
    for row, gone in zip(rows_of(table, lens, size, len(table[0]) * size), release):
        for p in row if gone else ():
            if 0 <= p < len(count):
                count[p] -= 1
    return count


def reserve(table, lens, new_lens, count, size):
    """table, count, reserved and the copies (from, to, tokens)."""
    P, N = len(table[0]), len(count)
    cap = P * size
    lens = [min(max(x, 0), cap) for x in lens]
    want = [max(x, min(w, cap)) for x, w in zip(lens, new_lens)]
    rows = rows_of(table, lens, size, cap)
    before = list(count)
    count = list(count)
    free = [p for p in range(N) if before[p] <= 0]

    def shared(b):
        if want[b] == lens[b] or lens[b] % size == 0:
            return None
        p = rows[b][-1]
        return p if 0 <= p < N and before[p] > 1 else None

    writers = {}
    for b in range(len(rows)):
        if shared(b) is not None:
            writers.setdefault(shared(b), []).append(b)
    keepers = {w[-1] for p, w in writers.items() if len(w) >= before[p]}
    reserved, copies, asked = [], [], 0
    for b, row in enumerate(rows):
        copy = shared(b) is not None and b not in keepers
        n = entries(want[b], size) - entries(lens[b], size) + copy
        given = free[asked:asked + n]
        asked += n
        if asked > len(free) and (n > 0 or b in keepers):
            reserved.append(lens[b])
            continue
        reserved.append(want[b])
        for p in given:
            count[p] = 1
        if copy:
            copies.append((row[-1], given[0], lens[b] % size))
            count[row[-1]] -= 1
            row[-1] = given[0]
            given = given[1:]
        row.extend(given)
    return [r + [-1] * (P - len(r)) for r in rows], count, reserved, copies


def compact(table, lens, count, size):
    """table, count, live pages and the moves (from, to)."""
    P, N = len(table[0]), len(count)
    live = [p for p in range(N) if count[p] > 0]
    n = len(live)
    come = [p for p in live if p >= n]
    holes = [p for p in range(n) if count[p] <= 0]
    place = {p: p for p in live}
    count = list(count)
    for a, b in zip(come, holes):
        place[a] = b
        count[b], count[a] = count[a], 0
    rows = [[place.get(p, -1) for p in r] for r in rows_of(table, lens, size, P * size)]
    return [r + [-1] * (P - len(r)) for r in rows], count, n, list(zip(come, holes))
