"""Plain forms of the operators over a cache's pages: lists of numbers, one step after the other."""


def free_of(ref):
    return [p for p, x in enumerate(ref) if x == 0]


def copy(src, dst, NB):
    """Moves, and whether something was flagged."""
    inside = [0 <= s < NB and 0 <= d < NB for s, d in zip(src, dst)]
    times = {}
    for s, d, ok in zip(src, dst, inside):
        if ok:
            times[d] = times.get(d, 0) + 1
    moves, bad = [], False
    for s, d, ok in zip(src, dst, inside):
        if s == -1 or d == -1:
            continue
        if ok and times[d] == 1 and s not in times:
            moves.append((s, d))
        else:
            bad = True
    return moves, bad


def fork(table, lengths, parent, ref, bs, MB):
    """(moves, new table, new lengths, new ref, rows that found no page)."""
    free, moves, rows, new_lengths, failed, taken = free_of(ref), [], [], [], [], set()
    at = 0
    for i, a in enumerate(parent):
        if a < 0 or not 0 <= lengths[a] <= MB * bs:
            rows.append([-1] * MB)
            new_lengths.append(0)
            taken.add(a)
            continue
        n, row = -(-lengths[a] // bs), list(table[a])
        row[n:] = [-1] * (MB - n)
        ok = True
        if a in taken and lengths[a] % bs and row[n - 1] >= 0:
            ok = at < len(free)
            if ok:
                moves.append((row[n - 1], free[at]))
                row[n - 1] = free[at]
            at += 1
        if not ok:
            failed.append(i)
        taken.add(a)
        rows.append(row if ok else [-1] * MB)
        new_lengths.append(lengths[a] if ok else 0)
    ref = list(ref)
    for sign, t in ((-1, table), (1, rows)):
        for row in t:
            for p in row:
                if p >= 0:
                    ref[p] += sign
    return moves, rows, new_lengths, ref, failed


def resize(table, lengths, delta, ref, bs, MB):
    """(moves, new table, new lengths, new ref, rows left out)."""
    free, at, moves, failed = free_of(ref), 0, [], []
    before, table, ref, out = list(ref), [list(r) for r in table], list(ref), []
    for r, (was, d) in enumerate(zip(lengths, delta)):
        now = was + d
        if not (0 <= was <= MB * bs and 0 <= now <= MB * bs):
            failed.append(r)
            out.append(was)
            continue
        row = table[r]
        # entries that hold a position of [was, now): those of a page that other rows hold too become fresh pages, and
        # so do those without one, unless a position below `was` lies there as well
        want = [c for c in range(was // bs, -(-now // bs)) if now > was and
                (before[row[c]] > 1 if row[c] >= 0 else c * bs >= was)]
        need = len(want)
        first, at = at, at + need
        if need and at > len(free):
            failed.append(r)
            out.append(was)
            continue
        for k, c in enumerate(want):
            if row[c] >= 0:
                if c * bs < was:  # positions below `was` lie there: its bytes go along
                    moves.append((row[c], free[first + k]))
                ref[row[c]] -= 1
            row[c] = free[first + k]
            ref[free[first + k]] = 1
        for c in range(-(-now // bs), MB):
            if row[c] >= 0:
                ref[row[c]] -= 1
            row[c] = -1
        out.append(now)
    return moves, table, out, ref, failed


def compact(table, ref):
    """(moves, new table, new ref, pages in use)."""
    live = sum(x != 0 for x in ref)
    holes = [p for p in range(live) if ref[p] == 0]
    moves = list(zip([p for p in range(live, len(ref)) if ref[p]], holes))
    place, new = dict(moves), list(ref)
    for s, d in moves:
        new[d], new[s] = ref[s], 0
    return moves, [[place.get(p, p) for p in row] for row in table], new, live
