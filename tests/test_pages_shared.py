"""Rows that grow into pages which other rows hold too: no position of another row may lie where a row writes next.

The property is checked from its definition, on the plain form (CPU) and on the operator, with rows cut back into shared
pages, at their borders and across several of them."""

import pytest
import torch

import pages_ref
import paged_kv_cache_reshape_gb300 as pa


def shared_state(table, NB):
    """Reference counts of a table."""
    ref = [0] * NB
    for row in table:
        for p in row:
            if p >= 0:
                ref[p] += 1
    return ref


def drawn_state(seed, R, MB, bs):
    """Rows on common pages that reach behind their lengths (as after drafts that were refused), and how they change."""
    g = torch.Generator().manual_seed(seed)

    def some(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))

    NB = 2 * R * MB + 5
    ids = torch.randperm(NB, generator=g).tolist()
    table, lengths, delta = [], [], []
    for r in range(R):
        row = [ids.pop() for _ in range(some(0, MB))]
        if r and some(0, 3):
            other, k = table[some(0, r - 1)], some(0, MB)
            row = [p for p in other[:k] if p >= 0] + row[k:]
        row += [-1] * (MB - len(row))
        held = sum(p >= 0 for p in row)
        length = some(0, held * bs)
        if some(0, 1):
            length = length // bs * bs
        table.append(row)
        lengths.append(length)
        delta.append(some(-length, MB * bs - length) if some(0, 2) else some(0, min(2, MB * bs - length)))
    return table, lengths, delta, NB


CASES = {
    # rows 0 and 1 hold the same four pages
    "cut_at_a_border": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [64, 48], [0, 1]),
    "across_two_shared_pages": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [64, 40], [0, 40]),
    "across_all": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [64, 0], [1, 80]),
    "both_grow": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [40, 40], [1, 30]),
    "only_pages_of_new_positions": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [64, 16], [0, 16]),
    "own_page_after_a_shared_one": ([[0, 1, 2, -1, -1], [0, 1, 2, 7, -1]], [48, 32], [0, 20]),
    "hole_between_shared_ones": ([[0, 1, 2, 3, 4], [0, 1, -1, 3, 4]], [80, 20], [0, 60]),
    "one_shrinks_one_grows": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [64, 48], [-64, 8]),
    "three_rows": ([[0, 1, 2, -1, -1], [0, 1, 2, -1, -1], [0, 1, 2, -1, -1]], [48, 32, 33], [0, 17, 2]),
    "stays_as_long": ([[0, 1, 2, 3, -1], [0, 1, 2, 3, -1]], [64, 40], [0, 0]),
}


def all_cases():
    for table, lengths, delta in CASES.values():
        yield table, lengths, delta, 20, 16
    for seed in range(30):
        bs = [16, 1, 5, 32][seed % 4]
        yield (*drawn_state(seed, 2 + seed % 5, 3 + seed % 7, bs), bs)


def assert_apart(table, lengths, new_table, new_lengths, new_ref, content, new_content, bs):
    """Kept positions hold what they held, and where a row has new positions no other entry refers to."""
    users = {}
    for r, row in enumerate(new_table):
        for c, p in enumerate(row):
            if p >= 0:
                users.setdefault(p, []).append((r, c))
    assert new_ref == [len(users.get(p, [])) for p in range(len(new_ref))]
    for r, (was, now) in enumerate(zip(lengths, new_lengths)):
        for pos in range(min(was, now)):
            old, new = table[r][pos // bs], new_table[r][pos // bs]
            assert (old < 0) == (new < 0)
            if old >= 0:
                assert content[old][pos % bs] == new_content[new][pos % bs], (r, pos)
        for c in range(was // bs, -(-now // bs)):
            if now > was and new_table[r][c] >= 0:
                assert users[new_table[r][c]] == [(r, c)], (r, c)


def test_the_plain_form_keeps_rows_apart():
    for table, lengths, delta, NB, bs in all_cases():
        ref = shared_state(table, NB)
        moves, new, new_lengths, new_ref, failed = pages_ref.resize(table, lengths, delta, ref, bs, len(table[0]))
        assert not failed and new_lengths == [a + b for a, b in zip(lengths, delta)]
        content = [[(p, i) for i in range(bs)] for p in range(NB)]
        after = list(content)
        for s, d in moves:
            after[d] = content[s]
        assert_apart(table, lengths, new, new_lengths, new_ref, content, after, bs)


@pytest.mark.gpu
def test_rows_stay_apart():
    pa.build()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    for table, lengths, delta, NB, bs in all_cases():
        R, MB, ref = len(table), len(table[0]), shared_state(table, NB)
        pool = torch.arange(NB * bs * 4, dtype=torch.int32, device="cuda").view(NB, bs * 4)
        content = pool.view(NB, bs, 4)[:, :, 0].tolist()
        want = pages_ref.resize(table, lengths, delta, ref, bs, MB)
        op, t, new, count = pa.CachePages(bs, NB, MB, R, 16 * bs), ints(table), ints(lengths) * 0 - 9, ints(ref)
        op.resize(pa.page_pools([pool]), t, ints(lengths), ints(delta), new, count)
        assert op.device_error() == 0
        assert t.tolist() == want[1] and new.tolist() == want[2] and count.tolist() == want[3]
        assert_apart(table, lengths, t.tolist(), new.tolist(), count.tolist(), content,
                     pool.view(NB, bs, 4)[:, :, 0].tolist(), bs)


@pytest.mark.gpu
def test_long_rows_on_shared_pages():
    """More entries than a warp takes at a time, shared and missing ones in turn."""
    pa.build()
    MB, bs, NB = 150, 16, 500
    shared = list(range(100, 250))
    table = [shared, [p if c % 3 else -1 for c, p in enumerate(shared)], [-1] * MB]
    lengths, delta, ref = [2400, 20, 0], [0, 2380, 700], shared_state(table, NB)
    pool = torch.arange(NB * bs * 4, dtype=torch.int32, device="cuda").view(NB, bs * 4)
    content = pool.view(NB, bs, 4)[:, :, 0].tolist()
    want = pages_ref.resize(table, lengths, delta, ref, bs, MB)
    t, new, count = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, lengths, ref))
    op = pa.CachePages(bs, NB, MB, 3, 16 * bs)
    op.resize(pa.page_pools([pool]), t, new, torch.tensor(delta, dtype=torch.int32, device="cuda"), new, count)
    assert op.device_error() == 0
    assert t.tolist() == want[1] and new.tolist() == want[2] and count.tolist() == want[3]
    assert_apart(table, lengths, t.tolist(), new.tolist(), count.tolist(), content,
                 pool.view(NB, bs, 4)[:, :, 0].tolist(), bs)
