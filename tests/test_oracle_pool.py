"""Pins of the page-pool reference (CPU)."""

import random

from oracle import pool


def test_by_hand():
    # pages of 4 slots; two sequences share pages 0 and 1
    table = [[0, 1, 2, -1], [0, 1, 5, 6], [-1] * 4]
    t, n, refs, free = pool.resize(table, [9, 16, 0], [4, 0, 5], [2, 2, 1, 0, 0, 1, 1], [3, 4], 4)
    # gone: 1 2 | 0 1 5 6; page 0 is still named; freed: 2, 1 (its second release), 5, 6
    assert refs[0] == 1 and n == [4, 0, 5]
    assert t[2][:2] == [2, 1] and free == [3, 4, 6, 5]  # the first release stands at the list's end
    assert refs == [1, 1, 1, 0, 0, 0, 0]


def test_list_too_short():
    table = [[-1] * 3 for _ in range(4)]
    t, n, refs, free = pool.resize(table, [0, 0, 0, 0], [2, 5, 0, 1], [0] * 4, [0, 1, 2, 3], 2)
    assert n == [2, 5, 0, 0] and free == []   # 1 page, then the 3 that are left, then none
    assert t[0][0] == 3 and t[1] == [2, 1, 0]
    t, n, refs, free = pool.resize(table, [0, 0, 0, 0], [2, 5, 0, 1], [0] * 3, [0, 1, 2], 2)
    assert n == [2, 0, 0, 0] and free == [0, 1]  # the last would find one, but comes after the second


def test_undone():
    r = random.Random(0)
    for _ in range(200):
        ps, B = r.randint(1, 5), r.randint(1, 6)
        lens = [r.randint(0, 30) for _ in range(B)]
        new = [r.randint(0, 30) for _ in range(B)]
        pages = list(range(6 * 31))
        r.shuffle(pages)
        refs = [0] * len(pages)
        table = [[-1] * 31 for _ in range(B)]
        for b, n in enumerate(lens):
            for i in range(-(-n // ps)):
                table[b][i] = pages.pop()
                refs[table[b][i]] = 1
        t, n, f, free = pool.resize(table, lens, new, refs, pages, ps)
        assert n == new
        held = [t[b][i] for b in range(B) for i in range(-(-new[b] // ps))]
        assert sorted(held + free) == list(range(6 * 31))
        t2, n2, f2, free2 = pool.resize(t, new, lens, f, free, ps)
        assert n2 == lens and free2 == pages and f2 == refs
        assert all(t2[b][:-(-lens[b] // ps)] == table[b][:-(-lens[b] // ps)] for b in range(B))
