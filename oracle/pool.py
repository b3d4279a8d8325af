"""Reference of the page tables that follow lengths.

TEST INFRASTRUCTURE ONLY (see the package docstring). One page at a time, in
order, over Python lists:

    gone: the pages past each sequence's new length, by (sequence, index)
    a page is freed when its count reaches 0; its last release stands for it
    the list gets the freed pages in reverse order, then sequences take from its end
"""

from __future__ import annotations

__all__ = ["resize"]


def resize(table, lens, new_lens, refs, free, ps):
    """(table, lens, refs, free) after the resize, copies; free: the list in use."""
    table, refs, free = [list(r) for r in table], list(refs), list(free)
    count = lambda n: -(-n // ps)  # noqa: E731
    gone = [table[b][i] for b in range(len(lens)) for i in range(count(new_lens[b]), count(lens[b]))]
    for page in gone:
        refs[page] -= 1
    seen = set()
    for page in reversed(gone):
        if refs[page] == 0 and page not in seen:
            free.append(page)
        seen.add(page)
    out, stopped = [], False
    for b, (n, m) in enumerate(zip(lens, new_lens)):
        need = count(m) - count(n)
        stopped = stopped or need > len(free)
        if need > 0 and stopped:
            out.append(n)
            continue
        for i in range(count(n), count(m)):
            table[b][i] = free.pop()
            refs[table[b][i]] = 1
        out.append(m)
    return table, out, refs, free
