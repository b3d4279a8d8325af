"""Page tables that follow lengths, against the reference, entry by entry."""

import random

import pytest
import torch

from oracle import pool

pytestmark = pytest.mark.gpu


class Pool:
    """Tables, counts and a free list, with `shared` first pages common to all and
    room for `spare` pages more."""

    def __init__(self, lens, ps, width, shared=0, spare=0, seed=0):
        r = random.Random(seed)
        B = len(lens)
        held = [max(shared, -(-n // ps)) for n in lens]
        P = shared + sum(h - shared for h in held) + spare
        order = list(range(max(P, 1)))
        r.shuffle(order)
        self.ps, self.lens = ps, list(lens)
        self.refs = [0] * len(order)
        common = [order.pop() for _ in range(shared)]
        for p in common:
            self.refs[p] = B
        self.table = [common + [-7] * (width - shared) for _ in range(B)]
        for b in range(B):
            for i in range(shared, held[b]):
                self.table[b][i] = order.pop()
                self.refs[self.table[b][i]] = 1
        self.free = order
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.g = dict(table=t(self.table).view(B, width), refs=t(self.refs),
                      free_pages=t(self.free + [-9] * (len(self.refs) - len(self.free))), num_free=t([len(self.free)]))

    def step(self, fa2, new, **kw):
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out = fa2.cache_resize(self.g["table"], t(self.lens), t(new), self.g["refs"], self.g["free_pages"],
                               self.g["num_free"], self.ps, **kw)
        self.table, self.lens, self.refs, self.free = pool.resize(self.table, self.lens, new, self.refs, self.free, self.ps)
        assert out.tolist() == self.lens
        self.check()
        assert fa2.device_status() == 0
        return out

    def check(self):
        assert self.g["table"].tolist() == self.table
        assert self.g["refs"].tolist() == self.refs
        assert int(self.g["num_free"]) == len(self.free)
        assert self.g["free_pages"].tolist()[:len(self.free)] == self.free


@pytest.mark.parametrize("B,width,ps,shared,spare", [
    (1, 1, 1, 0, 2), (3, 5, 16, 2, 4), (17, 9, 7, 0, 50), (256, 40, 16, 3, 900), (1500, 12, 8, 0, 3000),
    (5000, 7, 3, 1, 9000), (9000, 2, 16, 0, 9000), (40, 700, 1, 5, 9000), (700, 64, 24, 10, 30000)])
def test_churn(cuda_device, fa2_lib, B, width, ps, shared, spare):
    r = random.Random(B + width)
    least, most = shared * ps, width * ps
    draw = lambda: r.choice([least, most, r.randint(least, most), r.randint(least, most)])  # noqa: E731
    p = Pool([draw() for _ in range(B)], ps, width, shared, spare, seed=B)
    for _ in range(4):
        p.step(fa2_lib, [draw() if r.random() < 0.5 else min(n + 1, most) for n in p.lens])
    p.step(fa2_lib, [0] * B)  # every sequence ends, the shared pages too
    assert len(p.free) == len(p.refs) and not any(p.refs)
    p.step(fa2_lib, [draw() for _ in range(B)])


def test_list_too_short(cuda_device, fa2_lib):
    for B, spare in ((6, 5), (300, 700), (6000, 9000)):
        r = random.Random(B)
        p = Pool([r.randint(0, 40) for _ in range(B)], 4, 20, spare=spare, seed=1)
        for _ in range(5):
            p.step(fa2_lib, [r.randint(0, 80) if r.random() < 0.3 else n for n in p.lens])
    p = Pool([0, 0], 1, 4)
    p.step(fa2_lib, [1, 0])  # one page in all, and none is free
    assert p.lens == [1, 0]


def test_undone(cuda_device, fa2_lib):
    r = random.Random(3)
    p = Pool([r.randint(0, 300) for _ in range(64)], 16, 20, spare=1300, seed=3)
    lens, free, table = p.lens, list(p.free), [row[:] for row in p.table]
    p.step(fa2_lib, [r.randint(0, 300) for _ in range(64)])
    p.step(fa2_lib, lens)
    assert p.free == free and p.lens == lens
    assert all(p.table[b][:-(-n // 16)] == table[b][:-(-n // 16)] for b, n in enumerate(lens))


def test_pages_named_several_times(cuda_device, fa2_lib):
    """Pages of two, three and all sequences, released in one call and one by one."""
    B, ps = 40, 4
    p = Pool([0] * B, ps, 6, spare=200)
    p.step(fa2_lib, [24] + [0] * (B - 1))
    for b in range(1, B):  # others take over a part of the first one's pages
        k = b % 7 if b % 7 < 6 else 6
        p.table[b][:k] = p.table[0][:k]
        for q in p.table[0][:k]:
            p.refs[q] += 1
        p.lens[b] = k * ps
    p.g["table"].copy_(torch.tensor(p.table, dtype=torch.int32))
    p.g["refs"].copy_(torch.tensor(p.refs, dtype=torch.int32))
    p.step(fa2_lib, [0 if b % 3 == 0 else n for b, n in enumerate(p.lens)])
    p.step(fa2_lib, [max(0, n - 5) for n in p.lens])
    p.step(fa2_lib, [0] * B)
    assert len(p.free) == 200 and not any(p.refs)


def test_bad_lengths_and_pages_stay_inside(cuda_device, fa2_lib):
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    guard = 64

    def boxed(v):
        x = torch.full((len(v) + 2 * guard,), 12345, dtype=torch.int32, device="cuda")
        x[guard:guard + len(v)] = t(v)
        return x, x[guard:guard + len(v)]

    for case in range(6):
        tb, table = boxed([0, 1, 2, 3, 4, 5])
        rb, refs = boxed([1, 1, 1, 1, 1, 1, 0, 0])
        fb, free = boxed([6, 7, -1, -1, -1, -1, -1, -1])
        lens, new, nf = [8, 8], [0, 12], [2]
        if case == 0:
            lens, new = [100, -3], [5, 12]               # lengths cut to 12 and 0
        elif case == 1:
            table[0], table[1] = 8, -2                    # pages that do not exist
        elif case == 2:
            refs[0] = refs[1] = 0                         # given back though not in use
        elif case == 3:
            nf = [50]                                     # a list longer than the pool
        else:
            free[0], free[1] = 99, -5                     # pages that do not exist in the list,
            new = [0, 12] if case == 4 else [8, 12]       # behind two that are freed, and at its end
        out = fa2_lib.cache_resize(table.view(2, 3), t(lens), t(new), refs, free, t(nf), 4)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == (0 if case == 4 else 9)
        for x, n in ((tb, 6), (rb, 8), (fb, 8)):
            assert (x[:guard] == 12345).all() and (x[guard + n:] == 12345).all()
        assert ((out >= 0) & (out <= 12)).all()
    assert fa2_lib.device_status() == 0


def test_graph_follows_lengths(cuda_device, fa2_lib):
    r = random.Random(5)
    B, ps, width = 30, 8, 10
    p = Pool([r.randint(0, 80) for _ in range(B)], ps, width, spare=400, seed=9)
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    new = lens.clone()
    out = torch.empty_like(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa2_lib.cache_resize(p.g["table"], lens, new, p.g["refs"], p.g["free_pages"], p.g["num_free"], ps, lens_out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa2_lib.cache_resize(p.g["table"], lens, new, p.g["refs"], p.g["free_pages"], p.g["num_free"], ps, lens_out=out)
        lens.copy_(out)
    for _ in range(6):
        want = [r.randint(0, 80) for _ in range(B)]
        new.copy_(torch.tensor(want, dtype=torch.int32))
        graph.replay()
        p.table, p.lens, p.refs, p.free = pool.resize(p.table, p.lens, want, p.refs, p.free, ps)
        torch.cuda.synchronize()
        assert lens.tolist() == p.lens
        p.check()


def test_refusals(cuda_device, fa2_lib):
    p = Pool([3, 4], 4, 2, spare=4)
    lens = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    a = dict(table=p.g["table"], lens=lens, new_lens=lens + 1, refs=p.g["refs"], free_pages=p.g["free_pages"],
             num_free=p.g["num_free"], page_size=4)
    for bad in (dict(table=a["table"].long()), dict(table=a["table"][0]), dict(table=a["table"].cpu()),
                dict(lens=lens[:1]), dict(new_lens=lens.cpu()), dict(refs=a["refs"].view(1, -1)),
                dict(free_pages=a["free_pages"][:-1]), dict(num_free=lens), dict(page_size=0), dict(page_size=2 ** 40),
                dict(page_size=1.5), dict(lens_out=lens.long()), dict(table=None)):
        with pytest.raises((ValueError, TypeError)):
            fa2_lib.cache_resize(**{**a, **bad})
    for bad, code in ((dict(lens_out=lens), 8), (dict(free_pages=a["refs"]), 8), (dict(page_size=2 ** 30), 1),
                      (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), 7)):
        with pytest.raises(fa2_lib.FA2Error) as e:
            fa2_lib.cache_resize(**{**a, **bad})
        assert e.value.code == code
    p.check()


def test_many_releases_of_pages_named_twice(cuda_device, fa2_lib):
    """More than 2^18 releases, over 32 to a lane, in which a page's last one counts."""
    B, width = 1600, 400
    r = random.Random(1)
    p = Pool([0] * B, 1, width, spare=B // 2 * width)
    p.step(fa2_lib, [width] * (B // 2) + [0] * (B // 2))
    for b in range(B // 2, B):
        n = r.randint(0, width)
        p.table[b][:n] = p.table[b - B // 2][:n]
        p.lens[b] = n
        for q in p.table[b][:n]:
            p.refs[q] += 1
    p.g["table"].copy_(torch.tensor(p.table, dtype=torch.int32))
    p.g["refs"].copy_(torch.tensor(p.refs, dtype=torch.int32))
    assert sum(p.lens) > 2 ** 18
    p.step(fa2_lib, [0] * B)
    assert len(p.free) == len(p.refs) and not any(p.refs)
