"""Decoding behind a shared prefix, against the fp64 oracle on the same tables."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, FP16, Cache, bits64, decode_bounds, score_error

pytestmark = pytest.mark.gpu


class Shared(Cache):
    """A cache whose sequences of at least P slots begin with those of the last one:
    whole pages by name, the page that the prefix ends in as a copy."""

    def __init__(self, B, Hkv, d, ps, P, lens, dtype, seed, width=None):
        lens = [int(n) for n in lens]
        assert lens[-1] >= P
        super().__init__(B, Hkv, d, ps, lens, dtype, seed, width=width)
        whole, rest = P // ps, P % ps
        first = self.table[-1].clone()
        for b in range(B - 1):
            if lens[b] < P:
                continue
            self.table[b, :whole] = first[:whole]
            if rest:
                for c in (self.k, self.v):
                    c[self.table[b, whole], :, :rest] = c[first[whole], :, :rest]
        self.P = P
        self.prefix = first[:max(1, -(-P // ps))].clone()
        self.prefix_len = torch.tensor([P], dtype=torch.int32)

    def args(self, q, room=False):
        """room: a list of the prefix's pages with room for 140000 slots; from its length
        the library decides which kernel attends to the prefix (more than 16 query rows)."""
        kc, vc, table, lens = self.gpu()
        prefix = self.prefix
        if room:
            prefix = torch.cat([prefix, torch.full((140000 // self.ps + 1,), -5, dtype=torch.int32)])
        return [q.cuda(), kc, vc, table, lens, prefix.cuda(), self.prefix_len.cuda()]


def _check(c, q, o, lse, scale, visible=None):
    k64, v64, n = bits64(c.k), bits64(c.v), int(c.lens.max())
    args = (c.table.numpy(), c.lens.numpy(), scale)
    o_ref, l_ref, _ = oc.paged_decode(bits64(q), k64, v64, *args, visible=visible)
    A, _, _ = oc.paged_decode(bits64(q), k64, np.abs(v64), *args, visible=visible)
    tol_o, tol_l, _ = decode_bounds(o_ref, l_ref, A, score_error(bits64(q), np.nan_to_num(k64), scale), n, c.dtype)
    assert (np.abs(bits64(o) - o_ref) <= tol_o).all(), np.max(np.abs(bits64(o) - o_ref) - tol_o)
    fin = np.isfinite(l_ref)
    got = bits64(lse)
    assert (got[~fin] == -np.inf).all() and (np.abs(got - np.where(fin, l_ref, 0))[fin] <= tol_l[fin]).all()


# B, Hq, Hkv, d, page size, prefix, slots behind it (-n: a sequence of n slots without the prefix)
CASES = [
    (1, 1, 1, 64, 16, 16, [1]),
    (1, 1, 1, 128, 16, 0, [5]),
    (2, 8, 2, 128, 16, 1, [0, 3]),
    (3, 4, 4, 64, 8, 127, [0, 1, 200]),
    (4, 6, 2, 128, 24, 129, [-128, 5, -1, 70]),
    (5, 8, 8, 128, 1, 140, [1, 2, -0, 0, 4]),
    (3, 7, 1, 64, 5, 263, [9, -100, 64]),
    (2, 2, 2, 128, 6, 45, [9, 1]),
    (2, 12, 4, 64, 4, 400, [30, 1]),
    (33, 4, 1, 128, 16, 300, None),          # 132 rows: a second tile of 4
    (64, 4, 1, 64, 32, 1000, None),          # 256 rows
    (65, 12, 3, 128, 64, 640, None),         # 260 rows: a second item of one tile
    (9, 34, 2, 128, 16, 777, None),          # 17 heads to a key head
    (3, 128, 1, 64, 128, 1500, [0, 40, 129]),
    (40, 32, 8, 128, 16, 512, None),
    (2, 2, 1, 128, 4096, 5000, [3, 200]),
    (6, 16, 16, 64, 48, 0, None),
    (3, 2, 2, 64, 64, 20011, [0, 1, 77]),    # a long prefix over few heads
]

# Enough units that a CTA of the prefix has several slot tiles, and pieces of two items
MANY = [
    (5, 160, 40, 128, 16, 1300, None),       # 20 rows: one tile, both row groups on it
    (8, 128, 32, 64, 16, 1500, None),        # 32 rows
    (34, 96, 24, 128, 16, 1500, None),       # 136 rows: two tiles
    (65, 64, 16, 64, 32, 1700, None),        # 260 rows: items of two tiles and of one
]


def _lens(case):
    B, P, own = case[0], case[5], case[6]
    if own is None:
        r = np.random.default_rng(B)
        own = [int(x) for x in r.integers(0, 150, B)]
        own[0] = -min(P - 1, 30) if P > 1 else 0
    return [(-n if n < 0 else P + n) for n in own]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c[:6])))
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_matches_the_oracle(cuda_device, fa2_lib, case, dtype):
    B, Hq, Hkv, d, ps, P, _ = case
    c = Shared(B, Hkv, d, ps, P, _lens(case), dtype, seed=Hq + ps)
    q = c.query(Hq, 1.5)
    for room in (False, True):
        a = c.args(q, room)
        o, lse = fa2_lib.prefix_decode(*a)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 0
        _check(c, q, o, lse, d ** -0.5)
        o2, lse2 = fa2_lib.prefix_decode(*a)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("case", MANY, ids=lambda c: "_".join(map(str, c[:6])))
def test_several_tiles_per_cta(cuda_device, fa2_lib, case):
    B, Hq, Hkv, d, ps, P, _ = case
    dtype = BF16 if d == 128 else FP16
    c = Shared(B, Hkv, d, ps, P, _lens(case), dtype, seed=Hq + ps)
    q = c.query(Hq, 1.5)
    a = c.args(q, True)
    first = fa2_lib.prefix_decode(*a)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    _check(c, q, *first, d ** -0.5)
    for _ in range(20):
        o, lse = fa2_lib.prefix_decode(*a)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


UNEVEN = [  # enough slots behind the prefix that its kernel's time decides the CTAs' shares
    (40, 64, 16, 64, 16, 1024, [200 + i for i in range(40)]),       # 12 parts to 4
    (40, 64, 16, 64, 16, 1024, [430 - i for i in range(40)]),       # 10 to 6
    (40, 64, 16, 64, 16, 1000, [900 - 3 * i for i in range(40)]),   # 9 to 7
    (2, 576, 8, 64, 16, 1024, [1300, 1290]),                        # by CTAs
    (36, 96, 12, 128, 32, 1500, [i % 5 * 90 for i in range(36)]),   # some with nothing of their own
]


@pytest.mark.parametrize("case", UNEVEN, ids=lambda c: "_".join(map(str, c[:6])) + f"_{c[6][0]}")
def test_uneven_shares(cuda_device, fa2_lib, case):
    test_several_tiles_per_cta(cuda_device, fa2_lib, case)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("std,scale", [(12.0, None), (0.0, None), (1.0, 1e-6), (3.0, 2.0)])
def test_sharp_and_flat_rows(cuda_device, fa2_lib, std, scale, dtype):
    c = Shared(20, 2, 128, 16, 900, [900 + 7 * i for i in range(20)], dtype, seed=4)
    q = c.query(8, std)
    for room in (False, True):
        o, lse = fa2_lib.prefix_decode(*c.args(q, room), scale=scale)
        _check(c, q, o, lse, scale or 128 ** -0.5)


def test_a_table_with_room_and_a_prefix_list_with_room(cuda_device, fa2_lib):
    c = Shared(5, 2, 64, 16, 200, [200, 0, 31, 260, 333], BF16, seed=1, width=60)
    q = c.query(6)
    a = c.args(q)
    a[5] = torch.cat([c.prefix, torch.full((40,), -5, dtype=torch.int32)]).cuda()  # not in use
    o, lse = fa2_lib.prefix_decode(*a)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    _check(c, q, o, lse, 0.125)


def test_outputs_are_the_rounded_exact_values(cuda_device, fa2_lib):
    """Rounded once: nearly every output is the exact value's nearest."""
    for dtype, most, room in ((BF16, 0.004, False), (FP16, 0.02, False), (BF16, 0.004, True), (FP16, 0.02, True)):
        c = Shared(32, 2, 128, 16, 2000, [2000 + 3 * i for i in range(32)], dtype, seed=2)
        q = c.query(8, 2.0)
        o, _ = fa2_lib.prefix_decode(*c.args(q, room))
        ref, _, _ = oc.paged_decode(bits64(q), bits64(c.k), bits64(c.v), c.table.numpy(), c.lens.numpy(), 128 ** -0.5)
        want = torch.from_numpy(ref).to(dtype)
        assert float((o.cpu() != want).float().mean()) <= most
        err = np.sqrt(np.mean((bits64(o) - ref) ** 2)) / np.sqrt(np.mean(ref ** 2))
        assert err <= torch.finfo(dtype).eps / 2 * 0.6  # uniform within half a step: 0.29 to 0.58 of it


def test_slots_far_below_the_largest_count(cuda_device, fa2_lib):
    """One slot of the largest score has V = 0; what is left of o are the others, 2^-18
    below it (fp16: pieces down to 2^-36 of the row's largest)."""
    for dtype, B in ((BF16, 3), (FP16, 3), (BF16, 40), (FP16, 40)):
        c = Shared(B, 1, 64, 16, 4096, [4096] * (B - 1) + [4100], dtype, seed=6)
        c.k.zero_()
        page, off = int(c.table[-1, 37]), 5
        c.k[page, 0, off, 0] = 1.0
        c.v[page, 0, off] = 0.0
        q = torch.zeros(B, 1, 64, dtype=dtype)
        q[..., 0] = 18.0
        o, lse = fa2_lib.prefix_decode(*c.args(q, B > 16), scale=float(np.log(2.0)))
        _check(c, q, o, lse, float(np.float32(np.log(2.0))))
        ref, _, _ = oc.paged_decode(bits64(q), bits64(c.k), bits64(c.v), c.table.numpy(), c.lens.numpy(),
                                    float(np.float32(np.log(2.0))))
        assert (np.abs(bits64(o) - ref) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -24).all()


def test_bad_pages_of_the_prefix_are_masked(cuda_device, fa2_lib):
    for ps, bad, B in ((16, (1, 3), 4), (5, (0, 20, 21), 4), (64, (2,), 4), (16, (1, 3), 40), (5, (0, 20, 21), 40),
                       (64, (2,), 40), (2, (60, 61, 63, 64, 100), 40), (4, (15, 31, 32), 40)):
        c = Shared(B, 2, 64, ps, 250, [250, 300, 13, 260] * (B // 4), BF16, seed=8)
        q = c.query(4)
        a = c.args(q, B > 16)
        prefix = a[5].cpu()
        for i, p in enumerate(bad):
            prefix[p] = -1 if i % 2 else c.k.shape[0]
        a[5] = prefix.cuda()
        o, lse = fa2_lib.prefix_decode(*a)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 9
        box = 16 if ps % 16 == 0 else ps if ps in (2, 4) else 1
        cut = 250 // box * box
        hide = [np.array([not (n >= 250 and j < cut and j // ps in bad) for j in range(n)], bool) for n in c.lens.tolist()]
        _check(c, q, o, lse, 0.125, visible=hide)


def test_lengths_out_of_range(cuda_device, fa2_lib):
    c = Shared(3, 1, 64, 16, 48, [50, 60, 64], BF16, seed=9)
    q = c.query(2)
    a = c.args(q)
    want = fa2_lib.prefix_decode(*a)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    a[6] = torch.tensor([1000], dtype=torch.int32, device="cuda")  # cut to 48
    got = fa2_lib.prefix_decode(*a)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9 and torch.equal(got[0], want[0])
    a[6] = torch.tensor([-3], dtype=torch.int32, device="cuda")    # no prefix
    got = fa2_lib.prefix_decode(*a)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9
    _check(c, q, *got, 0.125)
    a[6], a[4] = c.prefix_len.cuda(), torch.tensor([50, -4, 1000], dtype=torch.int32, device="cuda")
    got = fa2_lib.prefix_decode(*a)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][2], want[0][2])
    assert (got[0][1] == 0).all() and (got[1][1] == -float("inf")).all()


def test_a_wait_that_runs_out(cuda_device, fa2_lib):
    """V tiles of the prefix that never arrive: a status, and the next call is right."""
    for rows, P in ((40, 700), (300, 700)):
        c = Shared(rows, 1, 128, 16, P, [P + 3] * rows, BF16, seed=3)
        q = c.query(1)
        a = c.args(q, True)
        assert fa2_lib.load_library().fa2_debug_arm_fault(7, 30) == 0
        fa2_lib.prefix_decode(*a)
        assert fa2_lib.device_status() == 6
        o, lse = fa2_lib.prefix_decode(*a)
        assert fa2_lib.device_status() == 0
        _check(c, q, o, lse, 128 ** -0.5)


def test_infinite_values(cuda_device, fa2_lib):
    """An infinite V gives outputs that are not finite in its own column, and nothing
    elsewhere; in slots that a sequence does not have it gives nothing."""
    for rep in (1, 12):
        c = Shared(3 * rep, 1, 64, 16, 64, [70, 20, 80] * rep, BF16, seed=5)
        c.v[c.table[-1, 1], 0, 3, 7] = float("inf")
        q = c.query(2)
        o, _ = fa2_lib.prefix_decode(*c.args(q, rep > 1))
        bad = ~torch.isfinite(o.cpu())
        want = torch.zeros_like(bad)
        want[0::3, :, 7] = want[2::3, :, 7] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("B,Hq,Hkv,d,ps,P", [(3, 4, 2, 64, 16, 200), (30, 4, 2, 64, 16, 700), (40, 8, 2, 128, 5, 333),
                                             (90, 12, 2, 128, 64, 1500), (300, 2, 2, 64, 16, 150)])
def test_infinite_values_come_out_infinite(cuda_device, fa2_lib, B, Hq, Hkv, d, ps, P, dtype):
    """A V entry of +-inf makes its element of o +-inf, as p * inf does, in the prefix and
    behind it; both signs in one column, or NaN, make NaN; all other elements are as
    without it, and so are those of sequences that do not have the prefix."""
    lens = [P + b % 40 for b in range(B)]
    lens[1], lens[-1] = P - 9, P + 7
    c = Shared(B, Hkv, d, ps, P, lens, dtype, seed=B)
    q, g = c.query(Hq), Hq // Hkv
    bad = c.v.clone()

    def put(j, col, x, b=B - 1):
        bad[int(c.table[b, j // ps]), Hkv - 1, j % ps, col] = x

    inf, nan = float("inf"), float("nan")
    for j in (2, 17, 65, 99, P // 2 // ps * ps):    # whole pages of the prefix
        put(j, 3, inf)
        put(j, 9, -inf)
    put(5, 20, inf)
    put(101, 20, -inf)
    put(33, 30, nan)
    put(34, 30, inf)
    put(70, d - 1, inf)
    put(P + 3, d - 1, -inf)                        # the last sequence's own slot
    put(P + 4, 40, -inf)
    for room in (False, True):
        a = c.args(q, room)
        want, lse0 = (t.cpu() for t in fa2_lib.prefix_decode(*a))
        a[2] = bad.cuda()
        o, lse = (t.cpu() for t in fa2_lib.prefix_decode(*a))
        assert fa2_lib.device_status() == 0
        heads = slice(Hq - g, Hq)
        on = torch.tensor([n >= P for n in lens])
        for col, x in ((3, inf), (9, -inf), (20, nan), (30, nan), (d - 1, inf)):
            part = want[on]
            part[:, heads, col] = x
            want[on] = part
        want[-1, heads, d - 1], want[-1, heads, 40] = nan, -inf
        assert torch.equal(o.isnan(), want.isnan())
        assert torch.equal(o.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
        assert torch.equal(lse, lse0)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_infinite_values_of_slots_that_weigh_little(cuda_device, fa2_lib, dtype):
    """2^-60 of the largest is a weight; a score of -inf is none, and 0 * inf is NaN."""
    for B in (3, 40):
        c = Shared(B, 1, 64, 16, 512, [512] * (B - 1) + [515], dtype, seed=7)
        c.k.zero_()
        c.k[int(c.table[-1, 20]), 0, 5, 0] = 1.0                 # the largest score, 60
        c.k[int(c.table[-1, 3]), 0, 1, 0] = -float("inf")
        c.v[int(c.table[-1, 9]), 0, 2, 11] = float("inf")        # score 0
        c.v[int(c.table[-1, 3]), 0, 1, 12] = float("inf")
        q = torch.zeros(B, 1, 64, dtype=dtype)
        q[..., 0] = 60.0
        for o, _ in (fa2_lib.prefix_decode(*c.args(q, B > 16), scale=float(np.log(2.0))),
                     fa2_lib.paged_decode(*c.args(q)[:5], scale=float(np.log(2.0)))):
            o = o.cpu()
            assert (o[:, :, 11] == float("inf")).all() and o[:, :, 12].isnan().all()
            assert int((~torch.isfinite(o)).sum()) == 2 * B


@pytest.mark.parametrize("B", [6, 12])
def test_graph_follows_lengths_prefix_and_tables(cuda_device, fa2_lib, B):
    ps = 16
    c = Shared(B, 2, 128, ps, 400, [420 + 11 * i for i in range(B)], BF16, seed=12, width=45)
    q = c.query(8)
    a = c.args(q, B > 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa2_lib.prefix_decode(*a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa2_lib.prefix_decode(*a)
    for P in (400, 0, 37, 384, 129):
        a[6].fill_(P)
        lens = [(n if n < 420 else n - (P % 7)) for n in c.lens.tolist()]
        lens[1] = P - 1 if P > 1 else 0
        lens[2] = P
        a[4].copy_(torch.tensor(lens, dtype=torch.int32))
        a[0].copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(P)))
        graph.replay()
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 0
        c.lens = torch.tensor(lens, dtype=torch.int32)
        _check(c, a[0], o, lse, 128 ** -0.5)


def test_streams_and_calls_in_a_row(cuda_device, fa2_lib):
    """Calls that follow each other, among the cache's other ones, give the bits of calls
    one by one; and on other streams."""
    cs = [Shared(B, 2, 64, 16, P, [P + n for n in range(B)], FP16, seed=B) for B, P in ((2, 3000), (70, 200), (9, 16))]
    qs = [c.query(4) for c in cs]
    args = [c.args(q, c.B == 70) for c, q in zip(cs, qs)]
    want = []
    for a in args:
        want.append(fa2_lib.prefix_decode(*a))
        torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for a in args:
            got.append(fa2_lib.prefix_decode(*a))
            fa2_lib.paged_decode(*a[:5])
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = []
    for s, a in zip(streams, args):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
            a[0].mul_(2.0)
            out.append(fa2_lib.prefix_decode(*a))
    torch.cuda.synchronize()
    for a, (o, lse) in zip(args, out):
        ref = fa2_lib.prefix_decode(*a)
        assert torch.equal(ref[0], o) and torch.equal(ref[1], lse)
    assert fa2_lib.device_status() == 0


def test_nothing_around_the_outputs_is_written(cuda_device, fa2_lib):
    lib = fa2_lib.load_library()
    for B, Hq, Hkv, d, P in ((3, 4, 2, 128, 300), (20, 4, 2, 64, 1000), (90, 6, 2, 64, 129)):
        c = Shared(B, Hkv, d, 16, P, [P + 5 * (b % 9) for b in range(B)], BF16, seed=1)
        a = c.args(c.query(Hq), B == 90)
        n = lib.fa2_prefix_decode_workspace_size(B, Hq, Hkv, d, 16, c.table.shape[1])
        guard = 4096
        ws = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        ob = torch.full((B * Hq * d + 2 * guard,), 3.0, dtype=BF16, device="cuda")
        lb = torch.full((B * Hq + 2 * guard,), 3.0, device="cuda")
        o, lse = ob[guard:-guard].view(B, Hq, d), lb[guard:-guard].view(B, Hq)
        fa2_lib.prefix_decode(*a, out=o, lse=lse, workspace=ws[guard:-guard])
        want = fa2_lib.prefix_decode(*a)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        for x, v in ((ws, 0xA5), (ob, 3.0), (lb, 3.0)):
            assert (x[:guard] == v).all() and (x[-guard:] == v).all()


def test_refusals(cuda_device, fa2_lib):
    c = Shared(2, 2, 64, 16, 20, [25, 33], BF16, seed=0, width=4)
    q = c.query(4)
    a = c.args(q)
    names = ("q", "k_cache", "v_cache", "table", "lens", "prefix", "prefix_len")
    base = dict(zip(names, a))
    for bad in (dict(q=a[0].half()), dict(q=a[0][0]), dict(q=a[0].cpu()), dict(k_cache=a[1].float()), dict(v_cache=a[2][:-1]),
                dict(table=a[3].long()), dict(lens=a[4][:1]), dict(prefix=a[5].long()), dict(prefix=a[3]),
                dict(prefix=a[5].cpu()), dict(prefix_len=a[4]), dict(prefix_len=20), dict(out=a[0].float()),
                dict(lse=torch.zeros(2, 4)), dict(workspace=torch.zeros(8))):
        with pytest.raises((ValueError, TypeError)):
            fa2_lib.prefix_decode(**{**base, **bad})
    for bad, code in ((dict(q=a[0][:, :3].contiguous()), 1), (dict(scale=0.0), 1), (dict(out=a[0]), 8),
                      (dict(prefix=a[5][:0]), 1),
                      (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), 7)):
        with pytest.raises(fa2_lib.FA2Error) as e:
            fa2_lib.prefix_decode(**{**base, **bad})
        assert e.value.code == code
