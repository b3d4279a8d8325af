"""Attention of one new token over a paged cache, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, FP16, Cache, bits64, decode_bounds, score_error

pytestmark = pytest.mark.gpu

# B, Hq, Hkv, d, page size, lengths
CASES = [
    (1, 1, 1, 64, 16, [1]),
    (1, 8, 8, 128, 16, [513]),
    (6, 4, 4, 128, 16, [0, 1, 63, 64, 65, 300]),
    (3, 6, 2, 64, 5, [7, 129, 0]),
    (2, 24, 3, 128, 24, [1000, 17]),
    (2, 9, 1, 64, 64, [200, 333]),        # nine heads share a key head: two of 8, a tile of 16
    (2, 32, 2, 128, 32, [130, 511]),
    (1, 17, 1, 128, 16, [700]),           # more than one head tile
    (2, 66, 2, 64, 128, [260, 5]),
    (1, 2, 2, 128, 1, [257]),             # a page per slot
    (1, 1, 1, 64, 64, [40000]),           # one row, split over every SM
    (70, 8, 4, 64, 16, None),             # more items than CTAs, several per CTA
    (5, 16, 16, 128, 48, [0, 0, 600, 0, 1]),
    (4, 5, 5, 128, 4096, [100, 4096, 4097, 3]),
    (200, 2, 1, 128, 8, [0] * 60 + [9] * 60 + [0] * 40 + [33] * 40),  # whole warps of lengths empty
    (1, 128, 1, 64, 16, [300]),           # the largest group
]


def _check(fa2, c, Hq, std, with_weights, dtype, scale=None):
    B, Hkv, d = c.B, c.Hkv, c.d
    scale = scale or d ** -0.5
    q = c.query(Hq, std)
    kc, vc, table, lens = c.gpu()
    w = c.weights()
    wg = w.cuda() if with_weights else None
    o, lse = fa2.paged_decode(q.cuda(), kc, vc, table, lens, scale=scale, weights=wg)
    torch.cuda.synchronize()
    assert fa2.device_status() == 0
    k64, v64 = bits64(c.k), bits64(c.v)
    o_ref, lse_ref, p = oc.paged_decode(bits64(q), k64, v64, c.table.numpy(), c.lens.numpy(), scale)
    # sum of p |v|: the decode of the magnitudes
    A, _, _ = oc.paged_decode(bits64(q), k64, np.abs(v64), c.table.numpy(), c.lens.numpy(), scale)
    ds = score_error(bits64(q), k64, scale)
    n = int(c.lens.max())
    tol_o, tol_l, rel = decode_bounds(o_ref, lse_ref, A, ds, n, dtype)
    assert (np.abs(bits64(o) - o_ref) <= tol_o).all(), np.max(np.abs(bits64(o) - o_ref) - tol_o)
    fin = np.isfinite(lse_ref)
    got = bits64(lse)
    assert (got[~fin] == -np.inf).all()
    assert (np.abs(got - np.where(fin, lse_ref, 0))[fin] <= tol_l[fin]).all()
    if with_weights:
        want = bits64(w)
        for b in range(B):
            m = int(c.lens[b])
            want[b, :, :m] += p[b]
        tol = np.zeros_like(want)
        for b in range(B):
            m = int(c.lens[b])
            tol[b, :, :m] = p[b] * rel + 2.0 ** -23 * want[b, :, :m]
        assert (np.abs(bits64(wg) - want) <= tol).all()  # past the length: not touched
    return o, lse, wg


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c[:5])))
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
def test_decode_matches_the_oracle(cuda_device, fa2_lib, case, dtype, weights):
    B, Hq, Hkv, d, ps, lens = case
    if lens is None:
        lens = np.random.default_rng(B).integers(0, 150, B)
    c = Cache(B, Hkv, d, ps, lens, dtype, seed=Hq + ps)
    _check(fa2_lib, c, Hq, 1.0, weights, dtype)


@pytest.mark.parametrize("std,scale", [(12.0, None), (0.0, None), (1.0, 1e-6), (3.0, 2.0)])
def test_decode_sharp_and_flat_rows(cuda_device, fa2_lib, std, scale):
    c = Cache(2, 2, 128, 16, [777, 130], BF16, seed=3)
    _check(fa2_lib, c, 8, std, True, BF16, scale)


def test_decode_repeats_bit_for_bit_on_any_stream(cuda_device, fa2_lib):
    c = Cache(3, 4, 128, 16, [2000, 5, 900], BF16, seed=4)
    kc, vc, table, lens = c.gpu()
    q, w = c.query(16).cuda(), c.weights().cuda()
    first = None
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            w_out = torch.zeros_like(w)
            o, lse = fa2_lib.paged_decode(q, kc, vc, table, lens, weights=w, weights_out=w_out)
            got.append((o, lse, w_out))
    torch.cuda.synchronize()
    for t in got:
        first = first or t
        assert all(torch.equal(a, b) for a, b in zip(t, first))


def test_decode_in_a_graph_follows_lengths_and_pages(cuda_device, fa2_lib):
    c = Cache(3, 2, 64, 16, [600, 64, 333], BF16, seed=5, width=40)
    kc, vc, table, lens = c.gpu()
    q, w = c.query(6).cuda(), c.weights().cuda()
    w_out = torch.zeros_like(w)
    call = lambda wo: fa2_lib.paged_decode(q, kc, vc, table, lens, weights=w, weights_out=wo)  # noqa: E731
    call(w_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call(w_out)
    for new in ([600, 64, 333], [1, 0, 12], [0, 0, 0], [599, 2, 300]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        table.copy_(table.roll(0, 0))
        w_out.zero_()
        graph.replay()
        eager_w = torch.zeros_like(w)
        eo, el = call(eager_w)
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(lse, el) and torch.equal(w_out, eager_w)
    assert fa2_lib.device_status() == 0


def test_decode_shared_prefix_pages_are_counted_apart(cuda_device, fa2_lib):
    c = Cache(2, 1, 64, 16, [160, 160], FP16, seed=6)
    c.table[1, :5] = c.table[0, :5]
    _check(fa2_lib, c, 3, 1.0, True, FP16)


def test_decode_leaves_bad_pages_out_and_reports_them(cuda_device, fa2_lib):
    c = Cache(2, 2, 64, 16, [100, 90], BF16, seed=7)
    table = c.table.clone()
    table[0, 2] = -1
    table[1, :] = c.k.shape[0]  # nothing of the second sequence is in the cache
    kc, vc, _, lens = c.gpu()
    q, w = c.query(4), c.weights()
    wg = w.cuda()
    o, lse = fa2_lib.paged_decode(q.cuda(), kc, vc, table.cuda(), lens, weights=wg)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9
    assert fa2_lib.device_status() == 0
    see = [np.ones(100, bool), np.zeros(90, bool)]
    see[0][32:48] = False
    ref, lref, p = oc.paged_decode(bits64(q), bits64(c.k), bits64(c.v), c.table.numpy(), c.lens.numpy(),
                                   64 ** -0.5, visible=see)
    A, _, _ = oc.paged_decode(bits64(q), bits64(c.k), np.abs(bits64(c.v)), c.table.numpy(),
                              c.lens.numpy(), 64 ** -0.5, visible=see)
    tol_o, tol_l, rel = decode_bounds(ref, lref, A, score_error(bits64(q), bits64(c.k), 64 ** -0.5), 100, BF16)
    assert (np.abs(bits64(o) - ref) <= tol_o).all()
    assert (np.abs(bits64(lse)[0] - lref[0]) <= tol_l[0]).all() and (bits64(lse)[1] == -np.inf).all()
    assert (o[1] == 0).all()
    want = bits64(w)
    want[0, :, :100] += p[0]
    assert (np.abs(bits64(wg) - want) <= want * 2.0 ** -22 + rel).all()
    assert torch.equal(wg[1].cpu(), w[1])
    assert torch.equal(wg[0, :, 32:48].cpu(), w[0, :, 32:48])


def test_decode_cuts_lengths_to_the_table(cuda_device, fa2_lib):
    c = Cache(3, 1, 64, 16, [64, 10, 33], BF16, seed=8, nan=False)
    kc, vc, table, lens = c.gpu()
    q = c.query(2).cuda()
    bad = torch.tensor([65, -3, 2**31 - 1], dtype=torch.int32, device="cuda")
    cut = torch.tensor([64, 0, 64], dtype=torch.int32, device="cuda")
    o, lse = fa2_lib.paged_decode(q, kc, vc, table, bad)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9
    o2, lse2 = fa2_lib.paged_decode(q, kc, vc, table, cut)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa2_lib.device_status() == 0


def test_decode_offsets_past_32_bits(cuda_device, fa2_lib):
    """A cache of 2^33 bytes and more per tensor; the sequence lies at its end."""
    d, ps, n = 128, 256, 700
    pages = (1 << 25) // ps + 64
    kc = torch.empty(pages, 1, ps, d, dtype=BF16, device="cuda")
    vc = torch.empty(pages, 1, ps, d, dtype=BF16, device="cuda")
    c = Cache(1, 1, d, ps, [n], BF16, seed=9)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32)
    for p in range(3):
        kc[table[0, p]] = c.k[c.table[0, p]].cuda()
        vc[table[0, p]] = c.v[c.table[0, p]].cuda()
    q = c.query(2).cuda()
    o, lse = fa2_lib.paged_decode(q, kc, vc, table.cuda(), c.lens.cuda())
    ks, vs, ts, ls = c.gpu()
    o2, lse2 = fa2_lib.paged_decode(q, ks, vs, ts, ls)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_lets_nan_and_infinities_through(cuda_device, fa2_lib):
    """A NaN key makes its heads NaN, L too; a key with a score of -inf weighs
    nothing; other heads and sequences do not notice."""
    c = Cache(3, 2, 64, 16, [100, 100, 100], BF16, seed=10)
    kc, vc, table, lens = c.gpu()
    q = c.query(4).cuda().abs()
    want_o, want_l = fa2_lib.paged_decode(q, kc, vc, table, lens)
    page, off = int(c.table[0, 2]), 5
    kc[page, 1, off] = float("nan")
    kc[int(c.table[1, 0]), 0, 3] = -float("inf")
    w = torch.zeros(3, 2, c.L, device="cuda")
    o, lse = fa2_lib.paged_decode(q, kc, vc, table, lens, weights=w)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all() and w[0, 1, :100].isnan().all()
    assert torch.equal(o[0, :2], want_o[0, :2]) and torch.equal(o[2], want_o[2]) and torch.equal(lse[2], want_l[2])
    assert torch.equal(o[1, 2:], want_o[1, 2:])
    assert o[1].isfinite().all() and lse[1].isfinite().all() and w[1, 0, 3] == 0
    see = [np.ones(100, bool) for _ in range(3)]
    see[1][3] = False
    ref, lref, _ = oc.paged_decode(bits64(q), bits64(c.k), bits64(c.v), c.table.numpy(), c.lens.numpy(), 64 ** -0.5,
                                   visible=see)
    assert (np.abs(bits64(lse)[1, :2] - lref[1, :2]) < 1e-4).all()
