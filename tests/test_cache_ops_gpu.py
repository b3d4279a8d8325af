"""Append to and eviction from a paged cache: copies, so bit for bit."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, FP16, Cache

pytestmark = pytest.mark.gpu


def _raw(t):
    """16-bit values as integers, so that NaN compares."""
    return t.detach().cpu().view(torch.int16).numpy()


@pytest.mark.parametrize("B,Hkv,d,ps,lens,T,new", [
    (1, 1, 64, 16, [0], 1, None),
    (3, 2, 128, 16, [0, 15, 16], 1, None),
    (2, 3, 64, 5, [4, 0], 23, [23, 7]),
    (4, 1, 128, 64, [1, 60, 64, 100], 130, [0, 130, 64, 1]),
    (2, 8, 128, 24, [0, 0], 700, None),
    (65, 1, 64, 1, [3] * 65, 2, None),
])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_append(cuda_device, fa2_lib, B, Hkv, d, ps, lens, T, new, dtype):
    count = [T] * B if new is None else new
    width = max(-(-(a + b) // ps) for a, b in zip(lens, count)) + 1
    c = Cache(B, Hkv, d, ps, lens, dtype, seed=T, width=width)
    k, v = (torch.randn(B, Hkv, T, d, generator=c.g).to(dtype) for _ in range(2))
    w, nw = c.weights(), torch.rand(B, Hkv, T, generator=c.g)
    pos = torch.full(w.shape, -7, dtype=torch.int32)
    start = torch.tensor([100 + 3 * b for b in range(B)], dtype=torch.int32)
    kc, vc, table, ln = c.gpu()
    wg, pg = w.cuda(), pos.cuda()
    num = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    out = fa2_lib.cache_append(k.cuda(), v.cuda(), kc, vc, table, ln, num_new=num, weights=wg,
                               new_weights=nw.cuda(), positions=pg, next_pos=start.cuda())
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    assert out.tolist() == [a + b for a, b in zip(lens, count)] and ln.tolist() == list(lens)
    t = c.table.numpy()
    assert (_raw(kc) == oc.cache_append(_raw(k), _raw(c.k), t, lens, count)).all()
    assert (_raw(vc) == oc.cache_append(_raw(v), _raw(c.v), t, lens, count)).all()
    for b in range(B):
        w[b, :, lens[b]:lens[b] + count[b]] = nw[b, :, :count[b]]
        pos[b, :, lens[b]:lens[b] + count[b]] = start[b] + torch.arange(count[b], dtype=torch.int32)
    assert torch.equal(wg.cpu(), w) and torch.equal(pg.cpu(), pos)


def test_append_without_weights_and_with_fresh_ones(cuda_device, fa2_lib):
    c = Cache(2, 2, 64, 16, [3, 30], BF16, seed=1, width=3)
    k, v = (torch.randn(2, 2, 1, 64, generator=c.g).to(BF16) for _ in range(2))
    kc, vc, table, lens = c.gpu()
    w = c.weights()
    wg = w.cuda()
    a = fa2_lib.cache_append(k.cuda(), v.cuda(), kc, vc, table, lens)
    k1 = kc.clone()
    b = fa2_lib.cache_append(k.cuda(), v.cuda(), kc, vc, table, lens, weights=wg)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and (_raw(k1) == _raw(kc)).all()
    w[0, :, 3] = 0
    w[1, :, 30] = 0
    assert torch.equal(wg.cpu(), w)


def test_append_drops_and_reports_what_does_not_fit(cuda_device, fa2_lib):
    c = Cache(3, 1, 64, 16, [30, 5, 9], BF16, seed=2)  # 32 slots each
    c.table[1, 0] = 999
    k, v = (torch.randn(3, 1, 4, 64, generator=c.g).to(BF16) for _ in range(2))
    kc, vc, table, lens = c.gpu()
    out = fa2_lib.cache_append(k.cuda(), v.cuda(), kc, vc, table, lens,
                               num_new=torch.tensor([4, 4, -1], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9
    assert out.tolist() == [32, 9, 9]
    want = oc.cache_append(_raw(k), _raw(c.k), c.table.numpy(), [30, 0, 0], [2, 0, 0])
    assert (_raw(kc) == want).all()


def _evict_case(B, Hkv, d, ps, lens, dtype, seed, kind, width=None):
    c = Cache(B, Hkv, d, ps, lens, dtype, seed=seed, width=width)
    w = c.weights()
    if kind == "ties":
        w = torch.randint(0, 4, w.shape, generator=c.g).float()
    elif kind == "equal":
        w = torch.full(w.shape, 0.5)
    elif kind == "odd":
        pick = torch.randint(0, 7, w.shape, generator=c.g)
        vals = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-40, -1.0])
        w = vals[pick]
    elif kind == "rising":  # everything kept has to move
        w = torch.arange(c.L, dtype=torch.float32).expand(w.shape).contiguous()
    pos = torch.stack([torch.randperm(c.L, generator=c.g) for _ in range(B * Hkv)]).view(B, Hkv, c.L)
    return c, w, pos.to(torch.int32)


def _check_evict(fa2, c, w, pos, budget, recent, in_place, with_pos):
    kc, vc, table, lens = c.gpu()
    start = c.lens + 0
    wg, pg = w.cuda(), pos.cuda() if with_pos else None
    wo = wg if in_place else torch.full_like(wg, -5.0)
    po = None if not with_pos else (pg if in_place else torch.full_like(pg, -5))
    out = fa2.cache_evict(kc, vc, table, lens, wg, budget, recent=recent, positions=pg,
                          next_pos=start.cuda() if with_pos else None,
                          weights_out=None if in_place else wo, positions_out=None if in_place else po)
    torch.cuda.synchronize()
    assert fa2.device_status() == 0
    k2, v2, w2, p2, left = oc.cache_evict(_raw(c.k), _raw(c.v), c.table.numpy(), c.lens.numpy(),
                                          w.numpy(), budget, recent,
                                          pos.numpy() if with_pos else None, start.numpy())
    assert out.tolist() == left.tolist()
    assert (_raw(kc) == k2).all() and (_raw(vc) == v2).all()
    if not in_place:  # slots past the new length are left as they were
        for b in range(c.B):
            w2[b, :, left[b]:] = -5.0
            if with_pos:
                p2[b, :, left[b]:] = -5
    assert np.array_equal(wo.cpu().numpy().view(np.int32), w2.view(np.int32))
    if with_pos:
        assert np.array_equal(po.cpu().numpy(), p2)


@pytest.mark.parametrize("B,Hkv,d,ps,lens,budget,recent", [
    (1, 1, 64, 16, [2], 1, 0),
    (1, 1, 128, 16, [33], 32, 8),
    (3, 2, 64, 16, [100, 40, 41], 40, 5),
    (2, 3, 128, 5, [333, 0], 7, 7),
    (2, 1, 64, 24, [1000, 999], 999, 100),
    (1, 2, 128, 64, [2049], 2048, 256),
    (2, 2, 64, 16, [700, 650], 1, 1),
    (1, 2, 64, 64, [5000], 1237, 100),    # past 4096 slots: a cluster
    (2, 1, 64, 128, [9001, 4500], 4400, 0),
    (1, 2, 64, 64, [5001], 5000, 10),     # one too many, in a cluster
    (1, 1, 64, 64, [40000], 20000, 100),  # keys in shared memory
    (1, 1, 64, 64, [33001], 33000, 7),
])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd", "rising"])
def test_evict(cuda_device, fa2_lib, B, Hkv, d, ps, lens, budget, recent, kind):
    seed = sum(lens) + budget
    c, w, pos = _evict_case(B, Hkv, d, ps, lens, BF16 if d == 64 else FP16, seed, kind)
    _check_evict(fa2_lib, c, w, pos, budget, recent, in_place=seed % 2 == 0, with_pos=kind != "ties")


@pytest.mark.parametrize("n", [300, 5000, 20000])
@pytest.mark.parametrize("digit", range(4))
@pytest.mark.parametrize("extra", [-1, 0, 1])
def test_evict_at_a_digit_border(cuda_device, fa2_lib, n, digit, extra):
    """A budget at, or one off, the number of weights above the border of the
    keys' `digit`-th byte: 120 of them, the others below it."""
    high, low = ((0x3F000000, 0x3E000000), (0x3F800000, 0x3F7F0000), (0x3F808000, 0x3F807F00),
                 (0x3F808001, 0x3F808000))[digit]
    c, w, pos = _evict_case(1, 2, 64, 16, [n], BF16, digit, "plain")
    free = 8 * (3 - digit)
    bits = torch.randint(0, 1 << free, w.shape, generator=c.g, dtype=torch.int32)
    for h in range(2):
        top = torch.zeros(c.L, dtype=torch.bool)
        top[torch.randperm(n, generator=c.g)[:120]] = True
        bits[0, h] += torch.where(top, high, low).to(torch.int32)
    _check_evict(fa2_lib, c, bits.view(torch.float32), pos, 120 + extra, 0, in_place=False, with_pos=True)


def test_evict_in_place_is_evict_out_of_place(cuda_device, fa2_lib):
    c, w, pos = _evict_case(2, 2, 64, 16, [900, 600], BF16, 5, "plain")
    _check_evict(fa2_lib, c, w, pos, 500, 50, in_place=True, with_pos=True)
    _check_evict(fa2_lib, c, w, pos, 500, 50, in_place=False, with_pos=True)
    _check_evict(fa2_lib, c, w, pos, 500, 50, in_place=True, with_pos=False)


def test_evict_nothing_to_do(cuda_device, fa2_lib):
    c, w, pos = _evict_case(2, 2, 64, 16, [90, 0], BF16, 6, "plain")
    for budget in (90, 96, 1000):
        _check_evict(fa2_lib, c, w, pos, budget, 3, in_place=False, with_pos=True)


def test_evict_rows_longer_than_shared_memory(cuda_device, fa2_lib):
    """More slots than a cluster's shared memory holds keys for."""
    n, d = 8 * 49152 + 5000, 64
    ps, budget = 4096, 1000
    pages = -(-n // ps)
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.rand(1, 1, pages * ps, generator=g, device="cuda")
    kc = torch.empty(pages, 1, ps, d, dtype=BF16, device="cuda")
    mark = torch.arange(pages * ps, device="cuda")
    kc[:] = (mark % 251).to(BF16).view(pages, 1, ps, 1)
    vc = torch.empty_like(kc)
    vc[:] = (mark // 251 % 251).to(BF16).view(pages, 1, ps, 1)
    k0, v0 = kc.clone().view(-1, d), vc.clone().view(-1, d)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    wo = torch.zeros_like(w)
    out = fa2_lib.cache_evict(kc, vc, table, lens, w, budget, recent=10, weights_out=wo)
    torch.cuda.synchronize()
    assert out.tolist() == [budget] and fa2_lib.device_status() == 0
    first = np.arange(n) >= n - 10
    place = torch.tensor(oc.evict_places(w[0, 0].cpu().numpy(), n, budget, first), device="cuda")
    assert torch.equal(wo[0, 0, :budget], w[0, 0][place])
    assert torch.equal(kc.view(-1, d)[:budget], k0[place])
    assert torch.equal(vc.view(-1, d)[:budget], v0[place])
    assert torch.equal(kc.view(-1, d)[budget:], k0[budget:])


def test_evict_reports_bad_pages(cuda_device, fa2_lib):
    c, w, pos = _evict_case(1, 1, 64, 16, [64], BF16, 7, "rising")
    kc, vc, table, lens = c.gpu()
    table[0, 0] = -4
    before = _raw(kc)
    out = fa2_lib.cache_evict(kc, vc, table, lens, w.cuda(), 16)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9 and out.tolist() == [16]
    assert (_raw(kc) == before).all()  # the destinations lie in the bad page: nothing moved


def test_evict_in_a_graph(cuda_device, fa2_lib):
    c, w, pos = _evict_case(2, 2, 128, 16, [400, 390], BF16, 8, "plain")
    kc, vc, table, lens = c.gpu()
    k0, v0, wg = kc.clone(), vc.clone(), w.cuda()
    wo = torch.zeros_like(wg)
    call = lambda: fa2_lib.cache_evict(kc, vc, table, lens, wg, 256, recent=20, weights_out=wo)  # noqa: E731
    call()
    torch.cuda.synchronize()
    kc.copy_(k0), vc.copy_(v0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for n in ([400, 390], [256, 300], [10, 0]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        kc.copy_(k0), vc.copy_(v0), wo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        k2, _, w2, _, left = oc.cache_evict(_raw(k0), _raw(v0), c.table.numpy(), n, w.numpy(), 256, 20)
        assert (_raw(kc) == k2).all() and out.tolist() == left.tolist()
        for b in range(2):
            assert np.array_equal(wo[b, :, :left[b]].cpu().numpy(), w2[b, :, :left[b]])
            assert (wo[b, :, left[b]:] == 0).all()
