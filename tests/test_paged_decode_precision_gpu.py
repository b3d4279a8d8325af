"""What the decode's output carries: the one rounding at its end, and no rounding
of the probabilities that would show through it."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, FP16, Cache, bits64

pytestmark = pytest.mark.gpu


def _sink(d, ps, n, gap, dtype, sink_at=0):
    """One slot whose score lies `gap` log2 units above all others and whose V is
    0; the others have one score, and V of one sign. (q, cache, scale, q.k of the
    sink): the scores are exact."""
    c = Cache(1, 1, d, ps, [n], dtype, seed=n, nan=False)
    flat_k, flat_v = c.k.view(-1, d), c.v.view(-1, d)
    j = torch.arange(n)
    rows = c.table[0].long()[j // ps] * ps + j % ps
    flat_k[rows] = 0
    flat_k[rows[sink_at], 0] = 1.0
    flat_v[rows] = (1.0 + torch.rand(n, d, generator=c.g)).to(dtype)
    flat_v[rows[sink_at]] = 0
    q = torch.zeros(1, 1, d, dtype=dtype)
    q[0, 0, 0] = 1.0
    return c, q, gap * float(np.log(2.0))


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("gap", [20.0, 23.1, 25.2, 26.0, 31.5])
@pytest.mark.parametrize("d,ps,n,width", [(128, 16, 4096, 256), (64, 64, 4096, 64), (128, 16, 500, 32),
                                          (64, 16, 30, 2)])
def test_slots_far_below_the_largest_count(cuda_device, fa2_lib, dtype, gap, d, ps, n, width):
    """p of every slot but one is 2^-gap of the largest's: they are all that the
    output is made of."""
    c, q, scale = _sink(d, ps, n, gap, dtype, sink_at=n // 3)
    c.v *= 256  # so that the output stays a normal number in fp16
    kc, vc, table, lens = c.gpu()
    w = torch.zeros(1, 1, c.L, device="cuda")
    o, lse = fa2_lib.paged_decode(q.cuda(), kc, vc, table, lens, scale=scale, weights=w)
    o2, _ = fa2_lib.paged_decode(q.cuda(), kc, vc, table, lens, scale=scale)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    scale = float(np.float32(scale))
    ref, lref, p = oc.paged_decode(bits64(q), bits64(c.k), bits64(c.v), c.table.numpy(), c.lens.numpy(), scale)
    # The score times scale * log2(e) is a rounding of the factor (2^-24 of it) and
    # one of the product, each at most gap * 2^-24 log2 units: ln 2 of that in p;
    # exp2 2^-22. Up to n/4 terms of one sign in a warp, added 8 or 16 at a time by
    # instructions that may cut the sum (2^-23 each), then 40 further roundings.
    rel = gap * 2 * 2.0 ** -24 * 0.7 + 2.0 ** -22 + (n / 32 + 40) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * half  # half a step of a subnormal
    for got in (o, o2):
        err = np.abs(bits64(got) - ref)
        assert (err <= np.abs(ref) * (half * 1.01 + rel + 2.0 ** -19) + tiny).all(), np.max(err / np.abs(ref))
    want = p[0]
    assert (np.abs(bits64(w[0, :, :n]) - want) <= want * (rel + 2.0 ** -20)).all()


def _scale_of(gap):
    """A float32 near gap * ln 2 whose product with log2(e) is a float32 but for
    2^-28 of itself, so that the kernel's factor is the exact one."""
    f = np.float32(gap * np.log(2.0))
    while True:
        x = float(f) / np.log(2.0)
        if abs(float(np.float32(x)) / x - 1) < 2.0 ** -28:
            return float(f)
        f = np.nextafter(f, np.float32(100))


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("gap", [1.96, 3.96, 9.96, 11.95])
def test_rounded_once(cuda_device, fa2_lib, dtype, gap):
    """16 slots, one with a score `gap` log2 units above the others and V = 0. Every
    output that does not lie at a border between two steps is the rounded exact
    value. (At these gaps two bf16 numbers are 2^-17.2 off p, and two fp16 numbers,
    at the last two, 2^-15.4 and 2^-13.3.)"""
    B, H, d = 64, 16, 128
    c = Cache(B, H, d, 16, [16] * B, dtype, seed=int(gap * 100))
    c.k[:] = 0
    c.v[:] = (1.0 + torch.rand(c.v.shape, generator=c.g)).to(dtype)
    b = torch.arange(B)
    sink = torch.randint(0, 16, (B,), generator=c.g)
    page = c.table[:, 0].long()
    c.k[page[b], :, sink, 0] = 1.0
    c.v[page[b], :, sink] = 0.0
    q = torch.zeros(B, H, d, dtype=dtype)
    q[:, :, 0] = 1.0
    kc, vc, table, lens = c.gpu()
    scale = _scale_of(gap)
    o, _ = fa2_lib.paged_decode(q.cuda(), kc, vc, table, lens, scale=scale)
    torch.cuda.synchronize()
    e = np.exp(-scale)
    ref = bits64(c.v)[page.numpy()].sum(2) * (e / (1.0 + 15.0 * e))
    # Score and factor are exact; exp2 is good to 2^-22; 15 terms of one sign are
    # added by up to four instructions that may each cut 2^-23; the sum of p, its
    # reciprocal and the last product are off by 5, 2 and 1 half steps (2^-24); fp16
    # keeps p as two numbers of 11 bits: 2^-21.
    rel = 2.0 ** -28 * gap + 2.0 ** -22 + 4 * 2.0 ** -23 + 8 * 2.0 ** -24 + (2.0 ** -21 if dtype == FP16 else 0)
    assert rel < 2.0 ** -18.5
    sure = torch.from_numpy(ref * (1 - rel)).to(dtype) == torch.from_numpy(ref * (1 + rel)).to(dtype)
    assert sure.float().mean() > 0.99
    near = torch.from_numpy(ref).to(dtype)
    wrong = (o.cpu() != near) & sure
    assert not wrong.any(), int(wrong.sum())


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n,width", [(30, 4), (600, 80), (3000, 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_come_out_infinite(cuda_device, fa2_lib, dtype, n, width, d):
    """A V entry of +-inf makes its element of o +-inf, as p * inf does; both signs
    in one column, or NaN, make NaN; all other elements are as without it."""
    c = Cache(2, 2, d, 16, [n, n - 1], dtype, seed=n, width=width)
    kc, vc, table, lens = c.gpu()
    q = c.query(8).cuda()
    bad = vc.clone()

    def at(b, j):
        return int(c.table[b, j // 16]), j % 16

    p, s = at(0, n // 2)
    bad[p, 1, s, 3] = float("inf")
    bad[p, 1, s, 7] = -float("inf")
    bad[p, 1, s, d - 1] = -float("inf")
    p, s = at(0, n - 1)
    bad[p, 1, s, d - 1] = float("inf")
    p, s = at(1, 5)
    bad[p, 0, s, 1] = float("nan")
    for weights in (None, torch.zeros(2, 2, c.L, device="cuda")):
        want, lse0 = fa2_lib.paged_decode(q, kc, vc, table, lens, weights=weights)
        o, lse = fa2_lib.paged_decode(q, kc, bad, table, lens, weights=weights)
        torch.cuda.synchronize()
        want[0, 4:, 3], want[0, 4:, 7], want[0, 4:, d - 1] = float("inf"), -float("inf"), float("nan")
        want[1, :4, 1] = float("nan")
        assert torch.equal(o.isnan(), want.isnan())
        assert torch.equal(o.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
        assert torch.equal(lse, lse0)
    assert fa2_lib.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("B,Hq,Hkv,d,n,width", [(8, 16, 4, 128, 777, 60), (4, 32, 2, 64, 500, 32),
                                                (16, 8, 8, 128, 250, 16)])
def test_error_in_the_mean(cuda_device, fa2_lib, dtype, B, Hq, Hkv, d, n, width):
    """L and the weights are 32-bit sums of 32-bit terms: their errors' rms, not the
    largest that could be. Where a weight comes from, scores are about 2 and L is
    ln n + 1/2. A score is cut at each of d / 16 steps (2^-23 of it) and rounded with
    its factor (2^-23); L is a sum of n / 32 terms a lane (2^-24 each), a logarithm,
    and four roundings of L's size (2^-24); a weight has both errors, exp2's 2^-22
    and three roundings of L's size more."""
    c = Cache(B, Hkv, d, 16, [n] * B, dtype, seed=n, width=width)
    q = c.query(Hq)
    kc, vc, table, lens = c.gpu()
    w = torch.zeros(B, Hkv, c.L, device="cuda")
    o, lse = fa2_lib.paged_decode(q.cuda(), kc, vc, table, lens, weights=w)
    torch.cuda.synchronize()
    ref, lref, p = oc.paged_decode(bits64(q), bits64(c.k), bits64(c.v), c.table.numpy(), c.lens.numpy(),
                                   float(np.float32(d ** -0.5)))
    L, score = float(np.log(n)) + 0.5, 2 * (d / 16 + 1) * 2.0 ** -23
    tol = score + (n / 32 + 4 * L) * 2.0 ** -24 + 2.0 ** -22
    rms = lambda x: float(np.sqrt(np.mean(np.square(x))))  # noqa: E731
    assert rms(bits64(lse) - lref) <= tol
    want = np.stack(p)
    assert rms(bits64(w)[:, :, :n] - want) <= (tol + score + 3 * L * 2.0 ** -24 + 2.0 ** -22) * rms(want)
    # o: its rounding's own rms, whatever came before it.
    near = bits64(torch.from_numpy(ref).to(dtype))
    assert rms(bits64(o) - ref) <= 1.0005 * rms(near - ref)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n,width", [(30, 4), (600, 80)])
def test_a_slot_that_weighs_nothing_adds_nothing(cuda_device, fa2_lib, dtype, n, width):
    """Scores of -inf beside values as large as the type has: o is exactly what the
    other slots, whose V is 0, make of it; and a slot that weighs little adds no more
    than that."""
    d = 64
    c = Cache(1, 2, d, 16, [n], dtype, seed=n, width=width)
    j = torch.arange(n)
    page, off = c.table[0].long()[j // 16], j % 16
    c.k[page, :, off], c.v[page, :, off] = 0.0, 0.0
    heavy = torch.arange(0, n, 7)
    c.k[page[heavy], 0, off[heavy], 0] = -float("inf")
    c.k[page[heavy], 1, off[heavy], 0] = -100.0
    c.v[page[heavy], :, off[heavy]] = torch.finfo(dtype).max
    kc, vc, table, lens = c.gpu()
    q = torch.zeros(1, 2, d, dtype=dtype)
    q[:, :, 0] = 1.0
    o, lse = fa2_lib.paged_decode(q.cuda(), kc, vc, table, lens, scale=0.5)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    assert (o[0, 0] == 0).all()
    light = n - len(heavy)
    # e^-50 of each heavy one; what is left out of p or added to it is below 2^-20 of it.
    want = len(heavy) * np.exp(-50.0) * torch.finfo(dtype).max / light
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert (np.abs(bits64(o[0, 1]) - want) <= want * (torch.finfo(dtype).eps + 2.0 ** -12) + tiny).all()
    assert abs(float(lse[0, 0]) - np.log(light)) < 1e-5
