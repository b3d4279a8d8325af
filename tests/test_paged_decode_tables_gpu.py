"""Decode over tables of different widths: a narrow table gives each CTA a whole
(sequence, key head), a wide one an equal share of all slots."""

import numpy as np
import pytest
import torch

from tests.cache_cases import BF16, FP16, Cache
from tests.test_paged_decode_gpu import CASES, _check

pytestmark = pytest.mark.gpu


def _unit(d):
    return 64 * (128 // d)  # slots


@pytest.mark.parametrize("case", [c for c in CASES if c[5] is None or max(c[5]) < 1500],
                         ids=lambda c: "_".join(map(str, c[:5])))
@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
def test_short_lengths_in_a_wide_table(cuda_device, fa2_lib, case, weights):
    B, Hq, Hkv, d, ps, lens = case
    if lens is None:
        lens = np.random.default_rng(B).integers(0, 150, B)
    c = Cache(B, Hkv, d, ps, lens, BF16, seed=Hq + ps, width=-(-24 * _unit(d) // ps))
    _check(fa2_lib, c, Hq, 1.0, weights, BF16)


@pytest.mark.parametrize("units", [1, 4, 5, 8, 9])
@pytest.mark.parametrize("B,Hkv,g,d", [(1, 2, 4, 128), (16, 8, 2, 128), (32, 8, 1, 64), (40, 8, 1, 128),
                                       (2, 1, 24, 64)])
@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
def test_tables_of_few_units(cuda_device, fa2_lib, units, B, Hkv, g, d, weights):
    """Around the widths at which the form changes; full, ragged and empty rows."""
    L = units * _unit(d)
    lens = np.random.default_rng(units).integers(0, L + 1, B)
    lens[0] = L
    c = Cache(B, Hkv, d, 16, lens, FP16, seed=units + B, width=L // 16)
    _check(fa2_lib, c, Hkv * g, 2.0, weights, FP16)


def test_equal_share_and_whole_items_see_the_same(cuda_device, fa2_lib):
    """NaN, infinite scores and bad pages, in a narrow and in a wide table."""
    got = []
    for width in (20, 200):
        c = Cache(3, 2, 64, 16, [300, 300, 300], BF16, seed=10, width=20)
        kc, vc, table, lens = c.gpu()
        table = torch.cat([table, torch.full((3, width - 20), -7, dtype=torch.int32, device="cuda")], 1)
        q = c.query(4).cuda().abs()
        kc[int(c.table[0, 2]), 1, 5] = float("nan")
        kc[int(c.table[1, 0]), 0, 3] = -float("inf")
        table[2, 4] = -1
        table[2, 9] = kc.shape[0]
        w = torch.zeros(3, 2, width * 16, device="cuda")
        o, lse = fa2_lib.paged_decode(q, kc, vc, table.contiguous(), lens, weights=w)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 9
        assert (w[:, :, 300:] == 0).all()
        got.append((o.float(), lse, w[:, :, :300]))
    (o, lse, w), (o2, lse2, w2) = got
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all() and w[0, 1].isnan().all()
    assert (w[2, :, 64:80] == 0).all() and (w[2, :, 144:160] == 0).all() and w[1, 0, 3] == 0
    # Two roundings of values that differ by sums of 300 fp32 terms: a bf16 step
    # (2^-7 of the value), and 300 * 2^-24 of terms below 8.
    for a, b, rel in ((o, o2, 2.0 ** -7), (lse, lse2, 2.0 ** -20), (w, w2, 2.0 ** -14)):
        assert torch.equal(a.isnan(), b.isnan())
        a, b = a.nan_to_num(0.0), b.nan_to_num(0.0)
        assert ((a - b).abs() <= rel * a.abs() + 300 * 8 * 2.0 ** -24).all()


@pytest.mark.parametrize("units", [72, 80, 145, 147, 151, 154, 231])
def test_shares_of_unequal_length(cuda_device, fa2_lib, units):
    """32 items over the CTAs, shares of 7 or 8, of 15 or 16, ... units each, in a
    table with room for more."""
    n = units * 64
    c = Cache(4, 8, 128, 64, [n, n - 5, n, n - 63], BF16, seed=units, width=units + 60)
    _check(fa2_lib, c, 16, 1.0, True, BF16)


@pytest.mark.parametrize("n,width", [(300, 20), (300, 200), (3000, 200), (40000, 2500)])
def test_a_head_of_nan_keys_is_nan(cuda_device, fa2_lib, n, width):
    """Whatever the number of parts that are joined: none, few, many."""
    c = Cache(2, 2, 64, 16, [n, n], BF16, seed=n, width=width)
    kc, vc, table, lens = c.gpu()
    kc[table[0].long(), 1] = float("nan")
    w = torch.zeros(2, 2, c.L, device="cuda")
    q = c.query(2).cuda()
    o, lse = fa2_lib.paged_decode(q, kc, vc, table, lens, weights=w)
    o2, lse2 = fa2_lib.paged_decode(q, kc, vc, table, lens)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    for x, y in ((o, lse), (o2, lse2)):
        assert x[0, 1].isnan().all() and y[0, 1].isnan()
        assert x[0, 0].isfinite().all() and x[1].isfinite().all() and y[1].isfinite().all() and y[0, 0].isfinite()
    assert w[0, 1, :n].isnan().all() and w[0, 0].isfinite().all() and w[1].isfinite().all()
