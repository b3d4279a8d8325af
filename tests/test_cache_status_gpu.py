"""The device status word when several things went wrong since it was last read."""

import pytest
import torch

from tests.cache_cases import BF16, Cache

pytestmark = pytest.mark.gpu


def _time_out(fa2):
    """A key-weights call whose bounded wait runs out (the fault is armed on the host)."""
    q = torch.zeros(1, 2, 300, 64, dtype=BF16, device="cuda")
    assert fa2.load_library().fa2_debug_arm_fault(6, 20) == 0
    fa2.key_weights(q, q.clone(), torch.zeros(1, 2, 300, device="cuda"), causal=True)


def _bad_page(fa2, op):
    c = Cache(2, 2, 64, 16, [40, 33], BF16, seed=1, nan=False)
    c.table[1, 0] = -1
    kc, vc, table, lens = c.gpu()
    if op == "decode":
        fa2.paged_decode(c.query(4).cuda(), kc, vc, table, lens)
    elif op == "length":
        fa2.paged_decode(c.query(4).cuda(), kc, vc, c.table.clamp(min=0).cuda(), lens + 1000)
    elif op == "append":
        new = torch.zeros(2, 2, 1, 64, dtype=BF16, device="cuda")
        fa2.cache_append(new, new, kc, vc, table, lens * 0)
    else:
        w = torch.arange(c.L, dtype=torch.float32, device="cuda").expand(2, 2, c.L).contiguous()
        fa2.cache_evict(kc, vc, table, lens, w, 8)


@pytest.mark.parametrize("op", ["decode", "length", "append", "evict"])
def test_a_page_report_does_not_replace_a_timeout(cuda_device, fa2_lib, op):
    _bad_page(fa2_lib, op)
    assert fa2_lib.device_status() == 9
    _time_out(fa2_lib)
    _bad_page(fa2_lib, op)
    assert fa2_lib.device_status() == 6
    assert fa2_lib.device_status() == 0
    _bad_page(fa2_lib, op)
    _time_out(fa2_lib)
    assert fa2_lib.device_status() == 6
    assert fa2_lib.device_status() == 0
