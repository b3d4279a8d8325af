"""Appends whose slots would not fit in 31 bits."""

import pytest
import torch

from tests.cache_cases import BF16

pytestmark = pytest.mark.gpu


def test_a_prompt_longer_than_the_table(cuda_device, fa2_lib):
    """2^30 + 64 tokens behind 2^30 - 3 slots of 2^30: three fit, the others, whose
    slots run past 2^31, are dropped and reported. (137 GB of keys, of which three
    rows are read.)"""
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of free device memory")
    ps, d, T = 1 << 20, 64, (1 << 30) + 64
    k = torch.empty(1, 1, T, d, dtype=BF16, device="cuda")
    k[0, 0, :3] = torch.arange(3 * d, device="cuda").view(3, d).to(BF16)
    kc, vc = (torch.zeros(2, 1, ps, d, dtype=BF16, device="cuda") for _ in range(2))
    table = torch.zeros(1, 1024, dtype=torch.int32, device="cuda")
    table[0, 1023] = 1
    lens = torch.tensor([(1 << 30) - 3], dtype=torch.int32, device="cuda")
    out = fa2_lib.cache_append(k, k, kc, vc, table, lens)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 9
    assert out.tolist() == [1 << 30]
    for c in (kc, vc):
        assert torch.equal(c[1, 0, -3:], k[0, 0, :3])
        assert not c[0].any() and not c[1, 0, :-3].any()
    del k, kc, vc
    torch.cuda.empty_cache()
