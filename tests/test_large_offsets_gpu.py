"""Elements past 2^31 and bytes past 2^32: the rotary passes over tensors of that size,
and a cache whose pages lie there."""

import pytest
import torch

from tests.cache_cases import BF16

pytestmark = pytest.mark.gpu


def test_rotary(cuda_device, fa2_lib):
    B, H, N, d = 2, 35, 262144, 128  # 2.3e9 elements
    x = torch.zeros(B, N, H, d, dtype=BF16, device="cuda").transpose(1, 2)
    f = fa2_lib.rotary_frequencies(d).cuda()
    g = torch.Generator(device="cuda").manual_seed(0)
    for b, h in ((0, 0), (1, 34)):
        x[b, h] = torch.randn(N, d, generator=g, device="cuda").to(BF16)
    w = torch.rand(d, generator=g, device="cuda")
    for kw in ({}, {"q_weight": w}):
        y, _ = fa2_lib.rotary_forward(x, None, f, **kw)
        for b, h in ((0, 0), (1, 34)):
            want, _ = fa2_lib.rotary_forward(x[b:b + 1, h:h + 1], None, f, **kw)
            assert torch.equal(y[b, h], want[0, 0])
        assert not y[1, 33].any() and not y[0, 1].any()
    dx, _, dw, _ = fa2_lib.rotary_backward(y, None, f, q=x, q_weight=w)
    want, _, _, _ = fa2_lib.rotary_backward(y[1:, 34:], None, f, q=x[1:, 34:], q_weight=w)
    assert torch.equal(dx[1, 34], want[0, 0]) and torch.isfinite(dw).all()
    assert fa2_lib.device_status() == 0


def test_prefix_decode(cuda_device, fa2_lib):
    ps, d, Hkv, P = 16, 128, 2, 1000
    pages = 2 ** 31 // (ps * d * Hkv) + 200
    kc, vc = (torch.empty(pages, Hkv, ps, d, dtype=BF16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    for B in (4, 100):
        used = torch.arange(pages - 70 - B, pages, device="cuda").int()  # all past 2^31 elements
        kc[-200:] = torch.randn(200, Hkv, ps, d, generator=g, device="cuda").to(BF16)
        vc[-200:] = torch.randn(200, Hkv, ps, d, generator=g, device="cuda").to(BF16)
        table = torch.empty(B, 63, dtype=torch.int32, device="cuda")
        table[:, :62] = used[:62]
        table[:, 62] = used[70:70 + B]
        kc[table[1:, 62].long(), :, :8] = kc[table[0, 62].long(), :, :8]
        vc[table[1:, 62].long(), :, :8] = vc[table[0, 62].long(), :, :8]
        lens = torch.full((B,), P + 3, dtype=torch.int32, device="cuda")
        q = torch.randn(B, 8, d, generator=g, device="cuda").to(BF16)
        prefix = torch.cat([table[0], torch.full((9000,), -1, dtype=torch.int32, device="cuda")])
        plen = torch.tensor([P], dtype=torch.int32, device="cuda")
        o, lse = fa2_lib.prefix_decode(q, kc, vc, table, lens, prefix, plen)
        small = (table - (pages - 200)).contiguous()
        want, want_lse = fa2_lib.paged_decode(q, kc[-200:].contiguous(), vc[-200:].contiguous(), small, lens)
        assert (lse - want_lse).abs().max() <= 2e-5
        # each is rounded once from values that are equal to a few fp32 steps
        assert ((o.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-5).all()
    assert fa2_lib.device_status() == 0
