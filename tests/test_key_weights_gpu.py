"""Accumulated attention weight of a prompt's keys, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, FP16, bits64

pytestmark = pytest.mark.gpu


def _inputs(B, Hq, Hkv, N, Nk, d, dtype, causal, seed, std=1.0, scale=None):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, Hq, N, d, generator=g) * std).to(dtype)
    k = torch.randn(B, Hkv, Nk, d, generator=g).to(dtype)
    scale = scale or d ** -0.5
    s = scale * (q.double() @ k.double().repeat_interleave(Hq // Hkv, 1).transpose(-1, -2))
    if causal:
        s = s.masked_fill(torch.ones(N, Nk, dtype=torch.bool).triu(1), -float("inf"))
    return q, k, torch.logsumexp(s, -1).float(), scale


def _check(fa2, q, k, lse, causal, scale, q_lens=None, real_keys=None):
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda()
    w = fa2.key_weights(q.cuda(), k.cuda(), lse.cuda(), causal=causal, scale=scale, q_lens=ql)
    torch.cuda.synchronize()
    assert fa2.device_status() == 0
    q64, k64, l64 = bits64(q), bits64(k), bits64(lse)
    ref = oc.key_weights(q64, k64, l64, causal, scale, q_lens)
    d, n = q.shape[-1], q.shape[2] * (q.shape[1] // k.shape[1])
    # A score: d fp32 products and their sum, off by at most (d + 8) half steps
    # of the sum of magnitudes; L log2(e) by two half steps; exp2 by 2^-22; a sum
    # of n terms of one sign by n half steps of itself.
    big = scale * float((np.abs(np.nan_to_num(q64)).max((0, 1, 2)) * np.abs(np.nan_to_num(k64)).max((0, 1, 2))).sum())
    top = float(np.abs(np.where(np.isfinite(l64), l64, 0)).max())
    rel = ((d + 8) * big + 4 * top + 4 + n) * 2.0 ** -24
    got = bits64(w)
    err = np.abs(got - ref)
    assert (err <= ref * rel + 1e-30).all(), float(np.max(err / np.maximum(ref, 1e-30)))
    return w


@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,d", [
    (1, 1, 1, 1, 1, 64),
    (1, 2, 2, 127, 127, 128),
    (2, 3, 3, 129, 129, 64),
    (1, 4, 2, 256, 256, 128),
    (1, 1, 1, 257, 257, 64),
    (2, 6, 2, 640, 640, 128),
    (1, 2, 1, 1000, 1000, 64),
    (1, 1, 1, 300, 700, 128),     # keys that no causal query sees
    (1, 1, 1, 700, 300, 64),
    (3, 8, 1, 65, 65, 128),
    (40, 8, 4, 130, 130, 64),     # several items per CTA
    (1, 1, 1, 5000, 5000, 64),    # items cut over many CTAs
])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_key_weights(cuda_device, fa2_lib, B, Hq, Hkv, N, Nk, d, causal, dtype):
    q, k, lse, scale = _inputs(B, Hq, Hkv, N, Nk, d, dtype, causal, seed=N + Hq)
    _check(fa2_lib, q, k, lse, causal, scale)


@pytest.mark.parametrize("std,scale", [(8.0, None), (0.0, None), (1.0, 1e-5)])
def test_key_weights_sharp_and_flat_rows(cuda_device, fa2_lib, std, scale):
    q, k, lse, scale = _inputs(1, 2, 2, 400, 400, 128, BF16, True, 1, std, scale)
    _check(fa2_lib, q, k, lse, True, scale)


@pytest.mark.parametrize("lens", [[300, 1, 0, 128], [0, 0, 0, 0], [129, 300, 256, 255]])
def test_key_weights_of_a_padded_batch(cuda_device, fa2_lib, lens):
    """Padded rows hold NaN; padded keys come out as 0."""
    q, k, lse, scale = _inputs(4, 4, 2, 300, 300, 64, BF16, True, 2)
    for b, n in enumerate(lens):
        q[b, :, n:] = float("nan")
        k[b, :, n:] = float("nan")
        lse[b, :, n:] = float("nan")
    w = fa2_lib.key_weights(q.cuda(), k.cuda(), lse.cuda(), causal=True,
                            q_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    for b, n in enumerate(lens):
        assert (w[b, :, n:] == 0).all()
        if n:
            _check(fa2_lib, q[b:b + 1, :, :n].contiguous(), k[b:b + 1, :, :n].contiguous(),
                   lse[b:b + 1, :, :n].contiguous(), True, scale)
            part = fa2_lib.key_weights(q[b:b + 1, :, :n].contiguous().cuda(),
                                       k[b:b + 1, :, :n].contiguous().cuda(),
                                       lse[b:b + 1, :, :n].contiguous().cuda(), causal=True)
            assert torch.allclose(w[b:b + 1, :, :n], part, rtol=n * 2.0 ** -23, atol=0)


def test_key_weights_follow_the_forward_and_repeat(cuda_device, fa2_lib):
    B, H, N, d = 2, 4, 1500, 128
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(B, H, N, d, generator=g).to(BF16).cuda() for _ in range(3))
    _, lse = fa2_lib.forward(q, k, v, causal=True)
    w = fa2_lib.key_weights(q, k, lse, causal=True)
    for _ in range(3):
        assert torch.equal(w, fa2_lib.key_weights(q, k, lse, causal=True))
    # Rows of the attention matrix sum to one: over all keys the weights are N,
    # up to the forward's error in L (tested at 2e-3 on bf16) on every row.
    assert torch.allclose(w.double().sum(-1), torch.full((B, H), float(N), dtype=torch.float64, device="cuda"),
                          rtol=4e-3, atol=0)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0


def test_key_weights_in_a_graph_follows_lengths(cuda_device, fa2_lib):
    q, k, lse, scale = _inputs(2, 4, 2, 600, 600, 64, FP16, True, 4)
    q, k, lse = q.cuda(), k.cuda(), lse.cuda()
    ql = torch.tensor([600, 333], dtype=torch.int32).cuda()
    fa2_lib.key_weights(q, k, lse, causal=True, q_lens=ql)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w = fa2_lib.key_weights(q, k, lse, causal=True, q_lens=ql)
    for n in ([600, 333], [1, 600], [0, 0]):
        ql.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        want = fa2_lib.key_weights(q, k, lse, causal=True, q_lens=ql)
        torch.cuda.synchronize()
        assert torch.equal(w, want)


def test_key_weights_of_rows_without_weight(cuda_device, fa2_lib):
    """L = +inf gives a query no weight, as e^(s - L) does."""
    q, k, lse, scale = _inputs(1, 2, 1, 300, 300, 64, BF16, False, 5)
    lse[0, 0, 10:140] = float("inf")
    lse[0, 1, 299] = float("inf")
    _check(fa2_lib, q, k, lse, False, scale)


def test_key_weights_timeout_path(cuda_device, fa2_lib):
    """A Q tile that never arrives: the bounded wait runs out, the status says so,
    and the next call is correct."""
    q, k, lse, scale = _inputs(1, 2, 2, 700, 700, 128, BF16, True, 6)
    assert fa2_lib.load_library().fa2_debug_arm_fault(6, 20) == 0
    fa2_lib.key_weights(q.cuda(), k.cuda(), lse.cuda(), causal=True)
    assert fa2_lib.device_status() == 6
    assert fa2_lib.device_status() == 0
    _check(fa2_lib, q, k, lse, True, scale)
