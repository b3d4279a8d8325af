"""What the key weights are made of: the scale that was asked for, the forward's L,
sums in 32 bits."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, FP16, bits64

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def _scale_near(x):
    """A float32 whose product with log2(e), formed in float32, is exact but for 2^-28."""
    f = np.float32(x)
    while abs(float(f * np.float32(LOG2E)) / (float(f) * LOG2E) - 1) >= 2.0 ** -28:
        f = np.nextafter(f, np.float32(100))
    return float(f)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [20.0, 35.0, 55.0, 80.0])
def test_the_scale_is_the_one_that_was_asked_for(cuda_device, fa2_lib, d, e):
    """One query, keys of 2 against its 1: a score of 2 d scale, and L = 0. The
    product is exact, as is the score, 2 d being a power of two: what is left is
    2^-28 of an exponent of e, exp2's 2^-22, and the last rounding."""
    scale = _scale_near(e / (2 * d))
    q = torch.ones(1, 1, 1, d, dtype=BF16, device="cuda")
    k = torch.full((1, 1, 130, d), 2.0, dtype=BF16, device="cuda")
    w = fa2_lib.key_weights(q, k, torch.zeros(1, 1, 1, device="cuda"), scale=scale)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    want = np.exp(2 * d * scale)
    off = np.abs(bits64(w) / want - 1).max()
    assert off <= 1.1 * e * 2.0 ** -28 + 2.0 ** -22 + 2.0 ** -24, off


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d,std", [(64, 1.0), (128, 1.0), (128, 3.0)])
def test_error_in_the_mean(cuda_device, fa2_lib, dtype, d, std):
    """L and the oracle in 64 bits. A term is off by its exponent's error: the score's
    cut at each of its d / 16 steps (2^-23 of it), the factor's rounding (2^-24 of
    the score, 2^-26 from log2(e)'s), L's and L log2(e)'s (2^-23 of L together), the
    last one (2^-24 of up to L); exp2 2^-22. Where a weight comes from, scores and L
    are at most about 2 std^2 and 7 + std^2 / 2 (N = 1000)."""
    g = torch.Generator().manual_seed(d)
    N, H = 1000, 4
    q = (torch.randn(1, H, N, d, generator=g) * std).to(dtype)
    k = torch.randn(1, H, N, d, generator=g).to(dtype)
    scale = float(np.float32(d ** -0.5))
    lse = torch.logsumexp(scale * (q.double() @ k.double().transpose(-1, -2)), -1).float()
    w = fa2_lib.key_weights(q.cuda(), k.cuda(), lse.cuda(), scale=scale)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    ref = oc.key_weights(bits64(q), bits64(k), bits64(lse), False, scale)
    s, L = 2 * std * std, 7 + std * std / 2
    bound = s * (d / 16 * 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -26) + L * (2.0 ** -23 + 2.0 ** -24) + 2.0 ** -22
    err = bits64(w) - ref
    assert np.linalg.norm(err) <= bound * np.linalg.norm(ref), np.linalg.norm(err) / np.linalg.norm(ref)


@pytest.mark.parametrize("d,std", [(64, 1.0), (128, 1.0), (64, 4.0), (128, 4.0)])
def test_the_weights_of_a_query_sum_to_one(cuda_device, fa2_lib, d, std):
    """With the forward's own L, whose scores are the same products by the same
    factor, nothing that grows with the scores is left: in the mean over 32768
    queries the roundings of L (2^-24 of up to 20, twice, of either sign) leave
    less than 1e-7, and exp2 and log2 2^-22 each."""
    g = torch.Generator().manual_seed(d + 1)
    H, N = 8, 4096
    q, k = ((torch.randn(1, H, N, d, generator=g) * x).to(BF16).cuda() for x in (std, 1.0))
    _, lse = fa2_lib.forward(q, k, k, num_splits=1)
    w = fa2_lib.key_weights(q, k, lse)
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    off = float(w.double().sum()) / (H * N) - 1
    assert abs(off) <= 1e-7 + 2 * 2.0 ** -22, off
