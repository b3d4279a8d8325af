"""Pins of the paged-cache oracle: against the attention oracle, hand-worked
cases and invariants."""

import math

import numpy as np
import pytest

import oracle
from oracle import cache


def _paged(rng, B, Hkv, d, ps, width):
    pages = B * width + 2
    table = rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    return rng.standard_normal((pages, Hkv, ps, d)), rng.standard_normal((pages, Hkv, ps, d)), table


def test_decode_is_the_last_row_of_the_attention_oracle():
    rng = np.random.default_rng(0)
    B, H, d, ps, n = 2, 3, 64, 4, 11
    kc, vc, table = _paged(rng, B, H, d, ps, 3)
    q = rng.standard_normal((B, H, d))
    o, lse, p = cache.paged_decode(q, kc, vc, table, [n, n], 0.125)
    k = np.stack([cache.tokens(kc, table, b, n) for b in range(B)])
    v = np.stack([cache.tokens(vc, table, b, n) for b in range(B)])
    o_ref, lse_ref = oracle.forward(q[:, :, None], k, v, causal=False, scale=0.125)
    assert np.abs(o - o_ref[:, :, 0]).max() < 1e-12 and np.abs(lse - lse_ref[:, :, 0]).max() < 1e-12
    assert all(np.allclose(w.sum(1), 1.0) for w in p)


def test_decode_slots_follow_the_table():
    kc = np.arange(4 * 1 * 2 * 1, dtype=float).reshape(4, 1, 2, 1)
    assert cache.tokens(kc, np.array([[3, 0]]), 0, 3)[0, :, 0].tolist() == [6.0, 7.0, 0.0]


def test_decode_without_slots():
    rng = np.random.default_rng(1)
    kc, vc, table = _paged(rng, 1, 1, 64, 4, 1)
    o, lse, p = cache.paged_decode(np.ones((1, 2, 64)), kc, vc, table, [0], 1.0)
    assert (o == 0).all() and (lse == -math.inf).all() and p[0].shape == (1, 0)


def test_evict_by_hand():
    w = [5.0, 1.0, 4.0, 0.5, 3.0, 2.0]
    no = [False] * 6
    assert cache.evict_places(w, 6, 6, no) == [0, 1, 2, 3, 4, 5]
    assert cache.evict_places(w, 6, 3, no) == [0, 4, 2]      # 1 leaves, 4 takes its slot
    assert cache.evict_places(w, 6, 1, no) == [0]
    assert cache.evict_places(w, 6, 3, [False] * 4 + [True] * 2) == [0, 4, 5]
    assert cache.evict_places([1.0] * 5, 5, 2, [False] * 5) == [0, 1]  # ties: lower slots
    assert cache.evict_places([math.nan, -math.inf, 0.0], 3, 1, [False] * 3) == [2]
    assert cache.evict_places([math.nan, -math.inf, math.nan], 3, 2, [False] * 3) == [0, 1]


@pytest.mark.parametrize("recent", [0, 3])
def test_evict_keeps_a_set_and_its_tokens(recent):
    rng = np.random.default_rng(2)
    B, H, d, ps, budget = 2, 2, 3, 4, 7
    kc, vc, table = _paged(rng, B, H, d, ps, 4)
    lens = [15, 6]
    w = rng.random((B, H, 16))
    pos = np.tile(np.arange(16, dtype=np.int32), (B, H, 1))
    k2, v2, w2, p2, left = cache.cache_evict(kc, vc, table, lens, w, budget, recent, pos, [15, 6])
    assert left.tolist() == [7, 6]
    old, new = cache.tokens(kc, table, 0, 15), cache.tokens(k2, table, 0, 7)
    for h in range(H):
        assert (new[h] == old[h][p2[0, h, :7]]).all()
        assert (w2[0, h, :7] == w[0, h][p2[0, h, :7]]).all()
        assert set(range(15 - recent, 15)) <= set(p2[0, h, :7].tolist())
        rest = [x for x in range(15 - recent) if x not in p2[0, h, :7]]
        kept = [x for x in p2[0, h, :7] if x < 15 - recent]
        assert max(w[0, h, rest]) <= min(w[0, h, kept])
    assert (k2[table[1]] == kc[table[1]]).all()


@pytest.mark.parametrize("causal", [False, True])
def test_key_weights_sum_to_the_queries(causal):
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 4, 6, 8)), rng.standard_normal((1, 2, 6, 8))
    kk = np.repeat(k, 2, axis=1)
    lse = np.zeros((1, 4, 6))
    for x in range(4):
        s = 0.3 * q[0, x] @ kk[0, x].T
        if causal:
            s = np.where(np.tri(6, dtype=bool), s, -np.inf)
        lse[0, x] = np.log(np.exp(s).sum(1))
    w = cache.key_weights(q, k, lse, causal, 0.3)
    assert np.allclose(w.sum(2), 12.0)  # two heads, six queries, rows of sum one
    if causal:
        assert np.allclose(cache.key_weights(q, k, lse, True, 0.3, [4])[:, :, 4:], 0.0)
        assert np.allclose(cache.key_weights(q, k, lse, True, 0.3, [4]).sum(2), 8.0)


def test_append_writes_only_the_new_slots():
    rng = np.random.default_rng(4)
    kc, _, table = _paged(rng, 2, 1, 2, 2, 3)
    new = rng.standard_normal((2, 1, 3, 2))
    out = cache.cache_append(new, kc, table, [1, 0], [2, 0])
    t = cache.tokens(out, table, 0, 3)
    assert (t[0, 1:] == new[0, 0, :2]).all() and (t[0, 0] == cache.tokens(kc, table, 0, 1)[0, 0]).all()
    assert (out != kc).any(axis=-1).sum() == 2
