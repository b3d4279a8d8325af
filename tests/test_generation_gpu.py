"""The operators together, as a program that generates with a bounded cache uses
them: prompt -> forward, key weights, append; then per token append, decode
(weights gathered), eviction once the cache is over its budget."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, bits64, decode_bounds, score_error

pytestmark = pytest.mark.gpu


def _raw(t):
    return t.detach().cpu().view(torch.int16).numpy()


@pytest.mark.parametrize("d,ps,group", [(128, 16, 4), (64, 24, 1)])
def test_prompt_then_tokens_with_a_budget(cuda_device, fa2_lib, d, ps, group):
    B, Hkv, N, budget, recent, steps = 2, 2, 300, 200, 16, 12
    Hq, dev = Hkv * group, cuda_device
    prompt = [300, 211]
    width = -(-N // ps) + 1
    L = width * ps
    g = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev).to(BF16)  # noqa: E731
    q, k, v = rnd(B, Hq, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, N, d)
    q_lens = torch.tensor(prompt, dtype=torch.int32, device=dev)
    table = torch.randperm(B * width, generator=g, device=dev).to(torch.int32).view(B, width)
    kc, vc = (torch.full((B * width, Hkv, ps, d), float("nan"), dtype=BF16, device=dev) for _ in range(2))
    weights = torch.zeros(B, Hkv, L, device=dev)
    positions = torch.zeros(B, Hkv, L, dtype=torch.int32, device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)

    # Prompt.
    rep = lambda t: t.repeat_interleave(group, 1).contiguous()  # noqa: E731
    _, lse = fa2_lib.forward(q, rep(k), rep(v), causal=True)
    w0 = fa2_lib.key_weights(q, k, lse, causal=True, q_lens=q_lens)
    lens = fa2_lib.cache_append(k, v, kc, vc, table, lens, num_new=q_lens, weights=weights, new_weights=w0,
                                positions=positions, next_pos=torch.zeros_like(lens))
    next_pos = q_lens.clone()
    assert lens.tolist() == prompt
    text_k = [k[b, :, :prompt[b]] for b in range(B)]  # every token so far, by position

    for step in range(steps):
        # Eviction, against the oracle on the same weights.
        snap = [t.clone() for t in (kc, vc, weights, positions, lens)]
        lens = fa2_lib.cache_evict(kc, vc, table, lens, weights, budget, recent=recent, positions=positions,
                                   next_pos=next_pos)
        k2, v2, w2, p2, left = oc.cache_evict(_raw(snap[0]), _raw(snap[1]), table.cpu().numpy(),
                                              snap[4].cpu().numpy(), snap[2].cpu().numpy(), budget, recent,
                                              snap[3].cpu().numpy(), next_pos.cpu().numpy())
        assert lens.tolist() == left.tolist() == [min(budget, int(x)) for x in snap[4]]
        assert (_raw(kc) == k2).all() and (_raw(vc) == v2).all()
        assert np.array_equal(positions.cpu().numpy(), p2) and np.array_equal(weights.cpu().numpy(), w2)
        # Every slot still holds the key of the position it names, and the recent ones are there.
        for b in range(B):
            n = int(lens[b])
            slots = torch.arange(n, device=dev)
            for h in range(Hkv):
                pos = positions[b, h, :n].long()
                page = table[b].long()[slots // ps]
                assert torch.equal(kc[page, h, slots % ps], text_k[b][h][pos])
                assert set(range(int(next_pos[b]) - recent, int(next_pos[b]))) <= set(pos.tolist())
        # One token.
        qt, kt, vt = rnd(B, Hq, d), rnd(B, Hkv, 1, d), rnd(B, Hkv, 1, d)
        lens = fa2_lib.cache_append(kt, vt, kc, vc, table, lens, weights=weights, positions=positions,
                                    next_pos=next_pos)
        next_pos += 1
        text_k = [torch.cat([text_k[b], kt[b]], 1) for b in range(B)]
        before = weights.clone()
        o, lse_t = fa2_lib.paged_decode(qt, kc, vc, table, lens, weights=weights)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 0
        args = (bits64(qt), bits64(kc), bits64(vc), table.cpu().numpy(), lens.cpu().numpy(), d ** -0.5)
        o_ref, l_ref, p = oc.paged_decode(*args)
        A, _, _ = oc.paged_decode(args[0], args[1], np.abs(args[2]), *args[3:])
        tol_o, tol_l, rel = decode_bounds(o_ref, l_ref, A, score_error(args[0], np.nan_to_num(args[1]), d ** -0.5),
                                          int(lens.max()), BF16)
        assert (np.abs(bits64(o) - o_ref) <= tol_o).all() and (np.abs(bits64(lse_t) - l_ref) <= tol_l).all()
        for b in range(B):
            n = int(lens[b])
            want = bits64(before[b, :, :n]) + p[b]
            assert (np.abs(bits64(weights[b, :, :n]) - want) <= p[b] * rel + 2.0 ** -23 * want).all()
