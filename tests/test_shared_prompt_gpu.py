"""The operators together, as a program that serves a batch behind a common prompt uses
them: the prompt once (projection -> rotary -> forward -> pages -> append), then per
token pages, rotary, append and decode behind the shared prefix, with sequences that end
and others that begin."""

import random

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import rotary as orc
from tests.cache_cases import BF16, bits64, decode_bounds, score_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,group,d,ps,P,norm", [(5, 4, 128, 16, 100, True), (30, 2, 64, 8, 257, False)])
def test_batch_behind_a_prompt(cuda_device, fa2_lib, B, group, d, ps, P, norm):
    Hkv, steps, most = 2, 14, P + 40
    Hq, dev, scale = Hkv * group, cuda_device, d ** -0.5
    r, g = random.Random(B), torch.Generator(device="cuda").manual_seed(d)
    width = -(-most // ps)
    pages = width * (B + 1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    project = lambda rows, n: torch.randn(rows, n, Hq + 2 * Hkv, d, generator=g, device=dev).to(BF16)  # noqa: E731
    split = lambda x: (x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2),  # noqa: E731
                       x[:, :, Hq + Hkv:].transpose(1, 2).contiguous())
    freqs = fa2_lib.rotary_frequencies(d, factor=4.0, method="bands", original=64).to(dev)
    w = [1 + 0.1 * torch.randn(d, generator=g, device=dev) for _ in range(2)] if norm else [None, None]
    turn = lambda q, k, pos: fa2_lib.rotary_forward(q, k, freqs, pos, q_weight=w[0], k_weight=w[1])  # noqa: E731
    kc, vc = (torch.full((pages, Hkv, ps, d), float("nan"), dtype=BF16, device=dev) for _ in range(2))
    refs, free, num_free = ints([0] * pages), torch.randperm(pages, generator=g, device=dev).int(), ints([pages])
    # The last row is the prompt's own.
    table, lens = ints([[-1] * width] * (B + 1)), ints([0] * (B + 1))

    # The prompt, once.
    q, k, v = split(project(1, P))
    qr, kr = turn(q, k, None)
    rep = lambda t: t.repeat_interleave(group, 1).contiguous()  # noqa: E731
    o, _ = fa2_lib.forward(qr, rep(kr), rep(v), causal=True)
    ref = orc.rotary(bits64(k), freqs.cpu().numpy(), np.arange(P)[None], False,
                     None if w[1] is None else bits64(w[1]))
    assert np.max(np.abs(bits64(kr) - ref)) <= 2.0 ** -8 * np.abs(ref).max() + 1e-5
    shared = P // ps * ps  # whole pages; the rest of the prompt is every sequence's own
    lens = fa2_lib.cache_resize(table, lens, ints([0] * B + [shared]), refs, free, num_free, ps)
    fa2_lib.cache_append(kr[:, :, :shared].contiguous(), v[:, :, :shared].contiguous(), kc, vc, table[B:],
                         torch.zeros_like(lens[B:]))
    prefix, prefix_len = table[B, :max(1, shared // ps)].clone(), ints([shared])
    rest = [t[:, :, shared:].expand(B, Hkv, P - shared, d).contiguous() for t in (kr, v)]

    def begin(who, lens):
        """These sequences take over the prompt's pages, and get its last tokens."""
        table[who, :shared // ps] = prefix[:shared // ps]
        refs[prefix[:shared // ps].long()] += len(who)
        lens = lens.clone()
        lens[who] = shared
        want = lens.clone()
        want[who] = P
        got = fa2_lib.cache_resize(table, lens, want, refs, free, num_free, ps)
        assert torch.equal(got, want)
        if P > shared:
            new = ints([P - shared if b in who else 0 for b in range(B)])
            fa2_lib.cache_append(rest[0], rest[1], kc, vc, table[:B], lens[:B], num_new=new)
        return want

    lens = begin(list(range(B)), lens)
    alive = set(range(B))
    for step in range(steps):
        # Some end, some begin.
        ending = [b for b in sorted(alive) if r.random() < 0.15]
        want = lens.clone()
        want[ending] = 0
        lens = fa2_lib.cache_resize(table, lens, want, refs, free, num_free, ps)
        alive -= set(ending)
        new = [b for b in range(B) if b not in alive and r.random() < 0.5]
        if new:
            lens = begin(new, lens)
            alive |= set(new)
        # One token.
        on = ints([1 if b in alive else 0 for b in range(B)])
        want = lens.clone()
        want[:B] += on
        assert torch.equal(fa2_lib.cache_resize(table, lens, want, refs, free, num_free, ps), want)
        q, k, v = split(project(B, 1))
        qr, kr = turn(q, k, lens[:B].contiguous())
        now = fa2_lib.cache_append(kr, v, kc, vc, table[:B], lens[:B].contiguous(), num_new=on)
        assert torch.equal(now, want[:B])
        lens = want
        qd = qr.squeeze(2)
        o, lse = fa2_lib.prefix_decode(qd, kc, vc, table[:B], now, prefix, prefix_len)
        o2, lse2 = fa2_lib.paged_decode(qd, kc, vc, table[:B], now)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 0
        args = (bits64(qd), bits64(kc), bits64(vc), table[:B].cpu().numpy(), now.cpu().numpy(), scale)
        o_ref, l_ref, _ = oc.paged_decode(*args)
        A, _, _ = oc.paged_decode(args[0], args[1], np.abs(args[2]), *args[3:])
        tol_o, tol_l, _ = decode_bounds(o_ref, l_ref, A, score_error(args[0], np.nan_to_num(args[1]), scale),
                                        int(now.max()), BF16)
        for oo, ll in ((o, lse), (o2, lse2)):
            assert (np.abs(bits64(oo) - o_ref) <= tol_o).all()
            fin = np.isfinite(l_ref)
            assert (np.abs(bits64(ll) - np.where(fin, l_ref, 0))[fin] <= tol_l[fin]).all()
            assert (bits64(ll)[~fin] == -np.inf).all()
        # Every page is free or counted by those that name it.
        counts = np.zeros(pages, int)
        t, n = table.cpu().numpy(), lens.cpu().numpy()
        for b in range(B + 1):
            for i in range(-(-n[b] // ps)):
                counts[t[b, i]] += 1
        assert (counts == refs.cpu().numpy()).all()
        nf = int(num_free)
        assert sorted(free[:nf].tolist()) == np.flatnonzero(counts == 0).tolist()
    lens = fa2_lib.cache_resize(table, lens, torch.zeros_like(lens), refs, free, num_free, ps)
    assert int(num_free) == pages and not refs.any() and fa2_lib.device_status() == 0
