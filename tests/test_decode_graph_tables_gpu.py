"""A captured decode follows the page table and the lengths in device memory."""

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_cases import BF16, Cache, bits64, decode_bounds, score_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [8, 60], ids=["whole", "split"])
@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
def test_a_replay_follows_the_table(cuda_device, fa2_lib, width, weights):
    B, Hkv, d, ps, Hq = 3, 2, 64, 16, 6
    L = width * ps
    c = Cache(B, Hkv, d, ps, [L] * B, BF16, seed=width)
    c.k[:], c.v[:] = (torch.randn(c.k.shape, generator=c.g).to(BF16) for _ in range(2))  # every page holds keys
    kc, vc, table, lens = c.gpu()
    q = c.query(Hq)
    w0 = c.weights()
    qg, wg = q.cuda(), w0.cuda()
    w = torch.zeros_like(wg) if weights else None
    call = lambda: fa2_lib.paged_decode(qg, kc, vc, table, lens, weights=wg if weights else None, weights_out=w)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call()
    seen = []
    pages = c.k.shape[0]
    for step, n in enumerate(([L, 64, L - 7], [L, 64, L - 7], [1, 0, L], [L - 1, L, 33])):
        t = [c.table, c.table.roll(1, 1), c.table.flip(0),
             torch.randperm(pages, generator=c.g)[:B * width].to(torch.int32).view(B, width)][step]
        table.copy_(t)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        args = (bits64(q), bits64(c.k), bits64(c.v), t.numpy(), np.array(n), float(np.float32(d ** -0.5)))
        ref, lref, p = oc.paged_decode(*args)
        A, _, _ = oc.paged_decode(args[0], args[1], np.abs(args[2]), *args[3:])
        tol_o, tol_l, rel = decode_bounds(ref, lref, A, score_error(args[0], args[1], args[5]), L, BF16)
        assert (np.abs(bits64(o) - ref) <= tol_o).all()
        fin = np.isfinite(lref)
        assert (bits64(lse)[~fin] == -np.inf).all()
        assert (np.abs(bits64(lse) - np.where(fin, lref, 0))[fin] <= tol_l[fin]).all()
        if weights:
            for b in range(B):
                want = bits64(w0)[b, :, :n[b]] + p[b]
                assert (np.abs(bits64(w[b, :, :n[b]]) - want) <= p[b] * rel + 2.0 ** -23 * want).all()
        seen.append(o.clone())
    # Another order of the pages is another sequence, at the length that leaves some out.
    assert not torch.equal(seen[0][1], seen[1][1])
    assert fa2_lib.device_status() == 0
