"""README's example of positions, shared prompts and pages does what it says."""

import re
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import rotary as orc
from tests.cache_cases import BF16, bits64

pytestmark = pytest.mark.gpu

README = Path(__file__).resolve().parent.parent / "README.md"


def _example(heading):
    text = README.read_text()
    part = text[text.index(heading):]
    return re.search(r"```python\n(.*?)```", part, re.S).group(1)


def test_positions_shared_prompts_and_pages(cuda_device, fa2_lib):
    """Run token by token beside lists of each sequence's keys and values: a token stands at
    the position and in the slot of its number; one that finds no page is not appended."""
    B, Hq, Hkv, d, ps, P, N = 3, 4, 2, 64, 16, 32, 20
    code = compile(_example("### Positions, shared prompts and pages"), "README.md", "exec")
    g = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g).to(BF16).cuda()  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, pages = [40, 47, 48], 10
    table = torch.full((B, 5), -1, dtype=torch.int32)
    table[:, :2] = torch.tensor([7, 4], dtype=torch.int32)  # the prompt's pages
    table[:, 2] = torch.tensor([1, 5, 0], dtype=torch.int32)
    kc, vc = (torch.full((pages, Hkv, ps, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    keys, values = [[] for _ in range(B)], [[] for _ in range(B)]
    for b in range(B):
        for j in range(lens[b]):
            page = int(table[b, j // ps])
            if b == 0 or j >= P:
                kc[page, :, j % ps], vc[page, :, j % ps] = rand(Hkv, d), rand(Hkv, d)
            keys[b].append(bits64(kc[page, :, j % ps]))
            values[b].append(bits64(vc[page, :, j % ps]))
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[[7, 4]], refs[[1, 5, 0]] = B, 1
    free = torch.full((pages,), -1, dtype=torch.int32)
    free[:1] = 9  # one page for two sequences that will need one
    ns = dict(fa2=fa2_lib, Hq=Hq, Hkv=Hkv, d=d, page_size=ps, table=table.cuda(), lens=ints(lens), refs=refs.cuda(),
              free_pages=free.cuda(), num_free=ints([1]), k_cache=kc, v_cache=vc, prefix=ints([7, 4]), prefix_len=ints([P]),
              positions=ints([0, 5, 9]), x=rand(B, N, Hq + 2 * Hkv, d).requires_grad_(),
              wq=(1 + 0.1 * rand(d).float()).requires_grad_(), wk=(1 + 0.1 * rand(d).float()).requires_grad_())
    wk, scale = bits64(ns["wk"]), d ** -0.5
    for step, want in enumerate(([41, 48, 49], [42, 48, 50], [43, 48, 51])):
        q1, k1, v1 = rand(B, Hq, 1, d), rand(B, Hkv, 1, d), rand(B, Hkv, 1, d)
        k0, v0 = bits64(k1), bits64(v1)
        ns.update(q1=q1, k1=k1, v1=v1)
        exec(code, ns)
        torch.cuda.synchronize()
        assert fa2_lib.device_status() == 0 and ns["lens"].tolist() == want
        turned = orc.rotary(k0, bits64(ns["f"]), np.array(lens)[:, None], False, wk)
        assert np.abs(bits64(ns["k1"]) - turned).max() <= 2.0 ** -8 * np.abs(turned).max() + 1e-5
        for b in range(B):
            if want[b] > lens[b]:
                keys[b].append(bits64(ns["k1"])[b, :, 0])
                values[b].append(v0[b, :, 0])
            K, V, Q = np.array(keys[b]), np.array(values[b]), bits64(ns["q1"])[b, :, 0]
            assert len(K) == want[b]
            for h in range(Hq):
                s = scale * K[:, h // 2] @ Q[h]
                p = np.exp(s - s.max())
                o = p @ V[:, h // 2] / p.sum()
                # one rounding of o; p |v| sums off by far less than a step of the largest
                assert np.abs(bits64(ns["o"])[b, h] - o).max() <= 2.0 ** -8 * np.abs(o).max() + 2.0 ** -14 * np.abs(V).max()
        lens = want
    # the prompt's part, as a training step
    rep = lambda t: t.repeat_interleave(2, 1)  # noqa: E731
    fa2_lib.attention(ns["q"], rep(ns["k"]), rep(ns["v"]), causal=True).float().sum().backward()
    assert all(torch.isfinite(ns[n].grad).all() and ns[n].grad.abs().max() > 0 for n in ("x", "wq", "wk"))
