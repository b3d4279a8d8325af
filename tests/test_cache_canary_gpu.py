"""Guard canaries around everything that the paged-cache calls and the key weights
write: outputs, caches, weights, positions, lengths and workspaces lie inside
larger buffers of a byte pattern, whose margins must come back untouched."""

import ctypes

import pytest
import torch

from tests.cache_cases import BF16, Cache
from tests.test_canary_gpu import Guarded, _nbytes

pytestmark = pytest.mark.gpu


def _guard(t):
    g = Guarded(_nbytes(t.shape, t.dtype), "cuda")
    g.tensor(t.shape, t.dtype).copy_(t)
    return g


@pytest.mark.parametrize("d,ps,g,lens", [(64, 5, 1, [33, 0, 64]), (128, 16, 3, [1, 257, 100]), (64, 24, 17, [500, 7, 90])])
def test_paged_cache_writes_nothing_outside(cuda_device, fa2_lib, d, ps, g, lens):
    B, Hkv, budget, recent, T = 3, 2, 40, 4, 3
    lib = fa2_lib.load_library()
    c = Cache(B, Hkv, d, ps, lens, BF16, seed=d + ps, width=-(-(max(lens) + T) // ps))
    width, pages, L = c.table.shape[1], c.k.shape[0], c.L
    table, ln = c.table.cuda(), c.lens.cuda()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    kc, vc = _guard(c.k), _guard(c.v)
    w, pos = _guard(c.weights()), _guard(torch.arange(L, dtype=torch.int32).expand(B, Hkv, L).contiguous())
    q = c.query(Hkv * g).cuda()
    new = torch.randn(B, Hkv, T, d, generator=c.g).to(BF16).cuda()
    o, lse = Guarded(_nbytes(q.shape, BF16), "cuda"), Guarded(B * Hkv * g * 4, "cuda")
    l1, l2 = Guarded(B * 4, "cuda"), Guarded(B * 4, "cuda")
    nw = lib.fa2_paged_decode_workspace_size(B, Hkv * g, Hkv, d, ps, width, 1)
    ne = lib.fa2_cache_evict_workspace_size(B, Hkv, ps, width, budget)
    ws, we = Guarded(nw, "cuda"), Guarded(ne, "cuda")
    size = (B, Hkv, T, d, pages, ps, width, 1)
    assert lib.fa2_cache_append(new.data_ptr(), new.data_ptr(), kc.ptr, vc.ptr, table.data_ptr(), ln.data_ptr(), None,
                                w.ptr, None, pos.ptr, ln.data_ptr(), l1.ptr, *size, stream) == 0
    assert lib.fa2_paged_decode(q.data_ptr(), kc.ptr, vc.ptr, table.data_ptr(), l1.ptr, w.ptr, w.ptr, o.ptr, lse.ptr,
                                B, Hkv * g, Hkv, d, pages, ps, width, d ** -0.5, 1, ws.ptr, nw, stream) == 0
    assert lib.fa2_cache_evict(kc.ptr, vc.ptr, table.data_ptr(), l1.ptr, w.ptr, w.ptr, pos.ptr, pos.ptr, l1.ptr, l2.ptr,
                               B, Hkv, d, pages, ps, width, budget, recent, 1, we.ptr, ne, stream) == 0
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    for name, buf in dict(kc=kc, vc=vc, w=w, pos=pos, o=o, lse=lse, l1=l1, l2=l2, ws=ws, we=we).items():
        assert buf.margins_intact(), name
    assert l2.tensor((B,), torch.int32).tolist() == [min(n + T, budget) for n in lens]
    assert torch.isfinite(o.tensor(q.shape, BF16)).all()


@pytest.mark.parametrize("N,Nk,d,causal", [(1, 1, 64, 1), (129, 257, 128, 1), (300, 255, 64, 0), (1000, 1000, 128, 1)])
def test_key_weights_write_nothing_outside(cuda_device, fa2_lib, N, Nk, d, causal):
    lib = fa2_lib.load_library()
    B, Hq, Hkv = 2, 4, 2
    g = torch.Generator(device="cuda").manual_seed(N)
    q = torch.randn(B, Hq, N, d, generator=g, device="cuda").to(BF16)
    k = torch.randn(B, Hkv, Nk, d, generator=g, device="cuda").to(BF16)
    lse = torch.full((B, Hq, N), 5.0, device="cuda")
    need = lib.fa2_key_weights_workspace_size()
    out, ws = Guarded(B * Hkv * Nk * 4, "cuda"), Guarded(need, "cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.fa2_key_weights(q.data_ptr(), k.data_ptr(), lse.data_ptr(), None, out.ptr, B, Hq, Hkv, N, Nk, d, causal,
                               d ** -0.5, 1, ws.ptr, need, stream) == 0
    torch.cuda.synchronize()
    assert fa2_lib.device_status() == 0
    assert out.margins_intact() and ws.margins_intact()
    w = out.tensor((B, Hkv, Nk), torch.float32)
    assert (w >= 0).all() and (w[..., min(N, Nk):] == 0).all() == bool(causal or Nk <= N)
