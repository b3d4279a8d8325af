"""The Python entry points of the paged cache refuse what they cannot do, with
the framework's errors, and leave every tensor as it was; other devices'
tensors, streams and strides included."""

import pytest
import torch

from tests.cache_cases import BF16, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture
def cache(cuda_device, fa2_lib):
    c = Cache(2, 2, 64, 16, [20, 33], BF16, seed=0, width=4, nan=False)
    kc, vc, table, lens = c.gpu()
    return dict(k=kc, v=vc, table=table, lens=lens, q=c.query(4).cuda(), w=c.weights().cuda())


def _decode(fa2, c, **kw):
    a = {**c, **kw}
    return fa2.paged_decode(a["q"], a["k"], a["v"], a["table"], a["lens"],
                            **{x: a[x] for x in ("weights", "weights_out", "out", "lse", "workspace", "scale") if x in a})


def test_decode_refusals(fa2_lib, cache):
    before = [cache["k"].clone(), cache["w"].clone()]
    bad = [
        dict(q=cache["q"].cpu()), dict(q=cache["q"].half()), dict(q=cache["q"][0]), dict(q=cache["q"].transpose(0, 1)),
        dict(k=cache["k"].cpu()), dict(k=cache["k"].float()), dict(v=cache["v"][:-1]), dict(v=cache["v"].transpose(1, 2)),
        dict(table=cache["table"].long()), dict(table=cache["table"][0]), dict(table=cache["table"][:, ::2]),
        dict(lens=cache["lens"].long()), dict(lens=cache["lens"][:1]), dict(lens=cache["lens"].cpu()),
        dict(weights=cache["w"][..., :-1]), dict(weights=cache["w"].double()), dict(weights_out=cache["w"]),
        dict(out=cache["q"].float()), dict(lse=torch.zeros(2, 4)), dict(workspace=torch.zeros(10)),
        dict(q=None), dict(k=3),
    ]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            _decode(fa2_lib, cache, **kw)
    for kw, code in (
        (dict(q=cache["q"][:, :3].contiguous()), 1),       # 3 query heads, 2 key heads
        (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
        (dict(out=cache["q"]), 8),
        (dict(weights=cache["w"], weights_out=cache["k"].view(-1).view(torch.float32)[:cache["w"].numel()].view_as(cache["w"])), 8),
        (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), 7),
    ):
        with pytest.raises(fa2_lib.FA2Error) as e:
            _decode(fa2_lib, cache, **kw)
        assert e.value.code == code
    torch.cuda.synchronize()
    assert torch.equal(before[0], cache["k"]) and torch.equal(before[1], cache["w"])
    assert fa2_lib.device_status() == 0


def test_append_and_evict_refusals(fa2_lib, cache):
    k, v, table, lens, w = (cache[x] for x in ("k", "v", "table", "lens", "w"))
    new = torch.zeros(2, 2, 3, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda")
    before = k.clone()
    for kw in (dict(new_weights=torch.zeros(2, 2, 3, device="cuda")), dict(positions=pos), dict(next_pos=lens),
               dict(num_new=lens.long()), dict(weights=w[:1]), dict(lens_out=lens.cpu())):
        with pytest.raises(ValueError):
            fa2_lib.cache_append(new, new.clone(), k, v, table, lens, **kw)
    with pytest.raises(ValueError):
        fa2_lib.cache_append(new[..., :32], new, k, v, table, lens)
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.cache_append(new, new, k, v, table, lens, lens_out=lens)
    assert e.value.code == 8
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.cache_append(new[:, :, :0], new[:, :, :0], k, v, table, lens)
    assert e.value.code == 1
    for kw in (dict(budget=0), dict(budget=4, recent=5), dict(budget=4, recent=-1), dict(budget=4, positions=pos),
               dict(budget=4, positions_out=pos), dict(budget=4, next_pos=lens), dict(budget=4, weights_out=w[0])):
        with pytest.raises(ValueError):
            fa2_lib.cache_evict(k, v, table, lens, w, **kw)
    with pytest.raises(TypeError):
        fa2_lib.cache_evict(k, v, table, lens, w, 4.5)
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.cache_evict(k, v, table, lens, w, 4, lens_out=lens)
    assert e.value.code == 8
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.cache_evict(k, k, table, lens, w, 4)
    assert e.value.code == 8
    torch.cuda.synchronize()
    assert torch.equal(before, k) and fa2_lib.device_status() == 0


def test_key_weights_refusals(fa2_lib, cuda_device):
    q = torch.zeros(1, 4, 8, 64, dtype=BF16, device="cuda")
    k, lse = q[:, :2].contiguous(), torch.zeros(1, 4, 8, device="cuda")
    for a in ((q.float(), k, lse), (q, k.half(), lse), (q, k, lse.double()), (q, k, lse[:, :2]), (q[0], k, lse),
              (q.cpu(), k, lse), (q.transpose(2, 3), k, lse)):
        with pytest.raises(ValueError):
            fa2_lib.key_weights(*a)
    for kw in (dict(q_lens=torch.zeros(1, device="cuda")), dict(out=torch.zeros(1, 4, 8, device="cuda"))):
        with pytest.raises(ValueError):
            fa2_lib.key_weights(q, k, lse, **kw)
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.key_weights(q, q[:, :3].contiguous(), lse)
    assert e.value.code == 1


def test_calls_run_on_the_current_stream(fa2_lib, cache):
    """Each call is ordered with other work of the stream that is current."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
        lens = cache["lens"] - 10
        o, lse = _decode(fa2_lib, cache, lens=lens)
    side.synchronize()
    want, _ = _decode(fa2_lib, cache, lens=lens)
    torch.cuda.synchronize()
    assert torch.equal(o, want)
