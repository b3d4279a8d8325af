"""The paged-cache entry points refuse bad arguments before touching a device:
the C ABI with made-up addresses, and the Python binding with host tensors."""

import pytest
import torch

A = 0x100000000
STEP = 0x10000000


def _p(i):
    return A + i * STEP


def test_paged_decode_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    ws = lib.fa2_paged_decode_workspace_size(2, 8, 2, 64, 16, 4, 1)
    assert ws > lib.fa2_paged_decode_workspace_size(2, 8, 2, 64, 16, 4, 0) > 0

    def call(ptr=None, B=2, Hq=8, Hkv=2, d=64, pages=10, ps=16, mp=4, scale=0.1, dtype=1, wsz=ws):
        p = {n: _p(i) for i, n in enumerate(
            ("q", "k", "v", "table", "lens", "w", "wo", "o", "lse", "ws"))}
        p.update(ptr or {})
        return lib.fa2_paged_decode(p["q"], p["k"], p["v"], p["table"], p["lens"], p["w"], p["wo"],
                                    p["o"], p["lse"], B, Hq, Hkv, d, pages, ps, mp, scale, dtype,
                                    p["ws"], wsz, None)

    for n in ("q", "k", "v", "table", "lens", "o", "lse"):
        assert call({n: 0}) == 1
    assert call({"w": 0}) == 1 and call({"wo": 0}) == 1      # both or neither
    for kw in ({"B": 0}, {"Hq": 0}, {"Hkv": 0}, {"Hq": 7}, {"pages": 0}, {"ps": 0}, {"mp": 0},
               {"scale": 0.0}, {"scale": float("inf")}, {"dtype": 2}):
        assert call(**kw) == 1, kw
    for kw in ({"d": 96}, {"B": 70000}, {"Hq": 258, "Hkv": 2}, {"pages": 2**30, "ps": 16},
               {"pages": 2**31 - 1, "Hkv": 8}, {"mp": 2**30, "ps": 2}):
        assert call(**kw) == 2, kw
    for n, off in (("q", 8), ("k", 2), ("v", 4), ("o", 8), ("table", 2), ("lens", 1), ("lse", 2),
                   ("w", 2), ("ws", 16)):
        assert call({n: _p(50) + off}) == 3, n
    assert call({"ws": 0}) == 7 and call(wsz=ws - 1) == 7
    assert call({"o": _p(0)}) == 8 and call({"o": _p(1)}) == 8 and call({"lse": _p(3)}) == 8
    assert call({"lse": _p(7)}) == 8 and call({"wo": _p(5) + 4}) == 8 and call({"ws": _p(2)}) == 8
    assert lib.fa2_paged_decode_workspace_size(2, 7, 2, 64, 16, 4, 1) == 0
    assert lib.fa2_paged_decode_workspace_size(2, 8, 2, 96, 16, 4, 1) == 0


def test_cache_append_rejects(fa2_lib):
    lib = fa2_lib.load_library()

    def call(ptr=None, B=2, Hkv=2, T=3, d=64, pages=10, ps=16, mp=4, dtype=1):
        p = {n: _p(i) for i, n in enumerate(
            ("k", "v", "kc", "vc", "table", "lens", "num", "w", "nw", "pos", "next", "out"))}
        p.update(ptr or {})
        return lib.fa2_cache_append(*(p[n] for n in ("k", "v", "kc", "vc", "table", "lens", "num", "w",
                                                     "nw", "pos", "next", "out")),
                                    B, Hkv, T, d, pages, ps, mp, dtype, None)

    for n in ("k", "v", "kc", "vc", "table", "lens", "out", "pos", "next", "w"):
        assert call({n: 0}) == 1, n           # w: new weights without weights
    for kw in ({"B": 0}, {"Hkv": 0}, {"T": 0}, {"pages": 0}, {"ps": 0}, {"mp": 0}, {"dtype": -1}):
        assert call(**kw) == 1, kw
    for kw in ({"d": 32}, {"T": 2**30}, {"mp": 2**30}):
        assert call(**kw) == 2, kw
    for n in ("k", "v", "kc", "vc"):
        assert call({n: _p(50) + 8}) == 3
    for n in ("table", "lens", "num", "w", "nw", "pos", "next", "out"):
        assert call({n: _p(50) + 2}) == 3
    assert call({"out": _p(5)}) == 8          # lens_out is lens
    assert call({"kc": _p(0)}) == 8 and call({"vc": _p(2)}) == 8 and call({"pos": _p(7)}) == 8


def test_cache_evict_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    ws = lib.fa2_cache_evict_workspace_size(2, 2, 16, 4, 40)
    assert ws == 2 * (2 * 2 * 24 * 4 // 256 * 256 + 256 * (2 * 2 * 24 * 4 % 256 > 0)) + 256
    names = ("kc", "vc", "table", "lens", "w", "wo", "pos", "po", "next", "out")

    def call(ptr=None, B=2, Hkv=2, d=64, pages=10, ps=16, mp=4, budget=40, recent=4, dtype=0, wsz=ws):
        p = {n: _p(i) for i, n in enumerate(names + ("ws",))}
        p.update(ptr or {})
        return lib.fa2_cache_evict(*(p[n] for n in names), B, Hkv, d, pages, ps, mp, budget, recent,
                                   dtype, p["ws"], wsz, None)

    for n in names:
        assert call({n: 0}) == 1, n
    for kw in ({"budget": 0}, {"recent": -1}, {"recent": 41}, {"dtype": 9}, {"B": 0}):
        assert call(**kw) == 1, kw
    assert call(d=100) == 2 and call(B=65536) == 2
    for n in ("kc", "vc", "w", "wo", "pos", "po", "next", "out", "table", "lens", "ws"):
        assert call({n: _p(50) + 2}) == 3, n
    assert call({"ws": 0}) == 7 and call(wsz=ws - 1) == 7
    assert call({"out": _p(3)}) == 8 and call({"wo": _p(4) + 4}) == 8 and call({"po": _p(5)}) == 8
    assert call({"vc": _p(0)}) == 8 and call({"ws": _p(4)}) == 8


def test_key_weights_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    ws = lib.fa2_key_weights_workspace_size()

    def call(ptr=None, B=2, Hq=4, Hkv=2, N=100, Nk=90, d=64, causal=1, scale=0.1, dtype=1, wsz=ws):
        p = {n: _p(i) for i, n in enumerate(("q", "k", "lse", "ql", "out", "ws"))}
        p.update(ptr or {})
        return lib.fa2_key_weights(p["q"], p["k"], p["lse"], p["ql"], p["out"], B, Hq, Hkv, N, Nk, d,
                                   causal, scale, dtype, p["ws"], wsz, None)

    for n in ("q", "k", "lse", "out"):
        assert call({n: 0}) == 1
    for kw in ({"B": 0}, {"N": 0}, {"Nk": 0}, {"Hq": 5}, {"causal": 2}, {"scale": -1.0}, {"dtype": 3}):
        assert call(**kw) == 1, kw
    assert call(d=80) == 2 and call(Hq=260) == 2 and call(N=2**29) == 2 and call(Nk=2**30) == 2
    assert call({"q": _p(9) + 8}) == 3 and call({"lse": _p(9) + 1}) == 3 and call({"ws": _p(9) + 8}) == 3
    assert call({"ws": 0}) == 7 and call(wsz=ws - 1) == 7
    assert call({"out": _p(2)}) == 8 and call({"out": _p(0)}) == 8 and call({"ws": _p(4)}) == 8


def test_binding_rejects_host_tensors_and_shapes(fa2_lib):
    bf = torch.bfloat16
    kc = torch.zeros(4, 2, 16, 64, dtype=bf)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(1, 2, 32)
    with pytest.raises(ValueError):
        fa2_lib.paged_decode(torch.zeros(1, 4, 64, dtype=bf), kc, kc, table, lens)
    with pytest.raises(ValueError):
        fa2_lib.cache_append(torch.zeros(1, 2, 1, 64, dtype=bf), torch.zeros(1, 2, 1, 64, dtype=bf), kc,
                             kc.clone(), table, lens)
    with pytest.raises(ValueError):
        fa2_lib.cache_evict(kc, kc.clone(), table, lens, w, 8)
    with pytest.raises(ValueError):
        fa2_lib.key_weights(torch.zeros(1, 4, 8, 64, dtype=bf), torch.zeros(1, 2, 8, 64, dtype=bf),
                            torch.zeros(1, 4, 8))
