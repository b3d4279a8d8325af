"""The rotary entry points refuse bad arguments before touching a device: the C ABI
with made-up addresses, and the binding with host tensors."""

import ctypes
import random

import pytest
import torch

A, STEP = 0x100000000, 0x10000000


def _p(i):
    return A + i * STEP


def _strides(*rows):
    flat = [x for r in rows for x in r]
    return (ctypes.c_longlong * len(flat))(*flat)


B, HQ, HK, N, D = 2, 4, 2, 10, 64
CQ, CK = (HQ * N * D, N * D, D), (HK * N * D, N * D, D)


def _fwd(lib, ptr=None, st=None, B=B, Hq=HQ, Hk=HK, N=N, d=D, r=32, mode=1, inter=0, eps=1e-6, amp=1.0, dtype=1, wt=2):
    p = {n: _p(i) for i, n in enumerate(("q", "k", "f", "pos", "qw", "kw", "qo", "ko"))}
    p.update(ptr or {})
    s = st or (CQ, CK, CQ, CK)
    return lib.fa2_rotary_fwd(p["q"], p["k"], p["f"], p["pos"], p["qw"], p["kw"], p["qo"], p["ko"], _strides(*s), B, Hq,
                              Hk, N, d, r, mode, inter, eps, amp, dtype, wt, None)


def test_forward_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    for n in ("q", "k", "f", "pos", "kw", "qw", "qo", "ko"):
        assert _fwd(lib, {n: 0}) == 1, n
    for kw in (dict(B=0), dict(N=0), dict(Hq=0), dict(Hk=-1), dict(Hk=0), dict(mode=3), dict(mode=0), dict(inter=2),
               dict(eps=-1.0), dict(eps=float("nan")), dict(amp=float("inf")), dict(dtype=2), dict(dtype=3), dict(wt=0)):
        assert _fwd(lib, **kw) == 1, kw
    for kw in (dict(d=96), dict(r=8), dict(r=24), dict(r=80), dict(B=65536), dict(Hq=65536), dict(N=2 ** 29)):
        assert _fwd(lib, **kw) == 2, kw
    for n in ("q", "k", "qo", "ko", "qw", "kw"):
        assert _fwd(lib, {n: _p(50) + 8}) == 3, n
    assert _fwd(lib, {"f": _p(50) + 4}) == 3 and _fwd(lib, {"pos": _p(50) + 2}) == 3
    assert _fwd(lib, st=((HQ * N * D, N * D, D + 4), CK, CQ, CK)) == 3       # rows off 16 bytes
    assert _fwd(lib, st=((-1, N * D, D), CK, CQ, CK)) == 1
    assert _fwd(lib, {"qo": _p(0)}) == 8 and _fwd(lib, {"ko": _p(0)}) == 8 and _fwd(lib, {"qo": _p(2)}) == 8
    assert _fwd(lib, {"qo": _p(3)}) == 8 and _fwd(lib, {"ko": _p(4)}) == 8 and _fwd(lib, {"ko": _p(6)}) == 8
    # outputs whose own rows overlap, or that share rows with each other
    assert _fwd(lib, st=(CQ, CK, (HQ * N * D, 0, D), CK)) == 8
    assert _fwd(lib, st=(CQ, CK, (N * D, N * D, D), CK)) == 8
    packed = (N * 8 * D, D, 8 * D)
    assert _fwd(lib, {"ko": _p(6) + 3 * D * 2}, st=(CQ, CK, packed, packed)) == 8
    assert _fwd(lib, {"ko": _p(6) + 7 * D * 2}, st=(CQ, CK, packed, packed)) == 8  # runs into the next token
    other = (N * 8 * D, D, 16 * D)
    assert _fwd(lib, {"ko": _p(6) + 4 * D * 2}, st=(CQ, CK, packed, other)) == 8


def _layout(lib, ko, sq, sk, B, Hq, Hk, N, d=64):
    """Status of outputs at these offsets and strides; 3 (the weights' alignment, which is
    checked next) if they do not clash."""
    ptr = {"qo": _p(6), "ko": _p(6) + 2 * ko, "qw": _p(50) + 8}
    return _fwd(lib, ptr, ((Hq * N * d, N * d, d), (Hk * N * d, N * d, d), sq, sk), B, Hq, Hk, N, d)


def test_outputs_side_by_side(fa2_lib):
    """Heads of one buffer in a token's row or head by head, in any order and with room
    around them; never rows that share elements (against a count of the elements)."""
    lib = fa2_lib.load_library()
    d = 64
    for B in (1, 3):
        for Hq, Hk, N in ((4, 2, 10), (1, 1, 7), (8, 1, 1), (1, 5, 3)):
            H = Hq + Hk + 1  # a head of room behind
            token, head = (N * H * d, d, H * d), (H * N * d, N * d, d)
            for st in (token, head):
                assert _layout(lib, Hq * st[1], st, st, B, Hq, Hk, N) == 3, (B, Hq, Hk, N, st)
                swapped = {"qo": _p(6) + 2 * Hk * st[1], "ko": _p(6), "qw": _p(50) + 8}
                assert _fwd(lib, swapped, ((Hq * N * d, N * d, d), (Hk * N * d, N * d, d), st, st), B, Hq, Hk, N, d) == 3
                if Hq > 1:
                    assert _layout(lib, (Hq - 1) * st[1], st, st, B, Hq, Hk, N) == 8
    r = random.Random(3)
    seen = {3: 0, 8: 0}
    for _ in range(4000):
        B, Hq, Hk, N = (r.choice([1, 2, 3]) for _ in range(4))
        steps = sorted(d * r.choice([1, 1, 2, 3, 4, 6, 9]) for _ in range(3))
        order = r.sample(range(3), 3)
        sq = tuple(steps[i] for i in order)
        sk = sq if r.random() < 0.8 else tuple(r.sample(steps, 3))
        ko = r.choice([d * r.randint(0, 30), 8 * r.randint(0, 240)])
        rows = lambda off, st, H: [off + b * st[0] + h * st[1] + n * st[2]  # noqa: E731
                                   for b in range(B) for h in range(H) for n in range(N)]
        at = sorted(rows(0, sq, Hq) + rows(ko, sk, Hk))
        apart = all(y - x >= d for x, y in zip(at, at[1:]))
        got = _layout(lib, ko, sq, sk, B, Hq, Hk, N)
        assert got == 8 or (got == 3 and apart), (B, Hq, Hk, N, sq, sk, ko)
        seen[got] += 1
    assert seen[3] > 300


def test_backward_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    names = ("dq", "dk", "q", "k", "f", "pos", "qw", "kw", "qg", "kg", "qwg", "kwg", "ws")
    ws = lib.fa2_rotary_bwd_workspace_size(B, HQ, HK, N, D, 1)
    assert ws > 0 and lib.fa2_rotary_bwd_workspace_size(B, HQ, HK, N, 96, 1) == 0
    assert lib.fa2_rotary_bwd_workspace_size(0, HQ, HK, N, D, 1) == 0

    def call(ptr=None, st=None, d=D, r=32, wsz=ws, wt=1):
        p = {n: _p(i) for i, n in enumerate(names)}
        p.update(ptr or {})
        s = st or (CQ, CK, CQ, CK, CQ, CK)
        return lib.fa2_rotary_bwd(*(p[n] for n in names[:12]), _strides(*s), B, HQ, HK, N, d, r, 1, 0, 1e-6, 1.0, 1, wt,
                                  p["ws"], wsz, None)

    for n in names[:-1]:
        assert call({n: 0}) == 1, n
    assert call(d=32) == 2 and call(r=17) == 2 and call(wt=0) == 1
    for n in ("dq", "dk", "q", "k", "qg", "kg", "qw", "qwg", "kwg", "ws"):
        assert call({n: _p(50) + 8}) == 3, n
    assert call({"ws": 0}) == 7 and call(wsz=ws - 1) == 7
    for out in ("qg", "kg", "qwg", "kwg", "ws"):
        for other in names:
            if other != out:
                assert call({out: _p(names.index(other))}) == 8, (out, other)
    assert call(st=(CQ, CK, CQ, CK, (0, N * D, D), CK)) == 8


def test_binding_rejects_host_tensors(fa2_lib):
    x, f = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        fa2_lib.rotary_forward(x, x.clone(), f)
    with pytest.raises(ValueError):
        fa2_lib.rotary_backward(x, None, f)
    with pytest.raises(ValueError):
        fa2_lib.rotary(x, None, f)
