"""The rotary entry points refuse bad arguments before touching a device: the C ABI
with made-up addresses, and the binding with host tensors."""

import ctypes

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
