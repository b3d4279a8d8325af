"""fa2_prefix_decode refuses bad arguments before touching a device."""

A, STEP = 0x100000000, 0x10000000
NAMES = ("q", "k", "v", "table", "lens", "prefix", "plen", "o", "lse", "ws")


def test_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    ws = lib.fa2_prefix_decode_workspace_size(2, 8, 2, 64, 16, 4)
    assert ws > 0 and lib.fa2_prefix_decode_workspace_size(2, 7, 2, 64, 16, 4) == 0
    assert lib.fa2_prefix_decode_workspace_size(2, 8, 2, 96, 16, 4) == 0

    def call(ptr=None, B=2, Hq=8, Hkv=2, d=64, pages=10, ps=16, mp=4, pp=3, scale=0.1, dtype=1, wsz=ws):
        p = {n: A + i * STEP for i, n in enumerate(NAMES)}
        p.update(ptr or {})
        return lib.fa2_prefix_decode(*(p[n] for n in NAMES[:9]), B, Hq, Hkv, d, pages, ps, mp, pp, scale, dtype, p["ws"],
                                     wsz, None)

    for n in NAMES[:9]:
        assert call({n: 0}) == 1, n
    for kw in (dict(B=0), dict(Hq=7), dict(Hkv=0), dict(pages=0), dict(ps=0), dict(mp=0), dict(pp=0), dict(pp=-1),
               dict(scale=-1.0), dict(scale=float("nan")), dict(dtype=2)):
        assert call(**kw) == 1, kw
    for kw in (dict(d=96), dict(B=70000), dict(Hq=258), dict(pages=2 ** 30), dict(mp=2 ** 30), dict(pp=2 ** 28)):
        assert call(**kw) == 2, kw
    for n, off in (("q", 8), ("k", 2), ("v", 4), ("o", 8), ("table", 2), ("lens", 1), ("lse", 2), ("prefix", 2),
                   ("plen", 2), ("ws", 16)):
        assert call({n: A + 50 * STEP + off}) == 3, n
    assert call({"ws": 0}) == 7 and call(wsz=ws - 1) == 7
    for out in ("o", "lse", "ws"):
        for other in NAMES:
            if other != out:
                assert call({out: A + NAMES.index(other) * STEP}) == 8, (out, other)
    assert lib.fa2_debug_arm_fault(7, 10) == 0 and lib.fa2_debug_arm_fault(0, 0) == 0
    assert lib.fa2_debug_arm_fault(8, 10) == 1
