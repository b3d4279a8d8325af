"""fa2_cache_resize refuses bad arguments before touching a device."""

A, STEP = 0x100000000, 0x10000000
NAMES = ("table", "lens", "new", "refs", "free", "nf", "out", "ws")


def test_rejects(fa2_lib):
    lib = fa2_lib.load_library()
    ws = lib.fa2_cache_resize_workspace_size(3, 100, 16, 10)
    assert ws == 512 + 256 and lib.fa2_cache_resize_workspace_size(3, 0, 16, 10) == 0
    assert lib.fa2_cache_resize_workspace_size(65535, 100, 1, 2 ** 20) == 0

    def call(ptr=None, B=3, pages=100, ps=16, mp=10, wsz=ws):
        p = {n: A + i * STEP for i, n in enumerate(NAMES)}
        p.update(ptr or {})
        return lib.fa2_cache_resize(*(p[n] for n in NAMES[:7]), B, pages, ps, mp, p["ws"], wsz, None)

    for n in NAMES[:7]:
        assert call({n: 0}) == 1, n
        assert call({n: A + 50 * STEP + 2}) == 3, n
    for kw in (dict(B=0), dict(pages=0), dict(ps=0), dict(mp=0)):
        assert call(**kw) == 1, kw
    for kw in (dict(B=65536), dict(B=65535, mp=2 ** 20, ps=1), dict(mp=2 ** 20, ps=2 ** 11)):
        assert call(**kw) == 2, kw
    assert call({"ws": 0}) == 7 and call(wsz=ws - 1) == 7 and call({"ws": A + 50 * STEP + 16}) == 3
    outs = ("table", "refs", "free", "nf", "out", "ws")
    for o in outs:
        for other in NAMES:
            if other != o:
                assert call({o: A + NAMES.index(other) * STEP}) == 8, (o, other)


def test_numbers_of_pages_stay_below_two_to_the_31(fa2_lib):
    """A release's or a take's number may pass their count by a step of 8192."""
    lib = fa2_lib.load_library()
    size = lambda B, mp: lib.fa2_cache_resize_workspace_size(B, 100, 1, mp)  # noqa: E731
    most = 2 ** 31 - 2 ** 14
    assert size(2, most // 2) == 512 + most * 4
    for B, mp in ((2, most // 2 + 1), (49981, 42966), (3, 715827882)):  # the last two: 2^31 - 2
        assert most < B * mp < 2 ** 31 and size(B, mp) == 0
        p = [A + i * STEP * 16 for i in range(8)]
        assert lib.fa2_cache_resize(*p[:7], B, 100, 1, mp, p[7], 2 ** 40, None) == 2
