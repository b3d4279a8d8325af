"""An eviction whose moves no launch could hold is refused before anything runs."""

SPACE = 1 << 58  # between the made-up addresses: no two buffers overlap


def test_evict_refuses_more_moves_than_a_launch_holds(fa2_lib):
    lib = fa2_lib.load_library()

    def call(B, Hkv, ps, mp, budget):
        ws = 2 * B * Hkv * min(budget, ps * mp - budget) * 4 + 4 * B * Hkv + 4096
        return lib.fa2_cache_evict(*((i + 1) * SPACE for i in range(10)), B, Hkv, 64, 1, ps, mp, budget, 0, 1,
                                   11 * SPACE, ws, None)

    for B, Hkv, ps, mp, budget in ((65535, 2000, 1 << 20, 256, 1 << 27), (65535, 2048, 1100, 2, 1100),
                                   (65535, 2000, 1024, 4, 1025)):
        assert call(B, Hkv, ps, mp, budget) == 2, (B, Hkv)
        assert lib.fa2_cache_evict_workspace_size(B, Hkv, ps, mp, budget) == 0
    # One launch makes short lists itself: nothing to refuse for their length.
    assert lib.fa2_cache_evict_workspace_size(65535, 2000, 1024, 2, 256) > 0
    assert lib.fa2_cache_evict_workspace_size(65535, 2000, 1024, 2, 2048) > 0
