"""The cache's kernels are launched before what precedes them in the stream has
ended, and must still see all of it: results without a synchronisation, behind
work of other streams, and in graphs, bit for bit those of one call at a time."""

import ctypes

import pytest
import torch

from tests.cache_cases import BF16, Cache

pytestmark = pytest.mark.gpu

BUSY = 4_000_000  # clocks that a producer waits before it writes: some 2 ms


def _generate(fa2, steps, wait, d=128, ps=16, B=4, Hkv=2, g=4, start=190, budget=200):
    """Tokens appended, attended to and evicted over lengths in device memory
    that change in every step; `wait()` after each call."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    c = Cache(B, Hkv, d, ps, [start] * B, BF16, seed=3, width=-(-(budget + 1) // ps))
    kc, vc, table, lens = c.gpu()
    weights = c.weights().cuda()
    positions = torch.arange(c.L, dtype=torch.int32).expand(B, Hkv, c.L).contiguous().cuda()
    next_pos = lens.clone()
    tokens = [(rnd(B, Hkv * g, d), rnd(B, Hkv, 1, d), rnd(B, Hkv, 1, d)) for _ in range(steps)]
    torch.cuda.synchronize()
    out = []
    for q, k, v in tokens:
        lens = fa2.cache_append(k, v, kc, vc, table, lens, weights=weights, positions=positions, next_pos=next_pos)
        wait()
        next_pos = next_pos + 1
        o, lse = fa2.paged_decode(q, kc, vc, table, lens, weights=weights)
        wait()
        lens = fa2.cache_evict(kc, vc, table, lens, weights, budget, recent=16, positions=positions,
                               next_pos=next_pos)
        wait()
        out += [o, lse, lens]
    torch.cuda.synchronize()
    assert fa2.device_status() == 0
    return out + [weights.clone(), positions.clone()]


@pytest.mark.parametrize("kw", [{}, {"d": 64, "ps": 24, "g": 1}, {"B": 1, "start": 4200, "budget": 4210}],
                         ids=["d128", "d64", "cluster"])
def test_calls_in_a_row_are_calls_one_by_one(cuda_device, fa2_lib, kw):
    one = _generate(fa2_lib, 60, torch.cuda.synchronize, **kw)
    for _ in range(3):
        row = _generate(fa2_lib, 60, lambda: None, **kw)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(one, row))


class _Late:
    """Each operator on inputs that another stream writes late."""

    def __init__(self, fa2):
        self.c = Cache(2, 2, 64, 16, [300, 77], BF16, seed=5)
        self.real = [t.contiguous() for t in self.c.gpu()]
        self.q = self.c.query(4).cuda()
        self.new = torch.randn(2, 2, 1, 64, generator=self.c.g).to(BF16).cuda()
        self.w = self.c.weights().cuda()
        self.qp, self.kp = (torch.randn(2, 2, 300, 64, generator=self.c.g).to(BF16).cuda() for _ in range(2))
        self.lse = torch.full((2, 2, 300), 6.0, device="cuda")
        self.n = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
        self.buf = [torch.zeros_like(t) for t in self.real]
        self.qlen = torch.zeros_like(self.n)
        self.x = torch.zeros(64, device="cuda")
        self.fa2 = fa2

    def produce(self):
        torch.cuda._sleep(BUSY)
        for b, r in zip(self.buf, self.real):
            b.copy_(r)
        self.qlen.copy_(self.n)

    def call(self, op):
        kc, vc, table, lens = self.buf
        if op == "decode":
            return self.fa2.paged_decode(self.q, kc, vc, table, lens)
        if op == "append":
            return [self.fa2.cache_append(self.new, self.new, kc, vc, table, lens), kc, vc]
        if op == "evict":
            w = self.w.clone()
            return [self.fa2.cache_evict(kc, vc, table, lens, w, 60), w, kc, vc]
        return [self.fa2.key_weights(self.qp, self.kp, self.lse, causal=True, q_lens=self.qlen)]

    def reset(self):
        for b in self.buf + [self.qlen, self.x]:
            b.zero_()
        torch.cuda.synchronize()

    def step(self, op, before):
        """The producer on a stream of its own; on this one a kernel, a copy or
        nothing, the wait for it, and the call."""
        main, side = torch.cuda.current_stream(), torch.cuda.Stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            self.produce()
        done = torch.cuda.Event()
        done.record(side)
        if before == "kernel":
            self.x.add_(1)
        elif before == "copy":
            self.x.copy_(torch.zeros_like(self.x))
        main.wait_event(done)
        if before == "kernel":
            self.x.add_(1)
        return self.call(op)


@pytest.mark.parametrize("op", ["decode", "append", "evict", "key_weights"])
@pytest.mark.parametrize("before", ["nothing", "kernel", "copy"])
def test_inputs_of_another_stream(cuda_device, fa2_lib, op, before):
    s = _Late(fa2_lib)
    s.reset()
    s.produce()
    torch.cuda.synchronize()
    want = [t.clone() for t in s.call(op)]
    for _ in range(3):
        s.reset()
        got = s.step(op, before)
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, want))
    assert fa2_lib.device_status() == 0


@pytest.mark.parametrize("op", ["decode", "append", "evict", "key_weights"])
@pytest.mark.parametrize("before", ["nothing", "kernel"])
def test_inputs_of_another_stream_in_a_graph(cuda_device, fa2_lib, op, before):
    s = _Late(fa2_lib)
    s.reset()
    s.produce()
    torch.cuda.synchronize()
    want = [t.clone() for t in s.call(op)]
    s.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step(op, before)
        after = [t.clone() for t in got]
    for _ in range(3):
        s.reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(after, want))
    assert fa2_lib.device_status() == 0


@pytest.mark.parametrize("op", ["decode", "append", "evict", "key_weights"])
def test_the_default_stream_waits_for_blocking_streams(cuda_device, fa2_lib, op):
    """The producer on a stream that the default stream synchronises with, and
    no event."""
    s = _Late(fa2_lib)
    s.reset()
    s.produce()
    torch.cuda.synchronize()
    want = [t.clone() for t in s.call(op)]
    raw = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(raw))) == 0
    side = torch.cuda.ExternalStream(raw.value)
    try:
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        for _ in range(3):
            s.reset()
            s.x.add_(1)
            with torch.cuda.stream(side):
                s.produce()
            got = s.call(op)
            torch.cuda.synchronize()
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, want))
    finally:
        torch.cuda.synchronize()
        assert int(torch.cuda.cudart().cudaStreamDestroy(raw.value)) == 0
    assert fa2_lib.device_status() == 0
