"""Rotary positions and the per-head norm against the definition in 64 bits."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import rotary as orc
from tests.cache_cases import BF16, FP16, bits64

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _half(t):
    return torch.finfo(t).eps / 2


def _inputs(B, Hq, Hk, N, d, dtype, seed, packed=True, std=1.5):
    """q and k as views of a projection's output (packed), or contiguous."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, N, Hq + 2 * Hk, d, generator=g) * std).to(dtype).cuda()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    return (q, k, g) if packed else (q.contiguous(), k.contiguous(), g)


def _bound(u, y, f, pos, r, inter, amp, dtype, norm):
    """y is rounded once. cos and sin are off by 2^-22 (angle 2^-25 turns, function
    2 steps, amplitude), a product and a sum by a half step each; the norm's sum of d
    squares by d half steps, halved by the root, and the root and two products."""
    d = u.shape[-1]
    a, b = orc.pairs(r, inter)
    big = np.abs(u)
    big[..., a] = big[..., b] = abs(amp) * (np.abs(u[..., a]) + np.abs(u[..., b]))
    rel = 2.0 ** -21 + ((d / 2 + 8) * 2.0 ** -24 if norm else 0.0)
    return _half(dtype) * np.abs(y) * 1.01 + big * rel + (2.0 ** -25 if dtype == FP16 else 0.0)


def _positions(mode, B, N, g):
    if mode == "none":
        return None, np.tile(np.arange(N), (B, 1))
    if mode == "first":
        p = torch.randint(-5000, 2000000, (B,), generator=g, dtype=torch.int32)
        return p.cuda(), p.numpy()[:, None].astype(np.int64) + np.arange(N)
    p = torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, N), generator=g, dtype=torch.int64)
    p[0, 0], p[-1, -1] = 0, 2 ** 31 - 1
    return p.int().cuda(), p.numpy()


CASES = [  # B, Hq, Hk, N, d, r, dtype, interleaved, weights, positions, packed
    (1, 1, 1, 1, 64, 64, BF16, False, None, "none", True),
    (2, 4, 1, 1, 128, 128, FP16, True, F32, "first", True),
    (3, 5, 3, 37, 64, 16, BF16, False, "same", "first", True),
    (2, 9, 2, 70, 128, 96, FP16, False, None, "each", False),
    (2, 7, 7, 33, 128, 48, BF16, True, F32, "none", False),
    (1, 40, 8, 129, 64, 32, FP16, True, "same", "each", True),
    (40, 3, 1, 50, 128, 64, BF16, False, F32, "each", True),
    (2, 32, 8, 300, 128, 128, BF16, False, None, "first", True),
    (1, 2, 0, 19, 64, 48, FP16, True, F32, "first", False),
]


def _weights(spec, d, dtype, g, n=2):
    if spec is None:
        return [None] * n
    dt = dtype if spec == "same" else spec
    return [(1 + 0.2 * torch.randn(d, generator=g)).to(dt).cuda() for _ in range(n)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_forward(cuda_device, fa2_lib, case):
    B, Hq, Hk, N, d, r, dtype, inter, wspec, mode, packed = case
    q, k, g = _inputs(B, Hq, max(Hk, 1), N, d, dtype, seed=d + N, packed=packed)
    k = k if Hk else None
    f = fa2_lib.rotary_frequencies(r, base=10000.0)
    p, pos = _positions(mode, B, N, g)
    wq, wk = _weights(wspec, d, dtype, g)
    amp = 1.25
    qo, ko = fa2_lib.rotary_forward(q, k, f.cuda(), p, interleaved=inter, q_weight=wq,
                                    k_weight=wk if k is not None else None, eps=1e-5, amplitude=amp)
    assert (ko is None) == (k is None) and qo.is_contiguous()
    for x, y, w in ((q, qo, wq), (k, ko, wk)):
        if x is None:
            continue
        ref = orc.rotary(bits64(x), f.numpy(), pos, inter, None if w is None else bits64(w), 1e-5, amp)
        u = orc.rotary(bits64(x), f.numpy(), 0 * pos, inter, None if w is None else bits64(w), 1e-5, 1.0)
        # at far positions the angle of the fp64 reference itself is off by its product's half step
        far = np.abs(pos).max() * f.numpy().max() * 2.0 ** -52 * 2
        tol = _bound(u, ref, f, pos, r, inter, amp, dtype, w is not None) + far * 2 * amp * np.abs(u).max()
        assert (np.abs(bits64(y) - ref) <= tol).all()
    assert fa2_lib.device_status() == 0


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_backward(cuda_device, fa2_lib, case):
    B, Hq, Hk, N, d, r, dtype, inter, wspec, mode, packed = case
    q, k, g = _inputs(B, Hq, max(Hk, 1), N, d, dtype, seed=d + N + 1, packed=packed)
    k = k if Hk else None
    f = fa2_lib.rotary_frequencies(r, base=500.0)
    p, pos = _positions(mode, B, N, g)
    wq, wk = _weights(wspec, d, dtype, g)
    wk = wk if k is not None else None
    dq, dk, _ = _inputs(B, Hq, max(Hk, 1), N, d, dtype, seed=d + N + 2, packed=not packed, std=1.0)
    dk = dk if k is not None else None
    amp, eps = 0.75, 1e-5
    kw = dict(q=q, k=k) if wq is not None else {}
    qg, kg, qwg, kwg = fa2_lib.rotary_backward(dq, dk, f.cuda(), p, interleaved=inter, q_weight=wq, k_weight=wk,
                                               eps=eps, amplitude=amp, **kw)
    again = fa2_lib.rotary_backward(dq, dk, f.cuda(), p, interleaved=inter, q_weight=wq, k_weight=wk, eps=eps,
                                    amplitude=amp, **kw)
    for a, b in zip((qg, kg, qwg, kwg), again):
        assert (a is None and b is None) or torch.equal(a, b)
    for x, dy, got, w, wg in ((q, dq, qg, wq, qwg), (k, dk, kg, wk, kwg)):
        if x is None:
            continue
        X, G = bits64(x), bits64(dy)
        W = None if w is None else bits64(w)
        ref, dw = orc.rotary_backward(G, X, f.numpy(), pos, inter, W, eps, amp)
        gt = orc.turn(G, f.numpy(), pos, inter, amp, back=True)
        far = np.abs(pos).max() * f.numpy().max() * 2.0 ** -52 * 4 * amp * np.abs(G).max()
        turn_err = _bound(G, 0 * G, f, pos, r, inter, amp, FP16, False) + far
        if w is None:
            assert wg is None
            assert (np.abs(bits64(got) - ref) <= turn_err + _half(dtype) * np.abs(ref) * 1.01).all()
            continue
        n = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + eps)
        xh = np.abs(X * n)
        # g is off by turn_err; x n by (d / 2 + 8) half steps, the mean by d more
        rel = (2 * d + 32) * 2.0 ** -24
        ge = turn_err * np.abs(W)
        dot = (np.abs(W * gt) * xh).mean(-1, keepdims=True)
        tol = n * (ge + xh * (ge * xh).mean(-1, keepdims=True) + rel * (np.abs(W * gt) + xh * dot))
        assert (np.abs(bits64(got) - ref) <= tol + _half(dtype) * np.abs(ref) * 1.01 + 2.0 ** -25).all()
        # a sum of M = B H N terms in fp32: at most M half steps of the magnitudes
        M = X[..., 0].size
        terms = np.abs(gt) * xh
        tol = (turn_err * xh).sum((0, 1, 2)) + (rel + min(M, 4096) * 2.0 ** -24) * terms.sum((0, 1, 2))
        assert (np.abs(bits64(wg) - dw) <= tol + _half(w.dtype) * np.abs(dw) * 1.01).all()


@pytest.mark.parametrize("case", [
    (3, 61, 7, 2301, 64, 32, BF16, False, F32, "first", True),
    (1, 8, 1, 1793, 128, 128, FP16, True, "same", "each", False),
    (2, 130, 1, 45, 64, 64, BF16, True, F32, "none", False),
], ids=["large-and-small-ctas", "cuts-inside-tokens", "one-head-of-a-block-each"])
def test_backward_with_norm_dealt_to_many_ctas(cuda_device, fa2_lib, case):
    test_backward(cuda_device, fa2_lib, case)


# 1 / 2 pi, to 60 digits
TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


@pytest.mark.parametrize("N", [40, 1800])
def test_angles_at_far_positions_and_high_frequencies(cuda_device, fa2_lib, N):
    """An angle is right to 2^-31 turns for frequencies up to 2^40 at any position: against
    angles in exact arithmetic (an fp64 product of the two is off by up to 2^18 there). With
    half a step of fp16 and the bound that all turns are held to; N = 1800: by units."""
    d, H = 64, 60
    f = torch.tensor([2.0 ** 40 * 10 ** (-0.55 * j) for j in range(d // 2)], dtype=torch.float64)
    g = torch.Generator().manual_seed(N)
    p = torch.randint(-(2 ** 31), 2 ** 31 - 1, (1, N), generator=g, dtype=torch.int64)
    p[0, :4] = torch.tensor([2 ** 31 - 1, -(2 ** 31), 1, 0])
    x = torch.randn(1, H, N, d, generator=g).to(FP16)
    check = list(range(0, N, max(1, N // 40)))
    t = np.array([[float((int(pos) * Fraction(w) * TURN) % 1) for w in f.tolist()] for pos in p[0, check].tolist()])
    c, s = np.cos(2 * np.pi * t), np.sin(2 * np.pi * t)
    a, b = orc.pairs(d, False)
    u = bits64(x)[:, :, check]
    ref = np.empty_like(u)
    ref[..., a], ref[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
    y, _ = fa2_lib.rotary_forward(x.cuda(), None, f.cuda(), p.int().cuda())
    tol = _bound(u, ref, f, p.numpy(), d, False, 1.0, FP16, False)
    assert (np.abs(bits64(y)[:, :, check] - ref) <= tol).all()


@pytest.mark.parametrize("inter", [False, True])
def test_nothing_else_is_touched(cuda_device, fa2_lib, inter):
    """Passed-through elements keep their bits, and inputs that are not finite reach
    their own pair only."""
    x = torch.randn(2, 3, 9, 128).to(BF16).cuda()
    x[1, 2, 4, 5], x[0, 0, 0, 100] = float("inf"), float("nan")
    y, _ = fa2_lib.rotary_forward(x, None, fa2_lib.rotary_frequencies(32).cuda(), interleaved=inter)
    assert torch.equal(y[..., 32:].view(torch.int16), x[..., 32:].view(torch.int16))
    bad = ~torch.isfinite(y[..., :32])
    a, b = orc.pairs(32, inter)
    j = int(np.where((a == 5) | (b == 5))[0][0])
    want = torch.zeros_like(bad)
    want[1, 2, 4, int(a[j])] = want[1, 2, 4, int(b[j])] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("case", [
    (3, 61, 7, 2301, 64, 32, BF16, False, F32, "first", True),
    (2, 20, 4, 1111, 128, 96, FP16, True, None, "each", False),
    (1, 40, 0, 2500, 64, 48, BF16, False, None, "none", True),
    (5, 9, 8, 601, 128, 128, FP16, False, "same", "first", False),
], ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_turns_dealt_by_units(cuda_device, fa2_lib, case):
    test_forward(cuda_device, fa2_lib, case)
    test_backward(cuda_device, fa2_lib, case)


def test_nothing_else_is_touched_by_units(cuda_device, fa2_lib):
    """The same of a call that is dealt by units; also rows with gaps around the outputs."""
    x = torch.randn(2, 30, 1700, 128).to(BF16).cuda()
    x[1, 29, 1699, 5], x[0, 0, 0, 100], x[0, 7, 900, 127] = float("inf"), float("nan"), float("nan")
    buf = torch.full((2, 1700, 32, 128), 3.0, dtype=BF16, device="cuda")
    y = buf[:, :, 1:31].transpose(1, 2)
    fa2_lib.rotary_forward(x, None, fa2_lib.rotary_frequencies(32).cuda(), q_out=y)
    assert torch.equal(y[..., 32:].contiguous().view(torch.int16), x[..., 32:].contiguous().view(torch.int16))
    assert (buf[:, :, 0] == 3).all() and (buf[:, :, 31] == 3).all()
    bad = (~torch.isfinite(y[..., :32])).nonzero().tolist()
    assert bad == [[1, 29, 1699, 5], [1, 29, 1699, 21]]


def test_rows_of_zeros_and_eps(cuda_device, fa2_lib):
    x = torch.zeros(1, 2, 5, 64, dtype=FP16, device="cuda")
    w = torch.ones(64, device="cuda")
    f = fa2_lib.rotary_frequencies(64).cuda()
    y, _ = fa2_lib.rotary_forward(x, None, f, q_weight=w)
    g, _, wg, _ = fa2_lib.rotary_backward(torch.ones_like(x), None, f, q=x, q_weight=w, eps=1.0)
    assert (y == 0).all() and (wg == 0).all() and torch.isfinite(g).all()


def test_strided_outputs_side_by_side(cuda_device, fa2_lib):
    """Gradients written into the packed gradient of a projection; the values' part stays."""
    B, Hq, Hk, N, d = 2, 4, 2, 21, 64
    q, k, g = _inputs(B, Hq, Hk, N, d, BF16, seed=3)
    dq, dk = torch.randn(B, Hq, N, d).to(BF16).cuda(), torch.randn(B, Hk, N, d).to(BF16).cuda()
    f = fa2_lib.rotary_frequencies(64).cuda()
    w = [torch.rand(d, generator=g).cuda() for _ in range(2)]
    buf = torch.full((B, N, Hq + 2 * Hk, d), 7.0, dtype=BF16, device="cuda")
    qv, kv = buf[:, :, :Hq].transpose(1, 2), buf[:, :, Hq:Hq + Hk].transpose(1, 2)
    for norm in (True, False):
        kw = dict(q=q, k=k, q_weight=w[0], k_weight=w[1]) if norm else {}
        want = fa2_lib.rotary_backward(dq, dk, f, **kw)
        got = fa2_lib.rotary_backward(dq, dk, f, q_grad=qv, k_grad=kv, **kw)
        assert got[0].data_ptr() == qv.data_ptr()
        assert torch.equal(qv, want[0]) and torch.equal(kv, want[1]) and (buf[:, :, Hq + Hk:] == 7).all()
    qo, ko = fa2_lib.rotary_forward(q, k, f)
    buf.fill_(7.0)
    fa2_lib.rotary_forward(q, k, f, q_out=qv, k_out=kv)
    assert torch.equal(qv, qo) and torch.equal(kv, ko) and (buf[:, :, Hq + Hk:] == 7).all()
    e = q[:, :1].expand(B, Hq, N, d)  # a broadcast input
    qe, _ = fa2_lib.rotary_forward(e, None, f)
    want, _ = fa2_lib.rotary_forward(e.contiguous(), None, f)
    assert torch.equal(qe, want)


@pytest.mark.parametrize("norm", [False, True])
def test_autograd(cuda_device, fa2_lib, norm):
    """rotary() feeds attention(); its gradients are those of rotary_backward, also
    when only one output is used or the gradients come in another layout."""
    B, H, N, d = 2, 3, 40, 64
    q0, k0, g = _inputs(B, H, H, N, d, BF16, seed=5)
    f = fa2_lib.rotary_frequencies(32).cuda()
    pos = torch.tensor([3, 100], dtype=torch.int32, device="cuda")
    ws = _weights(F32 if norm else None, d, BF16, g)
    leaf = lambda t: None if t is None else t.detach().clone(memory_format=torch.preserve_format).requires_grad_()  # noqa: E731
    q, k, wq, wk = leaf(q0), leaf(k0), leaf(ws[0]), leaf(ws[1])
    v = torch.randn(B, H, N, d).to(BF16).cuda()
    qr, kr = fa2_lib.rotary(q, k, f, pos, q_weight=wq, k_weight=wk, amplitude=1.1)
    o = fa2_lib.attention(qr, kr, v, causal=True)
    do = torch.randn(B, H, N, d).to(BF16).cuda()
    o.backward(do)
    o2, lse = fa2_lib.forward(qr.detach(), kr.detach(), v, causal=True)
    dq, dk, _ = fa2_lib.backward(qr.detach(), kr.detach(), v, o2, lse, do, causal=True)
    kw = dict(q=q0, k=k0, q_weight=ws[0], k_weight=ws[1]) if norm else {}
    want = fa2_lib.rotary_backward(dq, dk, f, pos, amplitude=1.1, **kw)
    for t, w in zip((q, k, wq, wk), want):
        assert (t is None) == (w is None)
        if t is not None:
            assert torch.equal(t.grad, w)
    # only the keys are used, and their gradient is not in rows
    q, k, wq, wk = leaf(q0), leaf(k0), leaf(ws[0]), leaf(ws[1])
    _, kr = fa2_lib.rotary(q, k, f, pos, q_weight=wq, k_weight=wk, amplitude=1.1)
    kr.transpose(2, 3).backward(dk.transpose(2, 3).contiguous())
    assert q.grad is None and (wq is None or wq.grad is None)
    assert torch.equal(k.grad, want[1]) and (wk is None or torch.equal(wk.grad, want[3]))


def test_autograd_of_one_tensor(cuda_device, fa2_lib):
    q0, _, g = _inputs(2, 3, 1, 20, 64, FP16, seed=6)
    f = fa2_lib.rotary_frequencies(64).cuda()
    for w0 in (None, torch.rand(64, generator=g).cuda()):
        q = q0.detach().clone().requires_grad_()
        w = None if w0 is None else w0.clone().requires_grad_()
        y, none = fa2_lib.rotary(q, None, f, interleaved=True, q_weight=w)
        assert none is None
        dy = torch.randn(y.shape, generator=g).to(FP16).cuda()
        y.backward(dy)
        want = fa2_lib.rotary_backward(dy, None, f, interleaved=True, q=q0 if w is not None else None, q_weight=w0)
        assert torch.equal(q.grad, want[0]) and (w is None or torch.equal(w.grad, want[2]))


@pytest.mark.parametrize("norm", [False, True])
def test_a_second_gradient_raises(cuda_device, fa2_lib, norm):
    """create_graph gives the same first gradients; what depends on the norm's inputs or on
    gradients that want one raises when it is differentiated again, and a gradient that is a
    constant stays one. freqs, which has no gradient, must not want one."""
    q0, k0, g = _inputs(1, 2, 2, 9, 64, BF16, seed=7)
    f = fa2_lib.rotary_frequencies(64).cuda()
    w = [torch.rand(64, generator=g).cuda().requires_grad_() for _ in range(2)] if norm else [None, None]
    q, k = q0.detach().clone().requires_grad_(), k0.detach().clone().requires_grad_()
    leaves = [t for t in (q, k, *w) if t is not None]
    turn = lambda: fa2_lib.rotary(q, k, f, q_weight=w[0], k_weight=w[1])  # noqa: E731
    loss = lambda y: (y[0].float().square() + y[1].float() * q.detach().float()).sum()  # noqa: E731
    want = torch.autograd.grad(loss(turn()), leaves)
    got = torch.autograd.grad(loss(turn()), leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # beside a term that can be differentiated
    with pytest.raises(RuntimeError, match="differentiated"):
        torch.autograd.grad(got[0].float().square().sum() + q.float().square().sum(), q)
    got = torch.autograd.grad(turn()[1].float().sum(), k, create_graph=True)
    assert got[0].requires_grad == norm
    for t in leaves[1::2] if norm else ():
        with pytest.raises(RuntimeError, match="differentiated"):
            torch.autograd.grad(got[0].float().square().sum() + t.float().square().sum(), t, retain_graph=True)
    with pytest.raises(ValueError, match="freqs"):
        fa2_lib.rotary(q, k, f.clone().requires_grad_())
    with torch.no_grad():
        fa2_lib.rotary(q, k, f.clone().requires_grad_())


def test_gradient_against_differences(cuda_device, fa2_lib):
    """Differences of the forward itself along the gradient's signs, in its own 16 bits:
    both sides of a step h are rounded by a half step of y, over 2 h. x is on a grid
    that x +- h stays on."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(1, 2, 30, 64, generator=g).clamp(-3.5, 3.5) * 256).round().div(256).to(FP16).cuda()
    w = (1 + 0.1 * torch.randn(64, generator=g)).cuda()
    dy = torch.randn(1, 2, 30, 64, generator=g).to(FP16).cuda()
    f = fa2_lib.rotary_frequencies(64).cuda()
    y = lambda x, w: fa2_lib.rotary_forward(x, None, f, q_weight=w)[0].double()  # noqa: E731
    xg, _, wg, _ = fa2_lib.rotary_backward(dy, None, f, q=x, q_weight=w)
    noise = lambda h: float((dy.double().abs() * (y(x, w).abs() + 2 * h)).sum()) * 2.0 ** -11 / h  # noqa: E731
    for got, plus, minus, h in (
            (wg, y(x, w + 0.125 * wg.sign()), y(x, w - 0.125 * wg.sign()), 0.125),
            (xg, y(x + xg.sign() / 32, w), y(x - xg.sign() / 32, w), 1 / 32)):
        slope = float(got.double().abs().sum())
        assert noise(h) < 0.15 * slope
        # the curvature's part is of the size h^2
        assert abs(float(((plus - minus) * dy.double()).sum() / (2 * h)) - slope) <= noise(h) + 4 * h * h * slope


def test_refusals(cuda_device, fa2_lib):
    q, k, _ = _inputs(2, 4, 2, 8, 64, BF16, seed=0)
    f = fa2_lib.rotary_frequencies(64).cuda()
    w = torch.ones(64, device="cuda")
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(k=k[:1]), dict(q=q[0]), dict(freqs=f.float()),
                dict(freqs=f.cpu()), dict(positions=torch.zeros(2, device="cuda")),
                dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(q_weight=w),
                dict(q_weight=w, k_weight=w.half()), dict(q_weight=w[:32], k_weight=w), dict(q=q.transpose(2, 3)),
                dict(q_out=q.float()), dict(k=None, k_out=k), dict(k=None, k_weight=w), dict(q="x")):
        a = dict(q=q, k=k, freqs=f)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            fa2_lib.rotary_forward(**a)
    for bad, code in ((dict(freqs=f[:4]), 2), (dict(freqs=f[:31]), 2), (dict(eps=-1.0), 1),
                      (dict(amplitude=float("nan")), 1), (dict(q_out=q), 8)):
        a = dict(q=q, k=k, freqs=f)
        a.update(bad)
        with pytest.raises(fa2_lib.FA2Error) as e:
            fa2_lib.rotary_forward(**a)
        assert e.value.code == code
    x = torch.zeros(2 * 4 * 8 * 64 + 4, dtype=BF16, device="cuda")[4:].view(2, 4, 8, 64)  # 8 bytes off
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.rotary_forward(x, None, f)
    assert e.value.code == 3
    with pytest.raises(ValueError):
        fa2_lib.rotary_backward(q, k, f, q_weight=w, k_weight=w)
    with pytest.raises(ValueError):
        fa2_lib.rotary_backward(q, None, f, k=k)
    with pytest.raises(fa2_lib.FA2Error) as e:
        fa2_lib.rotary_backward(q, None, f, q=q, q_weight=w, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 7


def test_streams_and_graphs(cuda_device, fa2_lib):
    q, k, _ = _inputs(2, 8, 2, 100, 128, BF16, seed=9)
    f = fa2_lib.rotary_frequencies(128).cuda()
    pos = torch.tensor([5, 900], dtype=torch.int32, device="cuda")
    w = [torch.rand(128, device="cuda") for _ in range(2)]
    dq, dk = torch.randn(2, 8, 100, 128).to(BF16).cuda(), torch.randn(2, 2, 100, 128).to(BF16).cuda()
    step = lambda: (*fa2_lib.rotary_forward(q, k, f, pos, q_weight=w[0], k_weight=w[1]),  # noqa: E731
                    *fa2_lib.rotary_backward(dq, dk, f, pos, q=q, k=k, q_weight=w[0], k_weight=w[1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(2):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)))
        dk.copy_(torch.randn(dk.shape, generator=torch.Generator().manual_seed(seed + 9)))
        pos += 1000
        graph.replay()
        got = [t.clone() for t in out]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_captured_training_step(cuda_device, fa2_lib):
    """Forward and backward through autograd, captured; gradients by autograd.grad."""
    q, k, g = _inputs(2, 4, 4, 50, 64, BF16, seed=11)
    f = fa2_lib.rotary_frequencies(64).cuda()
    q, k = q.detach().clone().requires_grad_(), k.detach().clone().requires_grad_()
    w = [torch.rand(64, generator=g).cuda().requires_grad_() for _ in range(2)]
    v, do = torch.randn(2, 4, 50, 64).to(BF16).cuda(), torch.randn(2, 4, 50, 64).to(BF16).cuda()

    def step():
        qr, kr = fa2_lib.rotary(q, k, f, q_weight=w[0], k_weight=w[1])
        return torch.autograd.grad(fa2_lib.attention(qr, kr, v, causal=True), (q, k, *w), do)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(2):
        with torch.no_grad():
            q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)))
            w[1].copy_(torch.rand(64, generator=torch.Generator().manual_seed(seed + 5)))
        graph.replay()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
