"""Pins of the fp64 reference of rotary positions, and of the frequencies (CPU)."""

import math

import numpy as np
import pytest

from oracle import rotary as orc


def _case(seed, B=2, H=3, N=5, d=8, r=6):
    g = np.random.default_rng(seed)
    x = g.standard_normal((B, H, N, d))
    return x, 100.0 ** (-np.arange(r // 2) / r), g.integers(0, 1000, (B, N)), 1.0 + 0.1 * g.standard_normal(d)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turns(interleaved):
    x, f, pos, _ = _case(0)
    y = orc.rotary(x, f, pos, interleaved, amplitude=1.5)
    a, b = orc.pairs(6, interleaved)
    z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * pos[:, None, :, None] * f)
    assert np.allclose(y[..., a] + 1j * y[..., b], z, atol=1e-12) and (y[..., 6:] == x[..., 6:]).all()
    back, _ = orc.rotary_backward(y, None, f, pos, interleaved, amplitude=1.5)
    assert np.allclose(back[..., :6], 2.25 * x[..., :6])


def test_scores_depend_on_the_distance():
    q, f, _, _ = _case(1, B=1, H=1, N=1)
    k, _, _, _ = _case(2, B=1, H=1, N=1)
    at = lambda x, p: orc.rotary(x, f, np.array([[p]]))[0, 0, 0]  # noqa: E731
    assert math.isclose(at(q, 17) @ at(k, 11), at(q, 106) @ at(k, 100), rel_tol=1e-9)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(interleaved, norm):
    x, f, pos, w = _case(3, N=3)
    dy = np.random.default_rng(4).standard_normal(x.shape)
    kw = dict(interleaved=interleaved, weight=w if norm else None, amplitude=1.2)
    dx, dw = orc.rotary_backward(dy, x, f, pos, **kw)
    loss = lambda x, kw: (orc.rotary(x, f, pos, **kw) * dy).sum()  # noqa: E731
    h = 1e-6
    for i in np.random.default_rng(5).integers(0, x.size, 40):
        e = np.zeros(x.size)
        e[i] = h
        e = e.reshape(x.shape)
        assert math.isclose((loss(x + e, kw) - loss(x - e, kw)) / (2 * h), dx.flat[i], rel_tol=1e-6, abs_tol=1e-7)
    if norm:
        for i in range(8):
            e = h * (np.arange(8) == i)
            d = (loss(x, {**kw, "weight": w + e}) - loss(x, {**kw, "weight": w - e})) / (2 * h)
            assert math.isclose(d, dw[i], rel_tol=1e-6, abs_tol=1e-7)


def test_frequencies(fa2_lib):
    f = fa2_lib.rotary_frequencies
    plain = f(64, base=500000.0)
    assert plain.shape == (32,) and plain[0] == 1.0 and math.isclose(plain[16], 500000.0 ** -0.5)
    assert np.allclose(f(64, base=500000.0, factor=8), plain / 8)
    based = f(64, base=500000.0, factor=8, method="base")
    assert based[0] == 1.0 and math.isclose(based[-1], plain[-1] / 8)
    bands = f(64, base=500000.0, factor=8, method="bands", original=8192)
    turns = 8192 * plain / (2 * math.pi)
    assert (bands[turns >= 4] == plain[turns >= 4]).all() and np.allclose(bands[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((bands < plain) & (bands > plain / 8))[mid].all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, method="x"), dict(rotary_dim=2, method="base"),
                dict(rotary_dim=8, method="bands", low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            f(**bad)
