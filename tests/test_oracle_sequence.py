"""Pins of the sequence operators' oracle: against the decode recurrence, and
every gradient against central differences of the forward."""

import numpy as np
import pytest

from oracle import mamba2 as M
from oracle import sequence as Q

STARTS = np.array([0, 5, 5, 6, 11])


def _scan(rng, H=4, P=3, N=5, G=2):
    T, n = int(STARTS[-1]), len(STARTS) - 1
    return dict(x=rng.normal(size=(T, H, P)), dt=rng.uniform(0.05, 0.8, (T, H)),
                A=-rng.uniform(0.3, 3.0, H), B=rng.normal(size=(T, G, N)),
                C=rng.normal(size=(T, G, N)), D=rng.normal(size=H),
                init=rng.normal(size=(n, H, P, N)))


def _difference(f, v, g, rng, points=12, h=1e-6, tol=1e-6):
    """df along single elements of v against the gradient g."""
    flat = v.reshape(-1)
    for k in rng.choice(flat.size, min(points, flat.size), replace=False):
        old = flat[k]
        flat[k] = old + h
        up = f()
        flat[k] = old - h
        down = f()
        flat[k] = old
        assert (up - down) / (2 * h) == pytest.approx(g.reshape(-1)[k], rel=tol, abs=tol)


def test_scan_is_the_decode_recurrence():
    rng = np.random.default_rng(1)
    s = _scan(rng)
    y, last = Q.scan_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], STARTS, s["init"])
    pool = s["init"].copy()
    for i, (a, b) in enumerate(Q.spans(STARTS)):
        for t in range(a, b):
            got = M.ssu_standard_step(pool, np.array([i]), s["x"][t:t + 1], s["dt"][t:t + 1], s["A"],
                                      s["B"][t:t + 1], s["C"][t:t + 1], D=s["D"], dt_softplus=False,
                                      state_dtype="f64")
            np.testing.assert_allclose(got[0], y[t], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(pool, last, rtol=1e-12)


def test_scan_gradients_against_differences():
    rng = np.random.default_rng(2)
    s = _scan(rng)
    dy, dlast = rng.normal(size=s["x"].shape), rng.normal(size=s["init"].shape)
    g = Q.scan_backward(dy, **s, starts=STARTS, dlast=dlast)

    def loss():
        y, last = Q.scan_forward(**s, starts=STARTS)
        return (y * dy).sum() + (last * dlast).sum()
    for k in s:
        _difference(loss, s[k], g["d" + k], rng)
    m = Q.scan_backward(dy, **s, starts=STARTS, dlast=dlast, magnitude=True)
    assert all((abs(g[k]) <= m[k] * (1 + 1e-12)).all() for k in g if k != "dD")


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_gradients_against_differences(W, silu):
    rng = np.random.default_rng(3)
    T, C, n = int(STARTS[-1]), 3, len(STARTS) - 1
    x, w, b = rng.normal(size=(T, C)), rng.normal(size=(C, W)), rng.normal(size=C)
    init, dy = rng.normal(size=(n, W - 1, C)), rng.normal(size=(T, C))
    g = Q.conv_backward(dy, x, w, b, STARTS, init, silu)

    def loss():
        return (Q.conv_forward(x, w, b, STARTS, init, silu)[0] * dy).sum()
    for v, k in ((x, "dx"), (w, "dweight"), (b, "dbias"), (init, "dinit")):
        _difference(loss, v, g[k], rng)


def test_conv_steps_are_the_convolution():
    """Token by token with the final states carried equals the whole sequence."""
    rng = np.random.default_rng(4)
    x, w, st = rng.normal(size=(7, 2)), rng.normal(size=(2, 3)), rng.normal(size=(1, 2, 2))
    whole, last, _ = Q.conv_forward(x, w, None, [0, 7], st)
    for t in range(7):
        y, st, _ = Q.conv_forward(x[t:t + 1], w, None, [0, 1], st)
        np.testing.assert_allclose(y[0], whole[t], rtol=1e-13)
    np.testing.assert_array_equal(st, last)


@pytest.mark.parametrize("gate", [True, False])
def test_norm_gradients_against_differences(gate):
    rng = np.random.default_rng(5)
    h, w = rng.normal(size=(3, 12)), rng.normal(size=12)
    z = rng.normal(size=(3, 12)) if gate else None
    dy = rng.normal(size=(3, 12))
    g, m = Q.norm_backward(dy, h, w, z, 4, 1e-3)

    def loss():
        return (Q.norm_forward(h, w, z, 4, 1e-3) * dy).sum()
    for v, k in ((h, "dx"), (w, "dweight")) + (((z, "dz"),) if gate else ()):
        _difference(loss, v, g[k], rng)
        assert (abs(g[k]) <= m[k] * (1 + 1e-12)).all()
