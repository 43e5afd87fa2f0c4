"""Pins of the linear-attention operators' oracle: against the GDN decode
recurrence, every gradient against central differences, and the rotary turn
against complex numbers."""

import numpy as np
import pytest

from oracle import gdn as G
from oracle import mixer as X
from oracle import sequence as Q

STARTS = np.array([0, 5, 5, 6, 11])
SCALE = 0.4


def _inputs(rng, HK=2, HV=4, K=5, V=3):
    T, n = int(STARTS[-1]), len(STARTS) - 1
    return dict(q=rng.normal(size=(T, HK, K)), k=rng.normal(size=(T, HK, K)) / np.sqrt(K),
                v=rng.normal(size=(T, HV, V)), g=-rng.uniform(0.01, 1.0, (T, HV)),
                beta=rng.uniform(0.0, 1.0, (T, HV)), init=rng.normal(size=(n, HV, V, K)))


def test_delta_rule_is_the_decode_recurrence():
    s = _inputs(np.random.default_rng(1))
    o, last, size = X.mix_forward(**s, starts=STARTS, scale=SCALE)
    pool = s["init"].copy()
    for i, (a, b) in enumerate(Q.spans(STARTS)):
        for t in range(a, b):
            r = slice(t, t + 1)
            want = G.gdn_standard_step(pool, np.array([i]), s["q"][r], s["k"][r], s["v"][r],
                                       np.exp(s["g"][r]), s["beta"][r], scale=SCALE)
            np.testing.assert_allclose(o[t], want[0], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(last, pool, rtol=1e-12, atol=1e-12)
    assert (size >= np.sqrt((last ** 2).sum((2, 3))) - 1e-12).all()


def test_linear_attention_closed_form():
    """o_t = scale sum_{s<=t} e^{G_t - G_s} (q_t.k_s) v_s without initial states."""
    s = _inputs(np.random.default_rng(2))
    s["init"][:] = 0.0
    o, _, _ = X.mix_forward(**{**s, "beta": None}, starts=STARTS, scale=SCALE)
    for a, b in Q.spans(STARTS):
        c = np.cumsum(s["g"][a:b], 0)
        for t in range(b - a):
            for h in range(4):
                w = [np.exp(c[t, h] - c[r, h]) * (s["q"][a + t, h // 2] @ s["k"][a + r, h // 2])
                     for r in range(t + 1)]
                want = SCALE * sum(x * s["v"][a + r, h] for r, x in enumerate(w))
                np.testing.assert_allclose(o[a + t, h], want, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("delta", [True, False])
def test_gradients_are_central_differences(delta):
    rng = np.random.default_rng(3)
    s = _inputs(rng)
    if not delta:
        s["beta"] = None
    do, dlast = rng.normal(size=s["v"].shape), rng.normal(size=s["init"].shape)
    got = X.mix_backward(do, **s, starts=STARTS, scale=SCALE, dlast=dlast)

    def loss():
        o, last, _ = X.mix_forward(**s, starts=STARTS, scale=SCALE)
        return (do * o).sum() + (dlast * last).sum()
    for name in ("q", "k", "v", "g", "init") + (("beta",) if delta else ()):
        flat, grad = s[name].reshape(-1), got["d" + name].reshape(-1)
        for i in rng.choice(flat.size, min(12, flat.size), replace=False):
            old = flat[i]
            flat[i] = old + 1e-6
            up = loss()
            flat[i] = old - 1e-6
            down = loss()
            flat[i] = old
            assert (up - down) / 2e-6 == pytest.approx(grad[i], rel=1e-6, abs=1e-6), name


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_complex_product(interleaved):
    rng = np.random.default_rng(4)
    x, pos, f = rng.normal(size=(5, 2, 10)), np.array([0, 1, 7, 1000, 123456]), np.array([1.0, 0.1, 0.003])
    y = X.rotary(x, pos, f, interleaved, amplitude=1.5)
    at = [(2 * i, 2 * i + 1) if interleaved else (i, i + 3) for i in range(3)]
    for i, (a, b) in enumerate(at):
        z = 1.5 * (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos * f[i])[:, None]
        np.testing.assert_allclose(y[..., a], z.real, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(y[..., b], z.imag, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    np.testing.assert_allclose(X.rotary(y, pos, f, interleaved, 1 / 1.5, inverse=True), x, rtol=1e-12, atol=1e-12)
