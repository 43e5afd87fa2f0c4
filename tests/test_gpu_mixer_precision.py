"""The fp32 results of linear attention and the delta rule by their norms.

Every one of them is a sum whose factors are fp32 values or inputs, and is off by
about 2^-23 of its norm: 64 tokens and 64 or 128 columns a chunk, each rounding
2^-25 as a rule and of either sign.  2^-20 leaves eight times that.  A single factor
that entered with two bf16 terms instead of three would be off by 2^-18.3 as a rule
(up to 2^-17), and its results with it: 2^-18 to 2^-18.8 of the final states' norms
in a simulation.  The elementwise bounds beside the other tests do not tell the two
apart.
"""

import numpy as np
import pytest
import torch

import linear_recurrence_amd as R
from oracle import mixer as X
from test_gpu_mixer import BF16, F32, Mix, _np

pytestmark = pytest.mark.gpu

SHAPES = [dict(delta=False, HK=2, HV=4, K=64, V=128, decay="head"), dict(delta=False, HK=3, HV=3, K=128, V=64),
          dict(delta=True, HK=2, HV=4, K=64, V=64), dict(delta=True, HK=2, HV=2, K=128, V=128)]
_ID = lambda s: ("delta" if s["delta"] else "linear") + "K{K}V{V}".format(**s)  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _near(got, want, axes, name, size=None, bound=2.0 ** -20):
    """The norms over these axes of what got is off by."""
    norm = lambda x: np.sqrt((x ** 2).sum(axes))  # noqa: E731
    off, most = norm(_np(got) - want), bound * (norm(want) if size is None else size)
    assert (off <= most).all(), f"{name}: up to {np.nanmax(off / (most + 1e-300)):.3g} times the bound"


def _rows(m, got, want, name, bound=2.0 ** -20):
    """Per token results, by sequence."""
    for i in range(m.n):
        at = slice(m.starts[i], m.starts[i + 1])
        _near(got[at], want[at], None, f"{name} of sequence {i}", bound=bound)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=_ID)
@pytest.mark.parametrize("lens", [[257, 40, 0, 200], [1300, 64]], ids=str)
def test_fp32_results(lens, shape, io):
    m = Mix(lens, io=io, seed=47, **shape)
    o = m.oracle()
    want, last, _ = X.mix_forward(**o)
    final = torch.zeros_like(m.pool)
    got = m.forward(final_state=final)
    _near(final[m.slot.long()], last, (2, 3), "final_state")
    g, w = m.backward(), X.mix_backward(_np(m.do), **o, dlast=_np(m.dlast))
    _near(g["dinitial_state"], w["dinit"] * _np(m.has)[:, None, None, None], (2, 3), "dinitial_state")
    if m.decay == "head":   # a sum of every token's, which may cancel
        _near(g["dlog_decay"], w["dg"].sum(0), (), "dlog_decay", np.abs(w["dg"]).sum(0))
    else:
        _rows(m, g["dlog_g" if m.delta else "dlog_decay"], w["dg"], "dlog")
    if m.delta:
        _rows(m, g["dbeta"], w["dbeta"], "dbeta")
    if io is F32:
        _rows(m, got, want, "o")
        for name in ("dq", "dk", "dv"):
            _rows(m, g[name], w[name], name)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("repeat", [1, 20])
@pytest.mark.parametrize("unit", [True, False], ids=["beta", "keys"])
def test_long_keys_and_large_betas(unit, repeat, K, io):
    """beta |k|^2 between 1 and 2, where a token turns its key's direction of the
    state round and the recurrence still enlarges nothing: beta from 1 to 2 on keys
    of unit norm, or beta = 1 and longer keys; and the same key 20 times in a row.
    A rounding passes the factors beta |k|^2 of a product and of the inverse that it
    goes through, 2 each: four times the bound above.  (In a simulation the results
    are off by 2^-21.2 with repeated keys, 2^-22.6 without.)"""
    m = Mix([200, 700], HK=2, HV=4, K=K, V=K, io=io, seed=53)
    gen = torch.Generator().manual_seed(5)
    size = torch.rand(m.beta.shape, generator=gen).cuda() * 0.98 + 1.0   # 1 to 1.98
    if repeat > 1:
        m.k = m.k[::repeat].repeat_interleave(repeat, 0)[:900].contiguous()
    if unit:
        m.beta = size
    else:
        m.beta[:] = 1.0
        m.k = (m.k.float() * size[:, ::2, None].sqrt()).to(io)
    o = m.oracle()
    k2 = (o["k"] ** 2).sum(2).repeat(2, axis=1) * o["beta"]
    assert 0.9 < k2.min() and k2.max() < 2.0
    want, last, _ = X.mix_forward(**o)
    final, b = torch.zeros_like(m.pool), 2.0 ** -18
    rounded = b + (2.0 ** -8 if io is BF16 else 0.0)
    _rows(m, m.forward(final_state=final), want, "o", rounded)
    _near(final[m.slot.long()], last, (2, 3), "final_state", bound=b)
    g, w = m.backward(), X.mix_backward(_np(m.do), **o, dlast=_np(m.dlast))
    _near(g["dinitial_state"], w["dinit"] * _np(m.has)[:, None, None, None], (2, 3), "dinitial_state", bound=b)
    for name, of, bound in (("dlog_g", "dg", b), ("dbeta", "dbeta", b), ("dq", "dq", rounded), ("dk", "dk", rounded),
                            ("dv", "dv", rounded)):
        _rows(m, g[name], w[of], name, bound)
