"""The scan rounds its bf16 results once and nothing before them.

Without D x, which outweighs the recurrence and hides what its operands lose.
The tolerance is that of the convolution and the norm: u |v| for the rounding
of the result (u = 2^-8) and E32 m for an fp32 computation whose terms add up
to m (E32 = 2^-16, derived beside the other operators' tests).  One bf16 factor
in each product would be off by up to u m: with m 3 to 20 times |v|, past it.
"""

import pytest
import torch

import linear_recurrence_amd as R
from oracle import sequence as Q
from test_gpu_sequence import BF16, E32, F32, HALF, Scan, _near, _np

pytestmark = pytest.mark.gpu

SHAPES = [dict(H=4, P=64, N=128, G=1), dict(H=2, P=32, N=16, G=1), dict(H=3, P=128, N=64, G=3),
          dict(H=4, P=64, N=256, G=2), dict(H=2, P=64, N=32, G=1)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "H{H}P{P}N{N}G{G}".format(**s))
@pytest.mark.parametrize("lens", [[100], [150, 70]], ids=["short", "long"])
def test_forward(lens, shape, io):
    s = Scan(lens, io=io, seed=5, **shape)
    a = s.oracle_inputs()
    a["D"] = None
    want, _ = Q.scan_forward(**a)
    mag, _ = Q.scan_magnitude(**a)
    _near(s.forward(D=None), want, HALF[io] * abs(want) + E32 * mag, "y")


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "H{H}P{P}N{N}G{G}".format(**s))
def test_backward(shape, io):
    s = Scan([150, 70], io=io, seed=6, **shape)
    a = s.oracle_inputs()
    a.update(D=None, dlast=_np(s.dlast))
    want = Q.scan_backward(_np(s.dy), **a)
    mag = Q.scan_backward(_np(s.dy), **a, magnitude=True)
    got = s.backward(D=None)
    for k in ("dx", "dB", "dC"):
        _near(got[k], want[k], HALF[io] * abs(want[k]) + E32 * mag[k], k)
