"""Linear attention and the delta rule round their bf16 results once, from sums that
carry what fp32 can hold.

An fp32 computation of these sizes is off by about 2^-23 of a result's norm (64
tokens and 64 or 128 columns a chunk, each rounding 2^-25 as a rule and of either
sign); 2^-20 leaves eight times that.  A factor cut to two bf16 terms is off by up
to 2^-17 of itself, 2^-18.3 as a rule, and so is what it is a factor of.

A bf16 result then differs from the 64-bit one, rounded, only where that lies so
close to the middle of two bf16 numbers.  Their distance is 2^-7.5 of an element as
a rule, so that an error of e times the norm shifts e 2^7.5 r of them, with r = 1.3
the mean of norm over size of the elements of at least a quarter of the root mean
square: fewer than 2^-12 of them for e = 2^-20, more than 2^-11.3 for 2^-18.5 (a
simulation with each of the factors cut to two terms gives 2^-10.2 to 2^-11.3,
without 2^-14.5).
"""

import numpy as np
import pytest
import torch

import linear_recurrence_amd as R
from oracle import mixer as X
from test_gpu_mixer import BF16, Mix, _np

pytestmark = pytest.mark.gpu

SHAPES = [dict(delta=False, HK=4, HV=4, K=64, V=128), dict(delta=False, HK=4, HV=4, K=128, V=128),
          dict(delta=True, HK=4, HV=4, K=64, V=64), dict(delta=True, HK=4, HV=4, K=128, V=128)]
_ID = lambda s: ("delta" if s["delta"] else "linear") + "K{K}V{V}".format(**s)  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _rounded_once(got, want, name):
    assert got.dtype is BF16 and tuple(got.shape) == want.shape
    rounded = torch.from_numpy(want).to(BF16).double().numpy()
    big = np.abs(want) >= np.sqrt((want ** 2).mean((0, 2), keepdims=True)) / 4   # by head
    off = ((_np(got) != rounded) & big).sum()
    assert big.sum() > 2 ** 16 and off <= big.sum() * 2.0 ** -12, f"{name}: {off} of {big.sum()}"


@pytest.mark.parametrize("shape", SHAPES, ids=_ID)
def test_bf16_results(shape):
    """Several chunks, and (700 tokens) two segments."""
    m = Mix([130, 700], seed=43, **shape)
    o = m.oracle()
    want, _, _ = X.mix_forward(**o)
    _rounded_once(m.forward(), want, "o")
    got, w = m.backward(), X.mix_backward(_np(m.do), **o, dlast=_np(m.dlast))
    for name in ("dq", "dk", "dv"):
        _rounded_once(got[name], w[name], name)
