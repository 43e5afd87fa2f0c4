"""What the binding of the linear-attention operators refuses at the ends of its
ranges."""

import pytest
import torch

import linear_recurrence_amd as R
from test_gpu_mixer import BF16, F32, Mix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e-46, 1e39, float("inf"), float("nan")])
def test_a_scale_is_a_float32_number(scale):
    """1e-46 is zero in 32 bits, which the library takes for 1/sqrt(dk)."""
    m = Mix([5, 4], delta=False, scale=scale)
    d = Mix([5, 4], delta=True, scale=scale)
    for call in (m.forward, m.backward, d.forward, d.backward,
                 lambda: R.linear_attention_decode(m.pool, None, m.q, m.k, m.v, m.g, scale=scale)):
        with pytest.raises(ValueError, match="scale"):
            call()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("lens", [[70, 3, 128], [1300, 5]], ids=str)
def test_outputs_over_the_values(lens, delta, io):
    """o may be v itself: the same bits as into a tensor of its own."""
    for shape in (dict(HK=2, HV=4, K=64, V=64), dict(HK=1, HV=2, K=128, V=128), dict(HK=16, HV=32, K=128, V=128)):
        m = Mix(lens, delta=delta, io=io, seed=71, **shape)
        want, v = m.forward(), m.v.clone()
        assert m.forward(o=m.v) is m.v and torch.equal(m.v, want)
        if delta:
            continue
        rows = len(m.pool)
        step = [x[:rows].contiguous() for x in (m.q, m.k, v, m.g)]
        want = R.linear_attention_decode(m.pool.clone(), None, *step)
        R.linear_attention_decode(m.pool, None, *step, o=step[2])
        assert torch.equal(step[2], want)
