"""What the binding of the linear-attention operators refuses at the ends of its
ranges."""

import pytest

import linear_recurrence_amd as R
from test_gpu_mixer import Mix

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
