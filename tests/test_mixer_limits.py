"""What the linear-attention operators refuse, and what they do not, at the ends of
their ranges: on the host, before any HIP call."""

import pytest

import linear_recurrence_amd as R
from test_mixer_refusals import EINVAL, OK, _mix


@pytest.fixture(scope="module")
def lib():
    return R.load()


def test_a_heads_decay_always_has_a_gradient(lib):
    """Its shape has no token in it: it is written for an empty batch too."""
    for seqs in (0, 2):
        assert _mix(lib, "linear_attention_backward", decay=1, tokens=0, seqs=seqs, gg=None) == EINVAL
    assert _mix(lib, "linear_attention_backward", decay=2, tokens=0, seqs=0, gg=None) == OK
