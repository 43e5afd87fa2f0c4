"""The gradient of a head's constant decay is a sum over all chunk slots of a call,
those without tokens too."""

import pytest
import torch

import linear_recurrence_amd as R
from linear_recurrence_amd import mixer as S
from test_gpu_mixer import Mix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _soil(*sizes):
    """Leaves NaN in the memory that the next allocations of these sizes take."""
    kept = [torch.full((-(-n // 4),), float("nan"), device="cuda") for n in sizes for _ in range(8)]
    torch.cuda.synchronize()
    del kept


@pytest.mark.parametrize("lens, K, HV", [([64, 64], 64, 320), ([3, 0], 64, 257), ([3, 0], 128, 520)], ids=str)
def test_more_value_heads_on_a_key_head_than_threads(lens, K, HV):
    """Two sequences of 64 tokens have four slots, two of them empty; an empty
    sequence has one."""
    m = Mix(lens, HK=1, HV=HV, K=K, V=64, delta=False, decay="head", seed=41)
    d = S.MixerDims(sum(lens), len(lens), 1, HV, K, 64, m.slots, 1, 1, 0.0)
    _soil(R.load().linear_attention_backward_workspace(d))
    m.check_backward(m.backward())
