"""The gradient of a head's constant decay is a sum over all chunk slots of a call,
those without tokens too; and over none where there is no sequence."""

import pytest
import torch

import linear_recurrence_amd as R
from linear_recurrence_amd import mixer as S
from test_gpu_mixer import BF16, Mix

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


def test_no_sequences():
    """Nothing to sum: zeros, not what the memory held."""
    m = Mix([5], HK=2, HV=32, K=64, V=64, delta=False, decay="head")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    none = torch.empty((0, 32, 64), dtype=BF16, device="cuda")
    qk = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    _soil(32 * 4)
    g = R.linear_attention_backward(none, qk, qk, none, m.g, cu_seqlens=cu)
    assert g["dlog_decay"].shape == (32,) and bool((g["dlog_decay"] == 0).all())
    assert g["dq"].shape == (0, 2, 64) and g["dv"].shape == (0, 32, 64)
    assert R.linear_attention_forward(qk, qk, none, m.g, cu_seqlens=cu).shape == (0, 32, 64)
