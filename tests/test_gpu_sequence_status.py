"""Malformed sequence tables are reported by every operator that takes one.

The kernels clamp what they read, so a bad table gives unspecified results and
no address out of range; the status word is how a caller learns of it.
"""

import pytest
import torch

import linear_recurrence_amd as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _table(*entries):
    return torch.tensor(entries, dtype=torch.int32, device="cuda")


def _word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("table, tokens", [((0, 9, 4), 4), ((0, 3, 2), 4), ((1, 2, 4), 4), ((0, -1, 4), 4),
                                           ((0, 300, 100, 500), 500), ((0, 1), 0)], ids=str)
def test_conv_backward_reports_a_bad_table(table, tokens, initial):
    x, w = torch.randn(tokens, 16, device="cuda"), torch.randn(16, 4, device="cuda")
    n, status = len(table) - 1, _word()
    init = torch.zeros(n, 3, 16, device="cuda") if initial else None
    R.causal_conv_backward(x, x, w, cu_seqlens=_table(*table), initial_state=init, status=status)
    assert int(status) == R.ST_BAD_SEQ
    status.zero_()
    good = [0] * n + [tokens]
    R.causal_conv_backward(x, x, w, cu_seqlens=_table(*good), initial_state=init, status=status)
    assert int(status) == 0


@pytest.mark.parametrize("table", [(0, 1000, 200, 2000), (1000, 200, 2000), (0, 2000, 100, 150, 2000),
                                   (0, 1999, 3, 2000), (0, 700, 1400, 2001)], ids=str)
def test_scan_reports_a_bad_table(table):
    """Entries that a search for a token's sequence passes over, too."""
    g = torch.Generator().manual_seed(0)
    T, H, P, N = 2000, 2, 32, 16
    x, dy = (torch.randn(T, H, P, generator=g).cuda() for _ in range(2))
    dt, B, C = (torch.randn(T, *s, generator=g).cuda() for s in ((H,), (1, N), (1, N)))
    A, status = -torch.ones(H, device="cuda"), _word()
    R.ssu_scan_forward(x, dt, A, B, C, cu_seqlens=_table(*table), status=status)
    assert int(status) == R.ST_BAD_SEQ
    status.zero_()
    R.ssu_scan_backward(dy, x, dt, A, B, C, cu_seqlens=_table(*table), status=status)
    assert int(status) == R.ST_BAD_SEQ
    status.zero_()
    good = _table(0, 0, 1000, 1000, T)
    R.ssu_scan_forward(x, dt, A, B, C, cu_seqlens=good, status=status)
    R.ssu_scan_backward(dy, x, dt, A, B, C, cu_seqlens=good, status=status)
    assert int(status) == 0
