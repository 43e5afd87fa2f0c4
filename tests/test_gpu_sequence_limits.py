"""Outputs beside their inputs in one buffer (near, and sharing nothing), and
inputs whose sizes the library's 32-bit fields cannot hold."""

import pytest
import torch

import linear_recurrence_amd as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def test_conv_output_next_to_its_input():
    T, C = 8, 40
    w = torch.randn(C, 4, device="cuda")
    buf = torch.randn(3 * T * C, device="cuda")
    x = buf[T * C:2 * T * C].view(T, C)
    want = R.causal_conv_forward(x.clone(), w)
    for at in (0, 2 * T * C):
        y = buf[at:at + T * C].view(T, C)
        assert R.causal_conv_forward(x, w, y=y) is y and torch.equal(y, want)
    with pytest.raises(R.RssmError):
        R.causal_conv_forward(x, w, y=x)
    with pytest.raises(R.RssmError):
        R.causal_conv_forward(x, w, y=buf[1:1 + T * C].view(T, C))
    assert torch.equal(R.causal_conv_forward(x, w), want)


def test_conv_output_in_the_gap_of_wide_rows():
    T, C = 8, 40
    w = torch.randn(C, 4, device="cuda")
    buf = torch.randn(T, 1000, device="cuda")
    x, flat = buf[:, :C], buf.view(-1)
    want = R.causal_conv_forward(x.clone(), w)
    for at in (C, 1000 - T * C, 7 * 1000 + C):      # 320 elements where 960 are free
        y = flat[at:at + T * C].view(T, C)
        assert torch.equal(R.causal_conv_forward(x, w, y=y), want)
    with pytest.raises(R.RssmError):
        R.causal_conv_forward(x, w, y=flat[1001 - T * C:1001].view(T, C))


def test_rows_past_32_bits_are_refused():
    x = torch.empty((1 << 32) + 4, 1, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, device="cuda")
    for call in (lambda: R.causal_conv_forward(x, torch.ones(1, 4, device="cuda")),
                 lambda: R.causal_conv_backward(x, x, torch.ones(1, 4, device="cuda")),
                 lambda: R.rms_norm_forward(x, w), lambda: R.rms_norm_backward(x, x, w),
                 lambda: R.rms_norm_forward(x.t(), torch.ones((1 << 32) + 4, device="cuda"))):
        with pytest.raises(ValueError, match="2\\^31 - 1"):
            call()
    with pytest.raises(ValueError, match="group_size"):
        R.rms_norm_forward(x[:4], w, group_size=(1 << 32) + 1)
