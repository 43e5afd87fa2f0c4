"""Differentiating through a result raises instead of ending without a gradient."""

import pytest
import torch

import linear_recurrence_amd as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _calls():
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, dt, B, C, A = rnd(9, 2, 32), rnd(9, 2), rnd(9, 1, 16), rnd(9, 1, 16), -torch.ones(2, device="cuda")
    rows, w, nw, state = rnd(5, 24), rnd(24, 4), torch.ones(24, device="cuda"), rnd(5, 3, 24)
    return [("ssu_scan_forward", lambda x, A: R.ssu_scan_forward(x, dt, A, B, C), [x, A]),
            ("causal_conv_forward", lambda x, w: R.causal_conv_forward(x, w), [rows, w]),
            ("causal_conv_decode", lambda x, w: R.causal_conv_decode(x, state, w, new_state=state.clone()),
             [rows, w]),
            ("rms_norm_forward", lambda x, w: R.rms_norm_forward(x, w)["out"], [rows, nw]),
            ("rms_norm_forward", lambda x, r: R.rms_norm_forward(x, nw, residual=r)["residual"],
             [rows, rows.flip(0)])]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("leaf", [0, 1])
def test_a_gradient_raises(which, leaf):
    name, call, args = _calls()[which]
    want = call(*args)
    assert not want.requires_grad
    args[leaf] = args[leaf].clone().requires_grad_()
    got = call(*args)
    assert torch.equal(got.detach(), want)
    with pytest.raises(RuntimeError, match=name):
        got.sum().backward()
    with torch.no_grad():
        got = call(*args)
    assert not got.requires_grad and torch.equal(got, want)


def test_inside_a_function_of_the_caller():
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return R.rms_norm_forward(x, w)["out"]

        @staticmethod
        def backward(ctx, dy):
            got = R.rms_norm_backward(dy.contiguous(), *ctx.saved_tensors)
            return got["dx"], got["dweight"]
    x, w = torch.randn(4, 48, device="cuda").requires_grad_(), torch.rand(48, device="cuda").requires_grad_()
    dy = torch.randn(4, 48, device="cuda")
    Norm.apply(x, w).backward(dy)
    with torch.no_grad():
        want = R.rms_norm_backward(dy, x, w)
    assert torch.equal(x.grad, want["dx"]) and torch.equal(w.grad, want["dweight"])
