"""Overlaps and sizes that the sequence operators refuse on the host, before any
HIP call.  Only refused calls are made here: the pointers are made up."""

import ctypes

import pytest
import torch

import linear_recurrence_amd as R
from linear_recurrence_amd import sequence as S

EINVAL, ESHAPE = -1, -4
BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return R.load()


def _conv(lib, x, out, dy=None, x_stride=0, dy_stride=0, tokens=8, channels=40, io=1, **dims):
    d = ctypes.byref(S.ConvDims(tokens, 1, channels, 4, 1, io, 1, 0, x_stride, dy_stride))
    p = ctypes.c_void_p(1 << 40)
    if dy is None:
        return lib.causal_conv_forward(d, x, p, p, p, None, None, None, None, out, None, None)
    return lib.causal_conv_backward(d, dy, x, p, p, p, None, None, None, out, p, p, None, p, 1 << 40,
                                    None, None)


@pytest.mark.parametrize("io, es", [(0, 4), (1, 2)])
def test_conv_refuses_an_output_over_its_input(lib, io, es):
    row, rows = 40 * es, 8 * 40 * es
    for at in (0, es, rows - es, es - rows):               # the same, and any overlap at all
        assert _conv(lib, BASE, BASE + at, io=io) == EINVAL
        assert _conv(lib, BASE, BASE + at, dy=1 << 30, io=io) == EINVAL
        assert _conv(lib, 1 << 30, BASE + at, dy=BASE, io=io) == EINVAL
    # rows of a wide matrix: an output that begins in the last row, or ends in the second
    wide = dict(x_stride=1000, io=io)
    assert _conv(lib, BASE, BASE + 7 * 1000 * es + row - es, **wide) == EINVAL
    assert _conv(lib, BASE, BASE + 1000 * es - rows + es, **wide) == EINVAL


def test_conv_refuses_grids_past_32_bits(lib):
    for tokens, channels in ((1 << 30, 1 << 12), ((1 << 31) - 1, 600), ((1 << 31) - 1, 1 << 24)):
        assert _conv(lib, BASE, BASE, tokens=tokens, channels=channels) == ESHAPE
        assert _conv(lib, BASE, BASE, dy=BASE, tokens=tokens, channels=channels) == ESHAPE
    d, p = S.ConvDims(1 << 28, 1, 1 << 10, 4, 1, 1, 1), ctypes.c_void_p(BASE)
    assert lib.causal_conv_decode(ctypes.byref(d), p, p, p, p, None, p, p, None, None) == ESHAPE


@pytest.mark.parametrize("rows, dim", [(1 << 26, 512), (1 << 24, 1032), (1 << 24, 4096), (1 << 24, 8192),
                                       (1 << 22, 8200), (1 << 22, 32768), ((1 << 31) - 1, 8)])
def test_norm_refuses_grids_past_32_bits(lib, rows, dim):
    """One workgroup a row, of 64, 256 or 1024 threads."""
    p = ctypes.c_void_p(BASE)
    d = ctypes.byref(S.NormDims(rows, dim, dim, 1, 1, 1, 0, 1e-5))
    assert lib.rms_norm_forward(d, p, p, None, None, None, p, None, None) == ESHAPE


def test_the_binding_refuses_sizes_past_32_bits():
    """2^32 + 4 rows would reach the library as 4."""
    S._sizes(torch.empty(2 ** 31 - 1, 0, device="meta"), "x")
    S._sizes(torch.empty((), device="meta"), "x")
    for shape in ((2 ** 31, 1), (2 ** 32 + 4, 1), (1, 2 ** 32 + 8), (3, 2 ** 31, 4)):
        with pytest.raises(ValueError, match="2\\^31 - 1"):
            S._sizes(torch.empty(shape, device="meta"), "x")


def test_launches_go_to_the_tensors_device(monkeypatch):
    """The default stream's handle is 0 on every device: without the device's
    context the launch would go to the current one."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    handle, ctx = S._on(None, torch.device("cuda", 0))
    assert handle == 100 and ctx is S._HERE
    handle, ctx = S._on(None, torch.device("cuda", 1))
    assert handle == 101 and isinstance(ctx, torch.cuda.device) and ctx.idx == 1

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 7
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        S._on(Stream(), torch.device("cuda", 0))
