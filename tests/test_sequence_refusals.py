"""What the sequence operators refuse: the C entry points check their
arguments on the host before any HIP call, so this runs without a GPU."""

import ctypes

import pytest
import torch

import linear_recurrence_amd as R
from linear_recurrence_amd import sequence as S

V = ctypes.c_void_p
P = V(0x1000)
OK, EINVAL, EDTYPE, ESHAPE = 0, -1, -2, -4


@pytest.fixture(scope="module")
def lib():
    return R.load()


def _scan(lib, fn="ssu_scan_forward", ws=1 << 40, **over):
    d = dict(tokens=8, seqs=2, nheads=4, headdim=64, dstate=16, ngroups=2, num_slots=2,
             io_dtype=1, state_dtype=0, dt_softplus=1)
    d.update({k: over.pop(k) for k in list(over) if k in [f[0] for f in S.ScanDims._fields_]})
    names = dict(
        ssu_scan_forward="x dt A B C D z dt_bias cu init has slot final y ws".split(),
        ssu_scan_backward=("dy x dt A B C D dt_bias cu init has slot dfinal dx ddt dB dC dA dD "
                           "ddt_bias dinit ws").split())[fn]
    return getattr(lib, fn)(ctypes.byref(S.ScanDims(**d)), *[over.get(n, P) for n in names], ws,
                            None, None)


@pytest.mark.parametrize("fn", ["ssu_scan_forward", "ssu_scan_backward"])
def test_scan_refusals(lib, fn):
    n = 15 if fn == "ssu_scan_forward" else 22
    assert getattr(lib, fn)(None, *([P] * n), 0, None, None) == EINVAL
    for bad, code in ((dict(tokens=-1), EINVAL), (dict(seqs=-1), EINVAL), (dict(nheads=0), EINVAL),
                      (dict(ngroups=3), EINVAL), (dict(ngroups=0), EINVAL),
                      (dict(num_slots=-1), EINVAL), (dict(io_dtype=2), EDTYPE),
                      (dict(state_dtype=7), EDTYPE), (dict(headdim=48), ESHAPE),
                      (dict(headdim=256), ESHAPE), (dict(dstate=24), ESHAPE),
                      (dict(dstate=512), ESHAPE), (dict(seqs=0), EINVAL),
                      (dict(x_stride=255), EINVAL), (dict(x_stride=257), EINVAL),
                      (dict(B_stride=31), EINVAL), (dict(dt_stride=3), EINVAL),
                      (dict(A=None), EINVAL), (dict(x=None), EINVAL), (dict(dt=None), EINVAL),
                      (dict(B=None), EINVAL), (dict(C=None), EINVAL), (dict(cu=None), EINVAL),
                      (dict(x=V(0x1008)), EINVAL), (dict(B=V(0x1002)), EINVAL),
                      (dict(C=V(0x1004)), EINVAL), (dict(init=V(0x1008)), EINVAL)):
        assert _scan(lib, fn, **bad) == code, bad
    assert _scan(lib, tokens=0, seqs=0) == OK       # nothing to do
    assert _scan(lib, "ssu_scan_forward", y=None) == EINVAL
    assert _scan(lib, "ssu_scan_forward", final=V(0x1001)) == EINVAL
    for k in ("dy", "dx", "ddt", "dB", "dC", "dA"):
        assert _scan(lib, "ssu_scan_backward", **{k: None}) == EINVAL
    # a workspace that is too small or missing
    assert _scan(lib, fn, ws=64, tokens=1 << 20) == EINVAL
    assert getattr(lib, fn + "_workspace")(None) == 0


def test_scan_workspace_sizes(lib):
    """Sizes are computed in 64 bits: a long packed batch passes 4 GiB."""
    d = S.ScanDims(1 << 20, 4, 80, 64, 128, 1, 4, 1, 1, 1)
    assert lib.ssu_scan_backward_workspace(ctypes.byref(d)) > 1 << 32
    assert lib.ssu_scan_forward_workspace(ctypes.byref(d)) > 1 << 29
    assert lib.ssu_scan_forward_workspace(ctypes.byref(S.ScanDims(8, 1, 4, 64, 48, 1, 1, 1, 1, 1))) == 0


def _conv(lib, fn="causal_conv_forward", ws=1 << 40, **over):
    d = dict(tokens=8, seqs=2, channels=40, width=4, num_slots=2, io_dtype=1, activation=1)
    d.update({k: over.pop(k) for k in list(over) if k in [f[0] for f in S.ConvDims._fields_]})
    names = dict(causal_conv_forward="x w b cu init has slot final y".split(),
                 causal_conv_backward="dy x w b cu init has slot dx dw db dinit ws".split(),
                 causal_conv_decode="x state w b slot new y".split())[fn]
    tail = ([ws] if "ws" in names else []) + [None, None]
    return getattr(lib, fn)(ctypes.byref(S.ConvDims(**d)), *[over.get(n, P) for n in names], *tail)


@pytest.mark.parametrize("fn", ["causal_conv_forward", "causal_conv_backward", "causal_conv_decode"])
def test_conv_refusals(lib, fn):
    for bad, code in ((dict(tokens=-1), EINVAL), (dict(channels=0), EINVAL),
                      (dict(channels=1 << 30), ESHAPE), (dict(width=1), ESHAPE),
                      (dict(width=5), ESHAPE), (dict(io_dtype=3), EDTYPE),
                      (dict(activation=2), EINVAL), (dict(num_slots=-1), EINVAL),
                      (dict(x_stride=39), EINVAL), (dict(w=None), EINVAL), (dict(x=None), EINVAL),
                      (dict(x=V(0x1001)), EINVAL),
                      (dict(tokens=1 << 30, channels=1 << 16), ESHAPE)):
        assert _conv(lib, fn, **bad) == code, bad
    if fn == "causal_conv_decode":
        assert _conv(lib, fn, tokens=0) == OK
        assert _conv(lib, fn, state=None) == EINVAL
        assert _conv(lib, fn, new=None) == EINVAL
    else:
        assert _conv(lib, fn, cu=None) == EINVAL
        assert _conv(lib, fn, seqs=0) == EINVAL
    if fn == "causal_conv_backward":
        assert _conv(lib, fn, ws=8) == EINVAL
        for k in ("dy", "dx", "dw"):
            assert _conv(lib, fn, **{k: None}) == EINVAL
    if fn == "causal_conv_forward":
        assert _conv(lib, fn, tokens=0, seqs=0) == OK


def _norm(lib, fn="rms_norm_forward", ws=1 << 40, **over):
    d = dict(rows=4, dim=512, group_size=256, io_dtype=1, residual_dtype=1, out_dtype=1,
             scale_block=0, eps=1e-5)
    d.update({k: over.pop(k) for k in list(over) if k in [f[0] for f in S.NormDims._fields_]})
    names = dict(rms_norm_forward="x w z res res_out out scale".split(),
                 rms_norm_backward="dy x w z dx dw dz ws".split())[fn]
    tail = ([ws] if "ws" in names else []) + [None]
    return getattr(lib, fn)(ctypes.byref(S.NormDims(**d)), *[over.get(n, P) for n in names], *tail)


@pytest.mark.parametrize("fn", ["rms_norm_forward", "rms_norm_backward"])
def test_norm_refusals(lib, fn):
    for bad, code in ((dict(rows=-1), EINVAL), (dict(dim=0), EINVAL), (dict(group_size=0), EINVAL),
                      (dict(group_size=200), EINVAL), (dict(eps=-1.0), EINVAL),
                      (dict(eps=float("nan")), EINVAL), (dict(io_dtype=2), EDTYPE),
                      (dict(residual_dtype=2), EDTYPE), (dict(io_dtype=0, residual_dtype=1), EDTYPE),
                      (dict(out_dtype=0), EDTYPE), (dict(x_stride=511), EINVAL),
                      (dict(dim=32776, group_size=32776), ESHAPE),
                      (dict(dim=32768, group_size=4), ESHAPE),   # 8192 vectors of eight
                      (dict(out_dtype=2, scale_block=64), ESHAPE),
                      (dict(out_dtype=2, scale_block=128, dim=192, group_size=96), ESHAPE),
                      (dict(scale_block=128), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL),
                      (dict(x=V(0x1001)), EINVAL), (dict(z=V(0x1001)), EINVAL)):
        assert _norm(lib, fn, **bad) == code, bad
    if fn == "rms_norm_forward":
        assert _norm(lib, rows=0) == OK
        assert _norm(lib, out=None) == EINVAL
        assert _norm(lib, res_out=None) == EINVAL
        assert _norm(lib, out_dtype=2, scale=None) == EINVAL
    else:
        assert _norm(lib, fn, ws=8) == EINVAL
        for k in ("dy", "dx", "dw", "dz"):
            assert _norm(lib, fn, **{k: None}) == EINVAL


def test_the_binding_refuses_tensors_elsewhere():
    x = torch.zeros(4, 2, 64)
    v = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        R.ssu_scan_forward(x, v, torch.zeros(2), torch.zeros(4, 1, 16), torch.zeros(4, 1, 16))
    with pytest.raises(ValueError, match="GPU tensor"):
        R.ssu_scan_backward(x, x, v, torch.zeros(2), torch.zeros(4, 1, 16), torch.zeros(4, 1, 16))
    with pytest.raises(ValueError, match="GPU tensor"):
        R.causal_conv_forward(v, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        R.causal_conv_backward(v, v, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        R.causal_conv_decode(v, torch.zeros(4, 3, 2), torch.zeros(2, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        R.rms_norm_forward(v, torch.zeros(2))
    with pytest.raises(ValueError, match="GPU tensor"):
        R.rms_norm_backward(v, v, torch.zeros(2))
