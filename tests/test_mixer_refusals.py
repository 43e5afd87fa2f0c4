"""What the linear-attention operators refuse: the C entry points check their
arguments on the host before any HIP call, so this runs without a GPU.  And the
host-side frequencies of the rotary positions."""

import ctypes
import math

import pytest
import torch

import linear_recurrence_amd as R
from linear_recurrence_amd import mixer as S

V = ctypes.c_void_p
P = V(0x1000)
OK, EINVAL, EDTYPE, ESHAPE = 0, -1, -2, -4
BIG = 1 << 45

NAMES = dict(
    linear_attention_forward="q k v g cu init has slot final o ws",
    linear_attention_backward="do q k v g cu init has slot dfinal gq gk gv gg dinit ws",
    linear_attention_decode="state slot q k v g new o",
    gdn_scan_forward="q k v g beta cu init has slot final o ws",
    gdn_scan_backward="do q k v g beta cu init has slot dfinal gq gk gv gg gbeta dinit ws")
SEQ = [n for n in NAMES if n != "linear_attention_decode"]


@pytest.fixture(scope="module")
def lib():
    return R.load()


def _mix(lib, fn, ws=BIG, **over):
    d = dict(tokens=8, seqs=2, k_heads=2, v_heads=4, dk=64, dv=64, num_slots=2, io_dtype=1, decay=2, scale=0.5)
    d.update({k: over.pop(k) for k in list(over) if k in [f[0] for f in S.MixerDims._fields_]})
    names = NAMES[fn].split()
    tail = ([ws] if "ws" in names else []) + [None, None]
    over = {dict(wsp="ws").get(k, k): v for k, v in over.items()}
    return getattr(lib, fn)(ctypes.byref(S.MixerDims(**d)), *[over.get(n, P) for n in names], *tail)


@pytest.mark.parametrize("fn", list(NAMES))
def test_mixer_refusals(lib, fn):
    names = NAMES[fn].split()
    tail = ([0] if "ws" in names else []) + [None, None]
    assert getattr(lib, fn)(None, *([P] * len(names)), *tail) == EINVAL
    for bad, code in ((dict(tokens=-1), EINVAL), (dict(k_heads=0), EINVAL), (dict(v_heads=0), EINVAL),
                      (dict(v_heads=3), EINVAL), (dict(num_slots=-1), EINVAL), (dict(io_dtype=2), EDTYPE),
                      (dict(io_dtype=-1), EDTYPE), (dict(decay=3), EINVAL), (dict(decay=-1), EINVAL),
                      (dict(dk=32), ESHAPE), (dict(dk=256), ESHAPE), (dict(dv=96), ESHAPE), (dict(dv=0), ESHAPE),
                      (dict(scale=float("nan")), EINVAL), (dict(q_stride=127), EINVAL),
                      (dict(k_stride=129), EINVAL), (dict(v_stride=255), EINVAL), (dict(v_stride=260), EINVAL),
                      (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL),
                      (dict(g=None), EINVAL)):
        assert _mix(lib, fn, **bad) == code, bad
    for n in {"o", "beta", "do", "gq", "gk", "gv", "gg", "gbeta", "state", "new"} & set(names):
        assert _mix(lib, fn, **{n: None}) == EINVAL, n
    for n in {"init", "final", "o", "do", "gq", "gk", "gv", "dfinal", "dinit", "state", "new"} & set(names):
        if fn == "linear_attention_decode" and n == "o":
            continue
        assert _mix(lib, fn, **{n: V(0x1004)}) == EINVAL, n
    if fn.startswith("gdn"):
        assert _mix(lib, fn, dv=128) == ESHAPE   # its states are square
        assert _mix(lib, fn, dk=128) == ESHAPE
    if fn == "linear_attention_decode":
        assert _mix(lib, fn, tokens=0) == OK
        assert _mix(lib, fn, tokens=(1 << 31) - 1) == ESHAPE
    else:
        assert _mix(lib, fn, seqs=-1) == EINVAL
        assert _mix(lib, fn, seqs=0) == EINVAL
        assert _mix(lib, fn, cu=None) == EINVAL
        assert _mix(lib, fn, tokens=0, seqs=0) == OK
        assert _mix(lib, fn, seqs=1 << 24) == ESHAPE   # 2^32 threads and more
    if "ws" in names:
        long = dict(tokens=1 << 15)
        assert _mix(lib, fn, ws=64, **long) == EINVAL
        assert _mix(lib, fn, wsp=None, **long) == EINVAL
        assert _mix(lib, fn, wsp=V(0x1008)) == EINVAL
        assert getattr(lib, fn + "_workspace")(None) == 0


def test_mixer_workspace_sizes(lib):
    """Sizes are computed in 64 bits: a long packed batch passes 4 GiB."""
    d = S.MixerDims(1 << 20, 4, 16, 32, 128, 128, 4, 1, 2, 0.0)
    for fn in ("gdn_scan_backward", "linear_attention_backward", "gdn_scan_forward"):
        assert getattr(lib, fn + "_workspace")(ctypes.byref(d)) > 1 << 32
    # one segment needs none; a longer call the segments' states
    assert lib.linear_attention_forward_workspace(ctypes.byref(S.MixerDims(64, 1, 4, 4, 64, 64, 1, 1, 2))) == 0
    assert lib.linear_attention_forward_workspace(ctypes.byref(d)) > 1 << 22
    assert lib.gdn_scan_forward_workspace(ctypes.byref(S.MixerDims(8, 1, 4, 4, 48, 48, 1, 1, 2))) == 0
    assert lib.gdn_scan_forward_workspace(ctypes.byref(S.MixerDims(0, 3, 4, 4, 64, 64, 1, 1, 2))) == 0


def _rot(lib, fn, x=P, pos=P, f=P, y=V(0x100000), **over):
    d = dict(tokens=8, heads=4, dim=64, rotary_dim=64, io_dtype=1, interleaved=0, pos_int64=1, amplitude=1.0,
             x_stride=0, y_stride=0)
    d.update(over)
    return getattr(lib, fn)(ctypes.byref(S.RotaryDims(**d)), x, pos, f, y, None)


@pytest.mark.parametrize("fn", ["rotary_forward", "rotary_backward"])
def test_rotary_refusals(lib, fn):
    assert getattr(lib, fn)(None, P, P, P, P, None) == EINVAL
    for bad, code in ((dict(tokens=-1), EINVAL), (dict(heads=0), EINVAL), (dict(dim=1), EINVAL),
                      (dict(rotary_dim=0), EINVAL), (dict(rotary_dim=7), EINVAL), (dict(rotary_dim=66), EINVAL),
                      (dict(io_dtype=3), EDTYPE), (dict(dim=1026), ESHAPE), (dict(x_stride=255), EINVAL),
                      (dict(y_stride=255), EINVAL), (dict(x=None), EINVAL), (dict(pos=None), EINVAL),
                      (dict(f=None), EINVAL), (dict(y=None), EINVAL), (dict(x=V(0x1001)), EINVAL),
                      (dict(pos=V(0x1004)), EINVAL),
                      # outputs over inputs, unless they are the same rows
                      (dict(y=V(0x1002)), EINVAL), (dict(y=V(0x1000 + 8 * 512 - 2)), EINVAL),
                      (dict(y=P, x_stride=512), EINVAL), (dict(y=V(0x11fe), x_stride=512, y_stride=512), EINVAL),
                      (dict(y=V(0x1202), x_stride=512, y_stride=512), EINVAL),
                      (dict(tokens=(1 << 31) - 1, heads=64, y=V(1 << 50)), ESHAPE)):
        assert _rot(lib, fn, **bad) == code, bad
    # two slices of the same rows are refused for their size alone
    wide = dict(tokens=(1 << 31) - 1, heads=64, x_stride=8192, y_stride=8192, y=V(0x1000 + 8192))
    assert _rot(lib, fn, **wide) == ESHAPE
    assert _rot(lib, fn, tokens=0, x=None, y=None) == OK


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(4, 2, 64)
    for fn in (lambda: R.linear_attention_forward(x, x, x), lambda: R.linear_attention_backward(x, x, x, x),
               lambda: R.linear_attention_decode(None, None, x, x, x),
               lambda: R.gdn_scan_forward(x, x, x, x[..., 0], x[..., 0]),
               lambda: R.gdn_scan_backward(x, x, x, x, x[..., 0], x[..., 0]),
               lambda: R.rotary_forward(x, torch.arange(4), torch.ones(4)),
               lambda: R.rotary_backward(x, torch.arange(4), torch.ones(4))):
        with pytest.raises(ValueError, match="GPU tensor"):
            fn()


def test_rotary_frequencies():
    f, amp = R.rotary_frequencies(8, base=10000.0, device="cpu")
    assert amp == 1.0 and f.dtype is torch.float32
    torch.testing.assert_close(f, torch.tensor([1.0, 0.1, 0.01, 0.001]))
    f, _ = R.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")
    torch.testing.assert_close(f, torch.tensor([0.25, 0.025, 0.0025, 0.00025]))
    f, _ = R.rotary_frequencies(8, scaling="ntk", factor=4.0, device="cpu")   # the ends: kept, and divided
    assert float(f[0]) == 1.0 and float(f[3]) == pytest.approx(0.001 / 4, rel=1e-6)
    plain = R.rotary_frequencies(128, device="cpu")[0].double()
    turns = 4096 * plain / (2 * math.pi)
    f = R.rotary_frequencies(128, scaling="bands", factor=8.0, original_length=4096, device="cpu")[0].double()
    assert torch.allclose(f[turns > 4], plain[turns > 4], rtol=1e-6)
    assert torch.allclose(f[turns < 1], plain[turns < 1] / 8, rtol=1e-6)
    mid = (turns > 1) & (turns < 4)
    w = (turns[mid] - 1) / 3
    assert mid.any() and torch.allclose(f[mid], plain[mid] * w + plain[mid] / 8 * (1 - w), rtol=1e-6)
    f, amp = R.rotary_frequencies(128, scaling="yarn", factor=8.0, original_length=4096, device="cpu")
    assert amp == pytest.approx(0.1 * math.log(8.0) + 1.0)
    ratio = f.double() / plain
    assert (ratio[turns > 33] > 1 - 1e-6).all() and torch.allclose(ratio[turns < 0.9], torch.tensor(0.125).double())
    assert (ratio.diff() <= 1e-9).all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="yarn"),
                dict(rotary_dim=2, scaling="ntk"), dict(rotary_dim=8, scaling="bands", original_length=64, low=4.0)):
        with pytest.raises(ValueError):
            R.rotary_frequencies(**bad, device="cpu")


@pytest.mark.parametrize("fn", ["gdn_scan_forward", "gdn_scan_backward"])
@pytest.mark.parametrize("decay", [0, 1])
def test_the_delta_rule_has_a_gate_for_every_token(lib, fn, decay):
    """With another kind of decay the gradient of beta was left unwritten."""
    assert _mix(lib, fn, decay=decay) == EINVAL
    d = S.MixerDims(tokens=8, seqs=2, k_heads=2, v_heads=4, dk=64, dv=64, num_slots=2, io_dtype=1, decay=decay,
                    scale=0.5)
    assert getattr(lib, fn + "_workspace")(ctypes.byref(d)) == 0
