"""Operators of linear-attention layers: linear attention with a decay for each
head, the gated delta rule over sequences, rotary positions.

The binding of the third part of ``include/replayssm.h``, by the conventions of
the sequence operators (``sequence.py``): packed sequences, operands that may be
slices of wider rows, dense results, workspaces on the calling stream, backward
passes as calls of their own.  The states are the pools of the GDN decode step:
float32 [slots, v_heads, dv, dk].
"""

import ctypes
import math

import torch

from . import _DT, _check
from .sequence import _dense, _first, _on, _p, _result, _rows, _seqs, _sizes, _slots

_NONE, _HEAD, _TOKEN = 0, 1, 2


class MixerDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tokens", "seqs", "k_heads", "v_heads", "dk", "dv", "num_slots", "io_dtype", "decay")] + [
            ("scale", ctypes.c_float)] + [(n, ctypes.c_int64) for n in (
                "q_stride", "k_stride", "v_stride", "do_stride")]


class RotaryDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tokens", "heads", "dim", "rotary_dim", "io_dtype", "interleaved", "pos_int64")] + [
            ("amplitude", ctypes.c_float)] + [("x_stride", ctypes.c_int64),
                                              ("y_stride", ctypes.c_int64)]


_lib = None


def bind(lib):
    """Declare the argument types of this part of the library."""
    global _lib
    P, Z = ctypes.c_void_p, ctypes.c_size_t
    for name, dims, n_ptr, ws in (
            ("linear_attention_forward", MixerDims, 11, True),
            ("linear_attention_backward", MixerDims, 16, True),
            ("linear_attention_decode", MixerDims, 8, False),
            ("gdn_scan_forward", MixerDims, 12, True), ("gdn_scan_backward", MixerDims, 18, True),
            ("rotary_forward", RotaryDims, 4, False), ("rotary_backward", RotaryDims, 4, False)):
        fn = getattr(lib, name)
        tail = [] if name.startswith("rotary") else [P]  # status
        fn.argtypes = [ctypes.POINTER(dims)] + [P] * n_ptr + ([Z] if ws else []) + tail + [P]
        fn.restype = ctypes.c_int
        if ws:
            w = getattr(lib, name + "_workspace")
            w.argtypes, w.restype = [ctypes.POINTER(dims)], Z
    _lib = lib


def _library():
    if _lib is None:
        from . import load
        load()
    return _lib


def _heads(q, k, v, decay, beta, scale, delta):
    """(device, io type, tokens, dims) of one call's q, k, v and gates."""
    dev, io = _first(q, "q", 3)
    T, HK, K = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("v must be a GPU tensor of 3 dimensions")
    _sizes(v, "v")
    HV, V = v.shape[1], v.shape[2]
    d = MixerDims(T, 1, HK, HV, K, V, 0, _DT[io], _NONE, 0.0 if scale is None else scale)
    if scale is not None and not 0 < d.scale < math.inf:   # as the library gets it, in 32 bits
        raise ValueError(f"scale is {scale}, expected a positive float32 number (None: 1/sqrt(dk))")
    d.q_stride = _rows(q, "q", io, (T, HK, K), dev)
    d.k_stride = _rows(k, "k", io, (T, HK, K), dev)
    d.v_stride = _rows(v, "v", io, (T, HV, V), dev)
    name = "log_g" if delta else "log_decay"
    if delta or (isinstance(decay, torch.Tensor) and decay.dim() == 2):
        if decay is None:
            raise ValueError(f"{name} is required")
        _dense(decay, name, torch.float32, (T, HV), dev)
        d.decay = _TOKEN
    elif decay is not None:
        _dense(decay, name, torch.float32, (HV,), dev)
        d.decay = _HEAD
    if delta:
        if beta is None:
            raise ValueError("beta is required")
        _dense(beta, "beta", torch.float32, (T, HV), dev)
    return dev, io, T, d


def _pools(d, dev, *named):
    """Checks state pools [slots, HV, V, K] that are one size, and notes it."""
    slots = None
    for name, pool in named:
        if pool is None:
            continue
        if not isinstance(pool, torch.Tensor) or pool.dim() != 4:
            raise ValueError(f"{name} must be a float32 GPU tensor [slots, v_heads, dv, dk]")
        _sizes(pool, name)
        slots = d.num_slots = pool.shape[0] if slots is None else slots
        _dense(pool, name, torch.float32, (d.num_slots, d.v_heads, d.dv, d.dk), dev)


def _forward(delta, q, k, v, decay, beta, scale, cu_seqlens, initial_state, has_initial, final_state,
             slot_idx, o, status, stream):
    name = "gdn_scan_forward" if delta else "linear_attention_forward"
    dev, io, T, d = _heads(q, k, v, decay, beta, scale, delta)
    d.seqs = n = _seqs(cu_seqlens, dev)
    _slots(slot_idx, has_initial, status, n, dev)
    _pools(d, dev, ("initial_state", initial_state), ("final_state", final_state))
    lib, (handle, ctx) = _library(), _on(stream, dev)
    size = getattr(lib, name + "_workspace")(ctypes.byref(d))
    shape = (T, d.v_heads, d.dv)
    _dense(o, "o", io, shape, dev)
    with ctx:
        if o is None:
            o = torch.empty(shape, dtype=io, device=dev)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        _check(name, getattr(lib, name)(
            ctypes.byref(d), _p(q), _p(k), _p(v), _p(decay), *([_p(beta)] if delta else []), _p(cu_seqlens),
            _p(initial_state), _p(has_initial), _p(slot_idx), _p(final_state), _p(o), _p(ws), size, _p(status),
            handle))
    return _result(name, o, q, k, v, decay, beta, initial_state)


def _backward(delta, do, q, k, v, decay, beta, scale, cu_seqlens, initial_state, has_initial, slot_idx,
              dfinal_state, status, stream):
    name = "gdn_scan_backward" if delta else "linear_attention_backward"
    dev, io, T, d = _heads(q, k, v, decay, beta, scale, delta)
    d.do_stride = _rows(do, "do", io, tuple(v.shape), dev)
    d.seqs = n = _seqs(cu_seqlens, dev)
    _slots(slot_idx, has_initial, status, n, dev)
    _pools(d, dev, ("initial_state", initial_state))
    states = (n, d.v_heads, d.dv, d.dk)
    _dense(dfinal_state, "dfinal_state", torch.float32, states, dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    size = getattr(lib, name + "_workspace")(ctypes.byref(d))
    f32 = torch.float32
    with ctx:
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        out = dict(dq=torch.empty(q.shape, dtype=io, device=dev),
                   dk=torch.empty(q.shape, dtype=io, device=dev),
                   dv=torch.empty(v.shape, dtype=io, device=dev))
        dg = None if decay is None else torch.empty(decay.shape, dtype=f32, device=dev)
        out["dlog_g" if delta else "dlog_decay"] = dg
        if delta:
            out["dbeta"] = torch.empty(beta.shape, dtype=f32, device=dev)
        out["dinitial_state"] = None if initial_state is None else torch.empty(states, dtype=f32, device=dev)
        _check(name, getattr(lib, name)(
            ctypes.byref(d), _p(do), _p(q), _p(k), _p(v), _p(decay), *([_p(beta)] if delta else []),
            _p(cu_seqlens), _p(initial_state), _p(has_initial), _p(slot_idx), _p(dfinal_state),
            _p(out["dq"]), _p(out["dk"]), _p(out["dv"]), _p(dg), *([_p(out["dbeta"])] if delta else []),
            _p(out["dinitial_state"]), _p(ws), size, _p(status), handle))
    return out


def linear_attention_forward(q, k, v, log_decay=None, cu_seqlens=None, initial_state=None,
                             has_initial=None, final_state=None, slot_idx=None, scale=None, o=None,
                             status=None, stream=None):
    """S = e^log_decay S + v k^T, o = scale S q, token by token; returns o [T, HV, V].

    q, k [T, HK, K], v [T, HV, V] (io dtype; K and V 64 or 128, HV a multiple of
    HK); log_decay float32 [HV] (constant), [T, HV] or None (no decay);
    cu_seqlens int32 [seqs + 1].  Sequence i starts from
    initial_state[slot_idx[i]] (float32 [slots, HV, V, K]; zeros without one or
    where has_initial[i], uint8, is 0) and stores final_state[slot_idx[i]],
    which may be the same pool.  o shares no memory with q, k or
    v, unless it is v.  scale None: 1/sqrt(K).
    """
    return _forward(False, q, k, v, log_decay, None, scale, cu_seqlens, initial_state, has_initial,
                    final_state, slot_idx, o, status, stream)


def linear_attention_backward(do, q, k, v, log_decay=None, cu_seqlens=None, initial_state=None,
                              has_initial=None, slot_idx=None, dfinal_state=None, scale=None,
                              status=None, stream=None):
    """Gradients of linear_attention_forward; returns a dict of dq, dk, dv (io
    dtype), dlog_decay (float32, log_decay's shape; None without) and
    dinitial_state.

    dfinal_state (or None) and dinitial_state (None without initial_state) are
    float32 [seqs, HV, V, K], by sequence and not by slot; the gradient of a
    sequence that started afresh (has_initial 0) is zero.
    """
    return _backward(False, do, q, k, v, log_decay, None, scale, cu_seqlens, initial_state,
                     has_initial, slot_idx, dfinal_state, status, stream)


def linear_attention_decode(state, slot_idx, q, k, v, log_decay=None, scale=None, new_state=None,
                            o=None, status=None, stream=None):
    """One token of every row; returns o [batch, HV, V].

    q, k [batch, HK, K], v [batch, HV, V]; state float32 [slots, HV, V, K], row b
    uses slot slot_idx[b] (None: b); the moved-on state goes to new_state (None:
    state itself, in place).  log_decay [HV], [batch, HV] or None.
    """
    dev, io, nb, d = _heads(q, k, v, log_decay, None, scale, False)
    if new_state is None:
        new_state = state
    if state is None:
        raise ValueError("state is required")
    _pools(d, dev, ("state", state), ("new_state", new_state))
    _dense(slot_idx, "slot_idx", torch.int32, (nb,), dev)
    _dense(status, "status", torch.int32, (1,), dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    shape = (nb, d.v_heads, d.dv)
    _dense(o, "o", io, shape, dev)
    with ctx:
        if o is None:
            o = torch.empty(shape, dtype=io, device=dev)
        _check("linear_attention_decode", lib.linear_attention_decode(
            ctypes.byref(d), _p(state), _p(slot_idx), _p(q), _p(k), _p(v), _p(log_decay), _p(new_state),
            _p(o), _p(status), handle))
    return _result("linear_attention_decode", o, q, k, v, log_decay, state)


def gdn_scan_forward(q, k, v, log_g, beta, cu_seqlens=None, initial_state=None, has_initial=None,
                     final_state=None, slot_idx=None, scale=None, o=None, status=None, stream=None):
    """The gated delta rule over packed sequences; returns o [T, HV, V].

    The recurrence of gdn_standard_decode with g = exp(log_g): log_g, beta
    float32 [T, HV]; dk == dv, 64 or 128; the other arguments as
    linear_attention_forward's.  The pools are the GDN decode step's.
    """
    return _forward(True, q, k, v, log_g, beta, scale, cu_seqlens, initial_state, has_initial,
                    final_state, slot_idx, o, status, stream)


def gdn_scan_backward(do, q, k, v, log_g, beta, cu_seqlens=None, initial_state=None, has_initial=None,
                      slot_idx=None, dfinal_state=None, scale=None, status=None, stream=None):
    """Gradients of gdn_scan_forward; returns a dict of dq, dk, dv (io dtype),
    dlog_g, dbeta (float32 [T, HV]) and dinitial_state, with dfinal_state and
    dinitial_state as linear_attention_backward's."""
    return _backward(True, do, q, k, v, log_g, beta, scale, cu_seqlens, initial_state, has_initial,
                     slot_idx, dfinal_state, status, stream)


# ------------------------------------------------------------------- positions

def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=None,
                       low=1.0, high=4.0, beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freqs, amplitude) for rotary_forward: float32 [rotary_dim / 2] on
    ``device``, and a float.

    Plain frequencies are base^(-2i / rotary_dim).  ``scaling`` stretches a
    context of original_length tokens by ``factor``:
      "linear"  every frequency divided by factor (position interpolation)
      "ntk"     base times factor^(rotary_dim / (rotary_dim - 2)), so that the
                lowest frequency alone is divided by factor
      "bands"   by how often pair i turns in original_length tokens: divided by
                factor below ``low`` turns, kept above ``high``, and linear in
                the turns between
      "yarn"    the same with a ramp over the pair's index between beta_slow and
                beta_fast turns; amplitude 0.1 ln(factor) + 1
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim is {rotary_dim}, expected an even number")
    if not factor >= 1.0:
        raise ValueError(f"factor is {factor}, expected at least 1")
    half, amplitude = rotary_dim // 2, 1.0
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError("scaling 'ntk' needs a rotary_dim above 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freqs = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    elif scaling in ("bands", "yarn"):
        if not original_length:
            raise ValueError(f"scaling '{scaling}' needs original_length")
        if scaling == "bands":
            if not low < high:
                raise ValueError("low must be below high")
            keep = [(original_length * f / (2 * math.pi) - low) / (high - low) for f in freqs]
        else:
            # the (fractional) index of the pair that turns n times
            def index(n):
                return rotary_dim * math.log(original_length / (n * 2 * math.pi)) / (2 * math.log(base))
            first, last = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rotary_dim - 1)
            keep = [1.0 - (i - first) / max(last - first, 1e-3) for i in range(half)]
            amplitude = 0.1 * math.log(factor) + 1.0
        keep = [min(max(w, 0.0), 1.0) for w in keep]
        freqs = [f * w + f / factor * (1.0 - w) for f, w in zip(freqs, keep)]
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk', 'bands' or 'yarn'")
    return torch.tensor(freqs, dtype=torch.float32, device=device), amplitude


def _rotary(name, x, positions, freqs, interleaved, amplitude, out, stream):
    dev, io = _first(x, "x", 3)
    T, H, D = x.shape
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a float32 GPU tensor [rotary_dim / 2]")
    _dense(freqs, "freqs", torch.float32, tuple(freqs.shape), dev)
    if not 1 <= freqs.shape[0] <= D // 2:
        raise ValueError(f"freqs has {freqs.shape[0]} entries, expected 1 to {D // 2}")
    wide = isinstance(positions, torch.Tensor) and positions.dtype is torch.int64
    if positions is None:
        raise ValueError("positions is required")
    _dense(positions, "positions", torch.int64 if wide else torch.int32, (T,), dev)
    d = RotaryDims(T, H, D, 2 * freqs.shape[0], _DT[io], 1 if interleaved else 0, 1 if wide else 0, amplitude,
                   _rows(x, "x", io, (T, H, D), dev), 0)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    if out is not None:
        d.y_stride = _rows(out, "out", io, (T, H, D), dev)
    with ctx:
        if out is None:
            out = torch.empty((T, H, D), dtype=io, device=dev)
        _check(name, getattr(lib, name)(ctypes.byref(d), _p(x), _p(positions), _p(freqs), _p(out), handle))
    return out


def rotary_forward(x, positions, freqs, interleaved=False, amplitude=1.0, out=None, stream=None):
    """Turns pairs of each head's first 2 * len(freqs) elements by positions *
    freqs; returns out [T, heads, dim].

    x [T, heads, dim] (io dtype; a slice of wider rows, q and k heads together
    for instance); positions int32 or int64 [T]; freqs float32, from
    rotary_frequencies (with its amplitude) or anywhere else.  Pairs are (2i,
    2i + 1) where interleaved, else (i, i + len(freqs)).  out may be x (in
    place) or any tensor of its shape that shares no memory with it.
    """
    return _result("rotary_forward",
                   _rotary("rotary_forward", x, positions, freqs, interleaved, amplitude, out, stream),
                   x, freqs)


def rotary_backward(dy, positions, freqs, interleaved=False, amplitude=1.0, out=None, stream=None):
    """The gradient of rotary_forward's x: the turn back of dy; out may be dy."""
    return _rotary("rotary_backward", dy, positions, freqs, interleaved, amplitude, out, stream)
