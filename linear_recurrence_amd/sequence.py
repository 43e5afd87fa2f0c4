"""Sequence operators of the Mamba2 layer: prefill and training.

The binding of the second half of ``include/replayssm.h``: the selective scan
over packed sequences, the short causal convolution and the root-mean-square
norm, each with its backward pass.  Argument marshalling only, as in the
decode binding.  Operands may be slices of wider rows (one token's row
contiguous, any token stride); what is returned is dense.  Workspaces and
outputs are allocated on the stream the call runs on; a caller whose inputs
live on another stream orders the two, as for any other work.  The operators are
not part of torch's automatic differentiation: their backward passes are calls of
their own, and differentiating through a result raises an error.
"""

import contextlib
import ctypes

import torch

from . import _DT, F32, _check

F8E4M3 = 2
_ACT = {None: 0, "none": 0, "silu": 1}
_IO = (torch.float32, torch.bfloat16)


class ScanDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tokens", "seqs", "nheads", "headdim", "dstate", "ngroups", "num_slots", "io_dtype",
        "state_dtype", "dt_softplus")] + [(n, ctypes.c_int64) for n in (
            "x_stride", "dt_stride", "B_stride", "C_stride", "z_stride", "dy_stride")]


class ConvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tokens", "seqs", "channels", "width", "num_slots", "io_dtype", "activation",
        "reserved")] + [("x_stride", ctypes.c_int64), ("dy_stride", ctypes.c_int64)]


class NormDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "rows", "dim", "group_size", "io_dtype", "residual_dtype", "out_dtype",
        "scale_block")] + [("eps", ctypes.c_float)] + [(n, ctypes.c_int64) for n in (
            "x_stride", "z_stride", "dy_stride")]


_lib = None


def bind(lib):
    """Declare the argument types of this half of the library."""
    global _lib
    P, Z = ctypes.c_void_p, ctypes.c_size_t
    for name, dims, n_ptr, ws in (
            ("ssu_scan_forward", ScanDims, 14, True), ("ssu_scan_backward", ScanDims, 21, True),
            ("causal_conv_forward", ConvDims, 9, False),
            ("causal_conv_backward", ConvDims, 12, True),
            ("causal_conv_decode", ConvDims, 7, False),
            ("rms_norm_forward", NormDims, 7, False), ("rms_norm_backward", NormDims, 7, True)):
        fn = getattr(lib, name)
        head = [ctypes.POINTER(dims)] + [P] * n_ptr
        tail = [] if name.startswith("rms_norm") else [P]  # status
        fn.argtypes = head + ([P, Z] if ws else []) + tail + [P]
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


def _p(t):
    return None if t is None else t.data_ptr()


def _bad(t, name, dtypes, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, dtype, shape, dev):
    """t: a contiguous tensor of this type and shape on dev, or None."""
    if t is not None and not (isinstance(t, torch.Tensor) and t.dtype is dtype and
                              t.shape == shape and t.is_cuda and t.device == dev and
                              t.is_contiguous()):
        _bad(t, name, (dtype,), shape, dev)


def _rows(t, name, dtype, shape, dev):
    """Like _dense, but the first dimension may have any stride; returns it
    (in elements; 0 where there is at most one row)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.is_cuda and t.device == dev):
        _bad(t, name, (dtype,), shape, dev)
    if t.is_contiguous() or shape[0] <= 1 and t[:1].is_contiguous():
        return 0
    if not t[0].is_contiguous() or t.stride(0) < t[0].numel():
        raise ValueError(f"{name}: one token's row must be contiguous, and rows must not overlap")
    return t.stride(0)


def _sizes(t, name):
    """The library's sizes are 32-bit: ctypes would cut a larger one short."""
    n = t.numel()
    if (n > 0x7fffffff or n == 0) and max(t.shape, default=0) > 0x7fffffff:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: sizes are limited to 2^31 - 1")


def _first(t, name, ndim):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {ndim} dimensions")
    if t.dtype not in _DT:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {_IO}")
    _sizes(t, name)
    return t.device, t.dtype


_HERE = contextlib.nullcontext()


def _on(stream, dev):
    """(the stream's handle, a context that allocates on it and launches on its
    device: the default stream's handle is the same on every device)"""
    if stream is None:   # the raw handle: a Stream object costs over a microsecond
        here = torch._C._cuda_getDevice() == dev.index
        return torch._C._cuda_getCurrentRawStream(dev.index), _HERE if here else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _seqs(cu_seqlens, dev):
    if cu_seqlens is None:
        return 1
    n = cu_seqlens.shape[0] - 1 if isinstance(cu_seqlens, torch.Tensor) and \
        cu_seqlens.dim() == 1 else -1
    if n < 0:
        raise ValueError("cu_seqlens must be a 1-D tensor of sequences + 1 entries")
    _sizes(cu_seqlens, "cu_seqlens")
    _dense(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
    return n


def _slots(slot_idx, has_initial, status, n, dev):
    _dense(slot_idx, "slot_idx", torch.int32, (n,), dev)
    _dense(has_initial, "has_initial", torch.uint8, (n,), dev)
    _dense(status, "status", torch.int32, (1,), dev)


class _OwnBackward(torch.autograd.Function):
    """Passes a result on; raises when a gradient comes back to it, which would
    otherwise end there without a word."""

    @staticmethod
    def forward(ctx, name, out, *inputs):
        ctx.name = name
        return out

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} is not differentiable by torch: call its backward pass "
                           "(in an autograd.Function of your own, for instance)")


def _result(name, out, *inputs):
    if torch.is_grad_enabled():
        need = [t for t in inputs if t is not None and t.requires_grad]
        if need:
            return _OwnBackward.apply(name, out, *need)
    return out


# ------------------------------------------------------------------- the scan

def _scan_dims(x, dt, A, B, C, D, dt_bias, cu_seqlens, slot_idx, has_initial, status, dt_softplus):
    dev, io = _first(x, "x", 3)
    T, H, P = x.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be a GPU tensor of 3 dimensions")
    _sizes(B, "B")
    G, N = B.shape[1], B.shape[2]
    n = _seqs(cu_seqlens, dev)
    _dense(A, "A", torch.float32, (H,), dev)
    if A is None:
        raise ValueError("A is required")
    _dense(D, "D", torch.float32, (H,), dev)
    _dense(dt_bias, "dt_bias", torch.float32, (H,), dev)
    _slots(slot_idx, has_initial, status, n, dev)
    d = ScanDims(T, n, H, P, N, G, n, _DT[io], F32, 1 if dt_softplus else 0,
                 _rows(x, "x", io, (T, H, P), dev), _rows(dt, "dt", io, (T, H), dev),
                 _rows(B, "B", io, (T, G, N), dev), _rows(C, "C", io, (T, G, N), dev), 0, 0)
    return dev, io, n, d


def ssu_scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, cu_seqlens=None,
                     initial_state=None, has_initial=None, final_state=None, slot_idx=None,
                     y=None, dt_softplus=True, status=None, stream=None):
    """The selective state update over packed sequences; returns y [T, H, P].

    x, z [T, H, P], dt [T, H], B, C [T, G, N] (io dtype); cu_seqlens int32
    [seqs + 1].  Sequence i starts from initial_state[slot_idx[i]] (a pool
    [slots, H, P, N], as the decode step's; zeros without one or where
    has_initial[i], uint8, is 0) and stores final_state[slot_idx[i]], which
    may be the same pool.  slot_idx None: slot i.
    """
    dev, io, n, d = _scan_dims(x, dt, A, B, C, D, dt_bias, cu_seqlens, slot_idx, has_initial,
                               status, dt_softplus)
    T, H, P = x.shape
    N = B.shape[2]
    pool = initial_state if initial_state is not None else final_state
    if pool is not None:
        if not isinstance(pool, torch.Tensor) or pool.dim() != 4 or pool.dtype not in _DT:
            raise ValueError("states must be float32 or bfloat16 GPU tensors [slots, H, P, N]")
        _sizes(pool, "the state pool")
        shape = (pool.shape[0], H, P, N)
        _dense(initial_state, "initial_state", pool.dtype, shape, dev)
        _dense(final_state, "final_state", pool.dtype, shape, dev)
        d.num_slots, d.state_dtype = pool.shape[0], _DT[pool.dtype]
    if z is not None:
        d.z_stride = _rows(z, "z", io, (T, H, P), dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    size = lib.ssu_scan_forward_workspace(ctypes.byref(d))
    _dense(y, "y", io, (T, H, P), dev)
    with ctx:
        if y is None:
            y = torch.empty((T, H, P), dtype=io, device=dev)
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        _check("ssu_scan_forward", lib.ssu_scan_forward(
            ctypes.byref(d), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z), _p(dt_bias),
            _p(cu_seqlens), _p(initial_state), _p(has_initial), _p(slot_idx), _p(final_state), _p(y),
            _p(ws), size, _p(status), handle))
    return _result("ssu_scan_forward", y, x, dt, A, B, C, D, z, dt_bias, initial_state)


def ssu_scan_backward(dy, x, dt, A, B, C, D=None, dt_bias=None, cu_seqlens=None,
                      initial_state=None, has_initial=None, slot_idx=None, dfinal_state=None,
                      dt_softplus=True, status=None, stream=None):
    """Gradients of ssu_scan_forward (without z); returns a dict of dx, ddt,
    dB, dC (io dtype), dA, dD, ddt_bias (float32) and dinitial_state.

    dfinal_state (or None) and dinitial_state (None without initial_state)
    are float32 [seqs, H, P, N], by sequence and not by slot; the gradient of
    a sequence that started afresh (has_initial 0) is zero.  dD and ddt_bias
    are None where D and dt_bias are.
    """
    dev, io, n, d = _scan_dims(x, dt, A, B, C, D, dt_bias, cu_seqlens, slot_idx, has_initial,
                               status, dt_softplus)
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    d.dy_stride = _rows(dy, "dy", io, (T, H, P), dev)
    if initial_state is not None:
        if not isinstance(initial_state, torch.Tensor) or initial_state.dim() != 4 or \
                initial_state.dtype not in _DT:
            raise ValueError("initial_state must be a float32 or bfloat16 GPU tensor "
                             "[slots, H, P, N]")
        _sizes(initial_state, "initial_state")
        _dense(initial_state, "initial_state", initial_state.dtype,
               (initial_state.shape[0], H, P, N), dev)
        d.num_slots, d.state_dtype = initial_state.shape[0], _DT[initial_state.dtype]
    _dense(dfinal_state, "dfinal_state", torch.float32, (n, H, P, N), dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    size = lib.ssu_scan_backward_workspace(ctypes.byref(d))
    f32 = torch.float32
    with ctx:
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        out = dict(dx=torch.empty((T, H, P), dtype=io, device=dev),
                   ddt=torch.empty((T, H), dtype=io, device=dev),
                   dB=torch.empty((T, G, N), dtype=io, device=dev),
                   dC=torch.empty((T, G, N), dtype=io, device=dev),
                   dA=torch.empty(H, dtype=f32, device=dev),
                   dD=None if D is None else torch.empty(H, dtype=f32, device=dev),
                   ddt_bias=None if dt_bias is None else torch.empty(H, dtype=f32, device=dev),
                   dinitial_state=None if initial_state is None else
                   torch.empty((n, H, P, N), dtype=f32, device=dev))
        _check("ssu_scan_backward", lib.ssu_scan_backward(
            ctypes.byref(d), _p(dy), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias),
            _p(cu_seqlens), _p(initial_state), _p(has_initial), _p(slot_idx), _p(dfinal_state),
            _p(out["dx"]), _p(out["ddt"]), _p(out["dB"]), _p(out["dC"]), _p(out["dA"]),
            _p(out["dD"]), _p(out["ddt_bias"]), _p(out["dinitial_state"]), _p(ws), size, _p(status),
            handle))
    return out


# ------------------------------------------------------- the short convolution

def _conv_dims(x, weight, bias, cu_seqlens, activation, status):
    dev, io = _first(x, "x", 2)
    T, C = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a GPU tensor [channels, width]")
    _sizes(weight, "weight")
    W = weight.shape[1]
    _dense(weight, "weight", torch.float32, (C, W), dev)
    _dense(bias, "bias", torch.float32, (C,), dev)
    _dense(status, "status", torch.int32, (1,), dev)
    if activation not in _ACT:
        raise ValueError("activation must be 'silu' or None")
    n = _seqs(cu_seqlens, dev)
    return dev, io, n, ConvDims(T, n, C, W, n, _DT[io], _ACT[activation], 0,
                                _rows(x, "x", io, (T, C), dev), 0)


def causal_conv_forward(x, weight, bias=None, cu_seqlens=None, initial_state=None,
                        has_initial=None, slot_idx=None, final_state=None, y=None,
                        activation="silu", status=None, stream=None):
    """Depthwise causal convolution over packed sequences; returns y [T, C].

    x [T, C]; weight float32 [C, W], W in 2..4; initial_state / final_state
    [slots, W-1, C] (io dtype, oldest row first; they may be one pool).
    """
    dev, io, n, d = _conv_dims(x, weight, bias, cu_seqlens, activation, status)
    T, C, W = d.tokens, d.channels, d.width
    pool = initial_state if initial_state is not None else final_state
    if pool is not None:
        shape = (pool.shape[0] if isinstance(pool, torch.Tensor) and pool.dim() else 0, W - 1, C)
        _dense(initial_state, "initial_state", io, shape, dev)
        _dense(final_state, "final_state", io, shape, dev)
        _sizes(pool, "the state pool")
        d.num_slots = shape[0]
    _slots(slot_idx, has_initial, None, n, dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    _dense(y, "y", io, (T, C), dev)
    with ctx:
        if y is None:
            y = torch.empty((T, C), dtype=io, device=dev)
        _check("causal_conv_forward", lib.causal_conv_forward(
            ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(cu_seqlens), _p(initial_state),
            _p(has_initial), _p(slot_idx), _p(final_state), _p(y), _p(status), handle))
    return _result("causal_conv_forward", y, x, weight, bias, initial_state)


def causal_conv_backward(dy, x, weight, bias=None, cu_seqlens=None, initial_state=None,
                         has_initial=None, slot_idx=None, activation="silu", status=None,
                         stream=None):
    """Gradients of causal_conv_forward's y; returns a dict of dx, dweight,
    dbias (None without bias) and dinitial_state (None without
    initial_state; by slot, rows of other slots are zero)."""
    dev, io, n, d = _conv_dims(x, weight, bias, cu_seqlens, activation, status)
    T, C, W = d.tokens, d.channels, d.width
    d.dy_stride = _rows(dy, "dy", io, (T, C), dev)
    if initial_state is not None:
        shape = (initial_state.shape[0] if isinstance(initial_state, torch.Tensor) and
                 initial_state.dim() else 0, W - 1, C)
        _dense(initial_state, "initial_state", io, shape, dev)
        _sizes(initial_state, "initial_state")
        d.num_slots = shape[0]
    _slots(slot_idx, has_initial, None, n, dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    size = lib.causal_conv_backward_workspace(ctypes.byref(d))
    with ctx:
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        # every slot is written when the sequences take slots 0..n-1
        alloc = torch.empty if slot_idx is None and d.num_slots == n else torch.zeros
        out = dict(dx=torch.empty((T, C), dtype=io, device=dev),
                   dweight=torch.empty((C, W), dtype=torch.float32, device=dev),
                   dbias=None if bias is None else torch.empty(C, dtype=torch.float32, device=dev),
                   dinitial_state=None if initial_state is None else
                   alloc((d.num_slots, W - 1, C), dtype=io, device=dev))
        _check("causal_conv_backward", lib.causal_conv_backward(
            ctypes.byref(d), _p(dy), _p(x), _p(weight), _p(bias), _p(cu_seqlens), _p(initial_state),
            _p(has_initial), _p(slot_idx), _p(out["dx"]), _p(out["dweight"]), _p(out["dbias"]),
            _p(out["dinitial_state"]), _p(ws), size, _p(status), handle))
    return out


def causal_conv_decode(x, conv_state, weight, bias=None, slot_idx=None, new_state=None, y=None,
                       activation="silu", status=None, stream=None):
    """One decode step of the convolution; returns y [batch, C].

    x [batch, C]; conv_state [slots, W-1, C]; row b uses slot slot_idx[b]
    (None: b).  The moved-on window goes to new_state (None: conv_state
    itself, in place).
    """
    dev, io, _, d = _conv_dims(x, weight, bias, None, activation, status)
    nb, C, W = d.tokens, d.channels, d.width
    if not isinstance(conv_state, torch.Tensor) or conv_state.dim() != 3:
        raise ValueError("conv_state must be a GPU tensor [slots, width - 1, channels]")
    shape = (conv_state.shape[0], W - 1, C)
    if new_state is None:
        new_state = conv_state
    _dense(conv_state, "conv_state", io, shape, dev)
    _dense(new_state, "new_state", io, shape, dev)
    _sizes(conv_state, "conv_state")
    d.num_slots = shape[0]
    _dense(slot_idx, "slot_idx", torch.int32, (nb,), dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    _dense(y, "y", io, (nb, C), dev)
    with ctx:
        if y is None:
            y = torch.empty((nb, C), dtype=io, device=dev)
        _check("causal_conv_decode", lib.causal_conv_decode(
            ctypes.byref(d), _p(x), _p(conv_state), _p(weight), _p(bias), _p(slot_idx),
            _p(new_state), _p(y), _p(status), handle))
    return _result("causal_conv_decode", y, x, conv_state, weight, bias)


# ------------------------------------------------------------------- the norm

def _norm_dims(x, weight, z, group_size, eps):
    dev, io = _first(x, "x", 2)
    R, M = x.shape
    if weight is None:
        raise ValueError("weight is required")
    if group_size is not None and not 1 <= group_size <= max(M, 1):
        raise ValueError(f"group_size is {group_size}, expected a divisor of {M}")
    _dense(weight, "weight", torch.float32, (M,), dev)
    zs = 0 if z is None else _rows(z, "z", io, (R, M), dev)
    return dev, io, NormDims(R, M, M if group_size is None else group_size, _DT[io], _DT[io],
                             _DT[io], 0, eps, _rows(x, "x", io, (R, M), dev), zs, 0)


def rms_norm_forward(x, weight, z=None, residual=None, group_size=None, eps=1e-5, out_dtype=None,
                     scale_block=0, residual_out=None, stream=None):
    """Root-mean-square norm of x (+ residual) (* silu(z)); returns a dict of
    out, scale (8-bit output only) and residual (with residual only).

    x, z [rows, dim]; weight float32 [dim]; residual [rows, dim] float32 or
    x's dtype; out_dtype x's (None) or torch.float8_e4m3fn with one float32
    scale per row (scale_block 0) or per 128 elements (scale_block 128).
    residual_out may be residual (in place); None: a new tensor.
    """
    dev, io, d = _norm_dims(x, weight, z, group_size, eps)
    shape = (d.rows, d.dim)
    fp8 = out_dtype is torch.float8_e4m3fn
    if not fp8 and out_dtype is not None and out_dtype is not io:
        raise ValueError(f"out_dtype must be {io} or torch.float8_e4m3fn")
    if fp8:
        d.out_dtype, d.scale_block = F8E4M3, scale_block
    elif scale_block:
        raise ValueError("scale_block needs an 8-bit output")
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (torch.float32, io):
            raise ValueError(f"residual must be a GPU tensor of torch.float32 or {io}")
        _dense(residual, "residual", residual.dtype, shape, dev)
        _dense(residual_out, "residual_out", residual.dtype, shape, dev)
        d.residual_dtype = _DT[residual.dtype]
    lib, (handle, ctx) = _library(), _on(stream, dev)
    with ctx:
        out = torch.empty(shape, dtype=out_dtype if fp8 else io, device=dev)
        scale = None
        if fp8:
            scale = torch.empty((d.rows, d.dim // 128 if scale_block else 1), dtype=torch.float32,
                                device=dev)
        if residual is not None and residual_out is None:
            residual_out = torch.empty(shape, dtype=residual.dtype, device=dev)
        _check("rms_norm_forward", lib.rms_norm_forward(
            ctypes.byref(d), _p(x), _p(weight), _p(z), _p(residual), _p(residual_out), _p(out),
            _p(scale), handle))
    if fp8:
        scale = _result("rms_norm_forward", scale, x, weight, z, residual)
    else:
        out = _result("rms_norm_forward", out, x, weight, z, residual)
    if residual is not None:
        residual_out = _result("rms_norm_forward", residual_out, x, residual)
    return dict(out=out, scale=scale, residual=residual_out)


def rms_norm_backward(dy, x, weight, z=None, group_size=None, eps=1e-5, stream=None):
    """Gradients of the norm (without residual: its gradient is dx, added by
    the caller to the residual stream's); returns a dict of dx, dweight, dz
    (None without z)."""
    dev, io, d = _norm_dims(x, weight, z, group_size, eps)
    shape = (d.rows, d.dim)
    d.dy_stride = _rows(dy, "dy", io, shape, dev)
    lib, (handle, ctx) = _library(), _on(stream, dev)
    size = lib.rms_norm_backward_workspace(ctypes.byref(d))
    with ctx:
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        out = dict(dx=torch.empty(shape, dtype=io, device=dev),
                   dweight=torch.empty(d.dim, dtype=torch.float32, device=dev),
                   dz=None if z is None else torch.empty(shape, dtype=io, device=dev))
        _check("rms_norm_backward", lib.rms_norm_backward(
            ctypes.byref(d), _p(dy), _p(x), _p(weight), _p(z), _p(out["dx"]), _p(out["dweight"]),
            _p(out["dz"]), _p(ws), size, handle))
    return out
