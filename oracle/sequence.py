"""Sequence operators of the Mamba2 layer (float64): selective scan, short
causal convolution, root-mean-square norm, each with its gradients.

Test infrastructure only; see the package docstring.  Everything is written
token by token from the definitions; sequences are packed along the token
axis and given by their ``starts`` (seqs + 1 entries).  The ``magnitude`` of a
scan is the same recursion over absolute values: the sum of the sizes of the
terms that a result adds up, which is what rounding errors are relative to.
"""

import numpy as np

from .mamba2 import head_groups


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * np.asarray(v, np.float64)))


def spans(starts):
    return [(int(a), int(b)) for a, b in zip(starts[:-1], starts[1:])]


def scan_dt(dt_raw, dt_bias, softplus=True):
    v = dt_raw + (0.0 if dt_bias is None else dt_bias)
    return np.logaddexp(0.0, v) if softplus else v


def scan_forward(x, dt, A, B, C, D, starts, init):
    """x [T, H, P], dt [T, H] (ready), B, C [T, G, N], init [n, H, P, N];
    returns y (without gate) and the final states."""
    H = x.shape[1]
    hg = head_groups(H, B.shape[1])
    y, last = np.zeros(x.shape), np.array(init, np.float64)
    for i, (a, b) in enumerate(spans(starts)):
        S = last[i]
        for t in range(a, b):
            S = np.exp(dt[t] * A)[:, None, None] * S \
                + (dt[t][:, None] * x[t])[:, :, None] * B[t][hg][:, None, :]
            y[t] = np.matmul(S, C[t][hg][:, :, None])[:, :, 0]
        last[i] = S
    return y + (0.0 if D is None else D[None, :, None] * x), last


def scan_magnitude(x, dt, A, B, C, D, starts, init):
    return scan_forward(abs(x), dt, A, abs(B), abs(C), None if D is None else abs(D), starts,
                        abs(init))


def scan_backward(dy, x, dt, A, B, C, D, starts, init, dlast, magnitude=False):
    """Gradients with respect to x, dt (ready), A, B, C, D and init.  With
    ``magnitude`` all inputs are taken by size and A's sign is dropped where
    it multiplies a gradient."""
    if magnitude:
        dy, x, B, C, init, dlast = (abs(v) for v in (dy, x, B, C, init, dlast))
        D = None if D is None else abs(D)
    Am = abs(A) if magnitude else A
    H, G = x.shape[1], B.shape[1]
    hg = head_groups(H, G)
    dx, ddt = np.zeros(x.shape), np.zeros(dt.shape)
    dB, dC, dA = np.zeros(B.shape), np.zeros(C.shape), np.zeros(H)
    dinit = np.array(dlast, np.float64)
    group = (hg[:, None] == np.arange(G)).astype(np.float64)      # [H, G]
    for i, (a, b) in enumerate(spans(starts)):
        before = [np.array(init[i], np.float64)]
        for t in range(a, b):
            before.append(np.exp(dt[t] * A)[:, None, None] * before[-1]
                          + (dt[t][:, None] * x[t])[:, :, None] * B[t][hg][:, None, :])
        L = dinit[i]
        for t in reversed(range(a, b)):
            S = before.pop()
            dC[t] = np.einsum("hn,hg->gn", np.einsum("hp,hpn->hn", dy[t], S), group)
            L = L + dy[t][:, :, None] * C[t][hg][:, None, :]
            Lb = np.einsum("hpn,hn->hp", L, B[t][hg])
            dx[t] = dt[t][:, None] * Lb
            dB[t] = np.einsum("hn,hg->gn", np.einsum("hp,hpn->hn", dt[t][:, None] * x[t], L), group)
            L = np.exp(dt[t] * A)[:, None, None] * L
            da = (L * before[-1]).sum((1, 2))
            ddt[t] = (Lb * x[t]).sum(1) + Am * da
            dA += da * dt[t]
        dinit[i] = L
    if D is not None:
        dx = dx + D[None, :, None] * dy
    return dict(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum((0, 2)), dinit=dinit)


def conv_rows(x, starts, init, i):
    """Rows of sequence i behind the W - 1 rows before it."""
    a, b = spans(starts)[i]
    return np.concatenate([init[i], x[a:b]])


def conv_forward(x, w, bias, starts, init, silu=True):
    """x [T, C], w [C, W], init [n, W-1, C]; returns y, final [n, W-1, C] and
    v (before the activation)."""
    W = w.shape[1]
    v, last = np.zeros(x.shape), np.zeros(init.shape)
    for i, (a, b) in enumerate(spans(starts)):
        r = conv_rows(x, starts, init, i)
        for j in range(W):
            v[a:b] += w[:, j] * r[j:j + b - a]
        last[i] = r[b - a:]
    v = v + (0.0 if bias is None else bias)
    return (v * sigmoid(v) if silu else v), last, v


def conv_backward(dy, x, w, bias, starts, init, silu=True, magnitude=False):
    W = w.shape[1]
    v = conv_forward(x, w, bias, starts, init, silu)[2]
    s = sigmoid(v)
    dv = dy * (s * (1.0 + v * (1.0 - s)) if silu else 1.0)
    if magnitude:   # dv itself is a sum, dy s + dy s v (1 - s), and may cancel
        dv = abs(dy) * (s * (1.0 + abs(v) * (1.0 - s)) if silu else 1.0)
        x, w, init = abs(x), abs(w), abs(init)
    dx, dw, dinit = np.zeros(x.shape), np.zeros(w.shape), np.zeros(init.shape)
    for i, (a, b) in enumerate(spans(starts)):
        r = conv_rows(x, starts, init, i)
        dr = np.zeros(r.shape)
        for j in range(W):
            dw[:, j] += (dv[a:b] * r[j:j + b - a]).sum(0)
            dr[j:j + b - a] += dv[a:b] * w[:, j]
        dx[a:b], dinit[i] = dr[W - 1:], dr[:W - 1]
    return dict(dx=dx, dweight=dw, dbias=dv.sum(0), dinit=dinit)


def norm_forward(h, weight, z, group, eps):
    u = h if z is None else h * z * sigmoid(z)
    v = u.reshape(u.shape[0], -1, group)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return (v * r).reshape(u.shape) * weight


def norm_backward(dy, h, weight, z, group, eps):
    """Gradients and the size of the terms that each adds up."""
    s = None if z is None else sigmoid(z)
    gate = 1.0 if z is None else z * s
    u = h * gate
    shape = (u.shape[0], -1, group)
    v, t = u.reshape(shape), (dy * weight).reshape(shape)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    du = (r * (t - v * r * r * (t * v).mean(-1, keepdims=True))).reshape(u.shape)
    size = (r * (abs(t) + abs(v) * r * r * abs(t * v).mean(-1, keepdims=True))).reshape(u.shape)
    one = dy * (v * r).reshape(u.shape)
    out = dict(dx=du * gate, dweight=one.sum(0))
    mag = dict(dx=size * abs(gate), dweight=abs(one).sum(0))
    if z is not None:
        d = s * (1.0 + z * (1.0 - s))
        out["dz"], mag["dz"] = du * h * d, size * abs(h * d)
    return out, mag
