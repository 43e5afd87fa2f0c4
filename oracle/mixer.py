"""Operators of linear-attention layers (float64): linear attention with a decay
for each head, the gated delta rule over sequences, rotary positions, with their
gradients.

Test infrastructure only; see the package docstring.  Token by token from the
definitions; sequences are packed along the token axis and given by ``starts``.
``beta`` None is linear attention.  Per value head, S [V, K]:

    S <- e^g S;  d = beta (v - S k)  (linear attention: d = v)
    S <- S + d k^T;  o = scale S q
"""

import numpy as np

from .gdn import key_head
from .sequence import spans


def mix_forward(q, k, v, g, beta, starts, init, scale):
    """q, k [T, HK, K], v [T, HV, V], g (log decay) and beta [T, HV], init
    [n, HV, V, K]; returns o, the final states and ``size`` [n, HV]: the largest
    Frobenius norm that a sequence's state and the terms |d| |k| reach."""
    HV = v.shape[1]
    kh = key_head(HV, k.shape[1])
    o, last = np.zeros(v.shape), np.array(init, np.float64)
    size = np.sqrt((last ** 2).sum((2, 3)))
    for i, (a, b) in enumerate(spans(starts)):
        S = last[i]
        for t in range(a, b):
            kt = k[t][kh]
            S = np.exp(g[t])[:, None, None] * S
            d = v[t]
            if beta is not None:
                pred = np.matmul(S, kt[:, :, None])[:, :, 0]
                size[i] = np.maximum(size[i], np.linalg.norm(pred, axis=1) * np.linalg.norm(kt, axis=1))
                d = beta[t][:, None] * (v[t] - pred)
            S = S + d[:, :, None] * kt[:, None, :]
            o[t] = scale * np.matmul(S, q[t][kh][:, :, None])[:, :, 0]
            for n in (np.sqrt((S ** 2).sum((1, 2))),
                      np.linalg.norm(v[t], axis=1) * np.linalg.norm(kt, axis=1)):
                size[i] = np.maximum(size[i], n)
        last[i] = S
    return o, last, size


def mix_backward(do, q, k, v, g, beta, starts, init, scale, dlast):
    """Gradients of sum(do * o) + sum(dlast * final) with respect to q, k, v, g
    [T, HV], beta and init; ``size`` [n, HV]: the largest norm that dS and the
    terms scale |q| |do| reach."""
    T, HV = v.shape[:2]
    HK = k.shape[1]
    kh = key_head(HV, HK)
    out = dict(dq=np.zeros((T, HV, k.shape[2])), dk=np.zeros((T, HV, k.shape[2])), dv=np.zeros(v.shape),
               dg=np.zeros((T, HV)), dbeta=np.zeros((T, HV)), dinit=np.array(dlast, np.float64))
    size = np.sqrt((out["dinit"] ** 2).sum((2, 3)))
    for i, (a, b) in enumerate(spans(starts)):
        S, seen = np.array(init[i], np.float64), []
        for t in range(a, b):
            kt = k[t][kh]
            S1 = np.exp(g[t])[:, None, None] * S
            e = v[t] if beta is None else v[t] - np.matmul(S1, kt[:, :, None])[:, :, 0]
            d = e if beta is None else beta[t][:, None] * e
            S = S1 + d[:, :, None] * kt[:, None, :]
            seen.append((kt, S1, e, d, S))
        dS = out["dinit"][i]
        for t in reversed(range(a, b)):
            kt, S1, e, d, S2 = seen[t - a]
            qt = q[t][kh]
            size[i] = np.maximum(size[i], scale * np.linalg.norm(qt, axis=1) * np.linalg.norm(do[t], axis=1))
            dS = dS + scale * do[t][:, :, None] * qt[:, None, :]
            size[i] = np.maximum(size[i], np.sqrt((dS ** 2).sum((1, 2))))
            out["dq"][t] = scale * (S2 * do[t][:, :, None]).sum(1)
            dd = (dS * kt[:, None, :]).sum(2)
            dk = (dS * d[:, :, None]).sum(1)
            if beta is not None:
                out["dbeta"][t] = (dd * e).sum(1)
                dd = beta[t][:, None] * dd
                dk = dk - (S1 * dd[:, :, None]).sum(1)
                dS = dS - dd[:, :, None] * kt[:, None, :]
            out["dk"][t], out["dv"][t] = dk, dd
            out["dg"][t] = (dS * S1).sum((1, 2))
            dS = np.exp(g[t])[:, None, None] * dS
        out["dinit"][i] = dS
    for n in ("dq", "dk"):
        out[n] = out[n].reshape(T, HK, HV // HK, k.shape[2]).sum(2)
    out["size"] = size
    return out


def rotary(x, positions, freqs, interleaved=False, amplitude=1.0, inverse=False):
    """x [T, heads, dim] with its first 2 len(freqs) elements turned."""
    y, half = np.array(x, np.float64), len(freqs)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs, np.float64)[None, :]
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    if inverse:
        s = -s
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = np.array(y[..., first]), np.array(y[..., second])
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    return y
