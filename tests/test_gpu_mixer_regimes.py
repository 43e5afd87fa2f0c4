"""Linear attention and the delta rule where the host's rules and the sequence table
take other ways than in the small tests: segments longer than the shortest, and
batches of more sequences than a wave has lanes."""

import math

import numpy as np
import pytest
import torch

import linear_recurrence_amd as R
from oracle import mixer as X
from test_gpu_mixer import BF16, F32, Mix, _near, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _definition(m):
    """Output, final states and gradients token by token in 64 bits, on the GPU."""
    r, T = m.HV // m.HK, len(m.q)
    q, k = (t.double().repeat_interleave(r, 1) for t in (m.q, m.k))
    v, do, scale = m.v.double(), m.do.double(), 1.0 / math.sqrt(m.K)
    g = torch.exp(m.g.double()).expand(T, m.HV)[:, :, None, None]
    beta = m.beta.double()[:, :, None] if m.delta else None
    o, last = torch.zeros_like(v), torch.empty(m.n, m.HV, m.V, m.K, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = (torch.zeros(T, m.HV, dtype=torch.float64, device="cuda") for _ in range(2))
    dinit = m.dlast.double().clone()
    for i in range(m.n):
        S, seen = m.pool[m.slot[i].long()].double() * float(m.has[i]), []
        at = range(int(m.starts[i]), int(m.starts[i + 1]))
        for t in at:
            S1 = S * g[t]
            e = v[t] - (S1 * k[t][:, None, :]).sum(2) if m.delta else v[t]
            d = beta[t] * e if m.delta else e
            S = S1 + d[:, :, None] * k[t][:, None, :]
            o[t] = scale * (S * q[t][:, None, :]).sum(2)
            seen.append((S1, e, d, S))
        last[i] = S
        dS = dinit[i]
        for t in reversed(at):
            S1, e, d, S2 = seen.pop()
            dS = dS + scale * do[t][:, :, None] * q[t][:, None, :]
            dq[t] = scale * (S2 * do[t][:, :, None]).sum(1)
            dd, dk[t] = (dS * k[t][:, None, :]).sum(2), (dS * d[:, :, None]).sum(1)
            if m.delta:
                db[t] = (dd * e).sum(1)
                dd = beta[t] * dd
                dk[t] -= (S1 * dd[:, :, None]).sum(1)
                dS = dS - dd[:, :, None] * k[t][:, None, :]
            dv[t], dg[t] = dd, (dS * S1).sum((1, 2))
            dS = dS * g[t]
        dinit[i] = dS * float(m.has[i])
    share = lambda x: x.unflatten(1, (m.HK, r)).sum(2)  # noqa: E731
    out = dict(o=o, final=last[:], dq=share(dq), dk=share(dk), dv=dv, dinitial_state=dinit)
    out["dlog_g" if m.delta else "dlog_decay"] = dg
    if m.delta:
        out["dbeta"] = db
    return out


@pytest.mark.parametrize("delta", [False, True])
def test_longer_segments(delta):
    """5101 tokens of 64 columns a token and head: segments of ten chunks instead of
    eight, in sequences of six, one and two of them.  By norms: fp32 results 2^-20,
    as in the tests of precision; bf16 ones their rounding, up to 2^-8 of each element."""
    shape = dict(HK=32, HV=64, K=64, V=64) if delta else dict(HK=32, HV=32, K=64, V=128)
    m = Mix([3300, 1, 1100, 0, 700], delta=delta, seed=59, **shape)
    final = torch.zeros_like(m.pool)
    got = dict(o=m.forward(final_state=final), **m.backward())
    got["final"] = final[m.slot.long()]
    for name, want in _definition(m).items():
        bound = 2.0 ** -20 + (2.0 ** -8 if got[name].dtype is BF16 else 0.0)
        of = [slice(None)] if len(want) == m.n else [slice(a, b) for a, b in zip(m.starts[:-1], m.starts[1:])]
        for at in of:
            off = float((got[name][at].double() - want[at]).norm())
            assert off <= bound * float(want[at].norm()), (name, at, off / float(want[at].norm()))


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", [dict(delta=False, HK=2, HV=4, K=64, V=128, decay="head"),
                                   dict(delta=True, HK=2, HV=4, K=64, V=64)],
                         ids=lambda s: "delta" if s["delta"] else "linear")
def test_many_sequences(shape, io):
    """75 short, empty and one-token sequences around three of several segments; the
    final states over the initial ones."""
    lens = [(7 * i) % 23 for i in range(30)] + [700] + [1] * 20 + [1200, 0, 513] + [(5 * i) % 9 for i in range(24)] + [0]
    m = Mix(lens, io=io, seed=61, **shape)
    pool = m.pool.clone()
    m.check_forward(m.forward(initial_state=pool, final_state=pool), pool)
    m.check_backward(m.backward())


def test_many_sequences_the_same_bits():
    """Two calls at once, and a captured pass replayed with other lengths."""
    m = Mix([3] * 40 + [600] + [2] * 30 + [1100, 5], HK=2, HV=4, K=64, V=64, seed=67)

    def both(stream=None):
        final = torch.zeros_like(m.pool)
        o = m.forward(final_state=final, stream=stream)
        g = m.backward(stream=stream)
        return [o, final] + [t for t in g.values() if t is not None]
    want, side = both(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    here = both()
    with torch.cuda.stream(side):
        there = both(stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, here, there):
        assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    starts = torch.tensor([0] + [1] * 20 + [900] * 20 + [901 + 2 * i for i in range(30)] + [1500, 1885, 1885],
                          dtype=torch.int32)
    for cu in (m.cu.cpu(), starts, m.cu.cpu()):
        assert len(cu) == len(m.cu) and int(cu[-1]) == len(m.q)
        m.cu.copy_(cu)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(both(), kept):
            assert torch.equal(a, b)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("T", [300, 16500])
def test_a_batch_of_16500_sequences(T, delta):
    """Of one token or none, from zeros: o = scale beta (q.k) v.  With 32 heads of 128
    the launches hold fewer than 2^32 threads, and those of segments, which such a
    batch has none of, do not count."""
    n, HK, HV, K = 16500, 16, 32, 128
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(T, h, K, generator=gen, device="cuda").to(BF16) for h in (HK, HK, HV))
    g, beta = -torch.rand(T, HV, generator=gen, device="cuda"), torch.rand(T, HV, generator=gen, device="cuda")
    cu = torch.arange(n + 1, device="cuda").clamp(max=T).to(torch.int32)
    if delta:
        o = R.gdn_scan_forward(q, k, v, g, beta, cu_seqlens=cu)
    else:
        o, beta = R.linear_attention_forward(q, k, v, g, cu_seqlens=cu), torch.ones_like(beta)
    qk = (q.double() * k.double()).sum(2).repeat_interleave(2, 1)
    want = (beta.double() * qk / math.sqrt(K))[:, :, None] * v.double()
    # 128 products, each and their sums off by 2^-24 of |q| |k|, and the bf16 result
    size = (q.double().norm(dim=2) * k.double().norm(dim=2)).repeat_interleave(2, 1) / math.sqrt(K)
    assert ((o.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * size[:, :, None] * v.double().abs()).all()


def test_rotary_of_the_most_tokens():
    """2^31 - 1 of them, one head of one pair: in place, a few against the oracle."""
    T = 2 ** 31 - 1
    x = torch.full((T, 1, 2), 0.5, dtype=BF16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = torch.tensor([0.37], device="cuda")
    R.rotary_forward(x, pos, f, out=x)
    at = torch.tensor([0, 1, 255, 256, 2 ** 24 + 3, 2 ** 30, T - 257, T - 1], device="cuda")
    want = X.rotary(np.full((len(at), 1, 2), 0.5), _np(pos[at]), _np(f))
    # the angle, up to 2^30, is off by 2^-53 of itself a step: 2^-20 covers it
    _near(x[at], want, 2.0 ** -8 * abs(want) + 2.0 ** -20, "turned")
