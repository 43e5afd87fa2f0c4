"""Linear attention, the gated delta rule over sequences and rotary positions on
the GPU against the 64-bit oracle.

Tolerances are element by element, with u = 2^-8 (bf16's half step; 0 for fp32
results) for a result's own rounding and E32 = 2^-16 times the size of what it is
made of.  That size is taken from the norms that the oracle's states reach (M of
S, |v||k| and |S k||k|; N of the gradient dS and scale |q||do|): with keys of unit
norm and beta <= 1 neither recurrence amplifies an error, so a chunk's 64 + K terms,
each off by at most 2^-24 of these norms, and its few fp32 factors (exp2 2^-22) stay
below 2^8 of 2^-24 whatever their signs, and the chunks before it add theirs as
roundings of either sign:
  o    scale |q| M;  final state  M
  dq   scale |do| M;  dv  N |k|;  dk  N D + N |k| M with D = |v| + M |k| (d's size)
  dbeta  N |k| (|v| + M);  dg  8 times N (D |k| + M): sums of up to 64 tokens'
  dinitial_state  N
A bf16 result adds u times itself and, where a fp32 factor enters its product as two
bf16 terms, 2^-16 of the same sizes (E32 again).
"""

import math

import numpy as np
import pytest
import torch

import linear_recurrence_amd as R
from oracle import mixer as X

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -16
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(got, want, tol, name):
    got = _np(got)
    assert got.shape == want.shape, name
    off = np.abs(got - want)
    bad = ~(off <= np.broadcast_to(tol, off.shape) + 1e-30)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, off by up to " \
        f"{np.nanmax(off[bad] / (np.broadcast_to(tol, off.shape)[bad] + 1e-30)):.3g} tolerances"


class Mix:
    """Inputs of one call; q, k, v and do are slices of wider rows (`wide`) or
    tensors of their own."""

    def __init__(self, lens, HK=2, HV=4, K=64, V=64, delta=True, io=BF16, decay="token", initial=True,
                 wide=False, seed=0, scale=None):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        T, n = sum(lens), len(lens)
        self.lens, self.io, self.n, self.delta, self.decay = lens, io, n, delta, decay
        self.HK, self.HV, self.K, self.V = HK, HV, K, V
        self.starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
        # a little below unit norm: rounded to bf16 they must not exceed it
        parts = [(0.99 * unit(rnd(T, HK, K))).to(io), (0.99 * unit(rnd(T, HK, K))).to(io),
                 rnd(T, HV, V).to(io), rnd(T, HV, V).to(io)]
        if wide:
            pad = torch.full((T, 8), float("nan"), dtype=io)
            row = torch.cat([pad] + [p for x in parts for p in (x.flatten(1), pad)], 1).cuda()
            at, views = 8, []
            for x in parts:
                size = x.shape[1] * x.shape[2]
                views.append(row[:, at:at + size].unflatten(1, x.shape[1:]))
                at += size + 8
            self.q, self.k, self.v, self.do = views
        else:
            self.q, self.k, self.v, self.do = (x.cuda() for x in parts)
        rate = torch.exp(torch.rand(HV, generator=g) * 5.0 - 5.0)   # slow and fast heads
        self.g = {"token": -rate * torch.rand(T, HV, generator=g) * 2, "head": -rate, "none": None}[decay]
        self.g = None if self.g is None else self.g.cuda()
        self.beta = torch.rand(T, HV, generator=g).cuda()
        self.slots = n + 3
        self.pool = (rnd(self.slots, HV, V, K) * 0.1).cuda()
        self.slot = torch.randperm(self.slots, generator=g)[:n].to(torch.int32).cuda()
        self.has = torch.tensor([i % 3 != 2 for i in range(n)], dtype=torch.uint8).cuda()
        self.initial, self.scale = initial, scale
        self.dlast = (rnd(n, HV, V, K) * 0.1).cuda()
        self.cu = torch.tensor(self.starts, dtype=torch.int32).cuda()

    def args(self, **over):
        a = dict(cu_seqlens=self.cu, slot_idx=self.slot, initial_state=self.pool if self.initial else None,
                 has_initial=self.has if self.initial else None, scale=self.scale)
        a.update(over)
        return a

    def forward(self, **over):
        if self.delta:
            return R.gdn_scan_forward(self.q, self.k, self.v, self.g, self.beta, **self.args(**over))
        return R.linear_attention_forward(self.q, self.k, self.v, self.g, **self.args(**over))

    def backward(self, **over):
        a = self.args(dfinal_state=self.dlast)
        a.update(over)
        if self.delta:
            return R.gdn_scan_backward(self.do, self.q, self.k, self.v, self.g, self.beta, **a)
        return R.linear_attention_backward(self.do, self.q, self.k, self.v, self.g, **a)

    def oracle(self):
        T = int(self.starts[-1])
        init = np.zeros((self.n, self.HV, self.V, self.K))
        if self.initial:
            init = _np(self.pool[self.slot.long()]) * _np(self.has)[:, None, None, None]
        g = np.zeros(self.HV) if self.g is None else _np(self.g)
        return dict(q=_np(self.q), k=_np(self.k), v=_np(self.v), g=np.broadcast_to(g, (T, self.HV)),
                    beta=_np(self.beta) if self.delta else None, starts=self.starts, init=init,
                    scale=self.scale or 1.0 / math.sqrt(self.K))

    def sizes(self, o, size):
        """Per token and value head: |q|, |k|, |v|, |do| and the sequence's M."""
        r = self.HV // self.HK
        norm = lambda x: np.linalg.norm(x, axis=2)  # noqa: E731
        q, k = (np.repeat(norm(o[x]), r, 1) for x in ("q", "k"))
        return q, k, norm(o["v"]), norm(_np(self.do)), np.repeat(size, self.lens, 0)

    def check_forward(self, got, final):
        o = self.oracle()
        want, last, size = X.mix_forward(**o)
        q, _, _, _, M = self.sizes(o, size)
        u = HALF[self.io]
        _near(got, want, u * abs(want) + E32 * (o["scale"] * q * M)[:, :, None], "o")
        if final is not None:
            _near(final[self.slot.long()], last, E32 * size[:, :, None, None], "final")

    def check_backward(self, got, dlast=True):
        o = self.oracle()
        dl = _np(self.dlast) if dlast else np.zeros(o["init"].shape)
        w = X.mix_backward(_np(self.do), **o, dlast=dl)
        _, _, size = X.mix_forward(**o)
        q, k, v, do, M = self.sizes(o, size)
        N = np.repeat(w["size"], self.lens, 0)
        u, D = HALF[self.io], v + (M * k if self.delta else 0.0)
        share = lambda x: x.reshape(x.shape[0], self.HK, self.HV // self.HK).sum(2)[:, :, None]  # noqa: E731
        _near(got["dq"], w["dq"], u * abs(w["dq"]) + E32 * share(o["scale"] * do * M), "dq")
        _near(got["dk"], w["dk"], u * abs(w["dk"]) + E32 * share(N * D + (N * k * M if self.delta else 0.0)), "dk")
        _near(got["dv"], w["dv"], u * abs(w["dv"]) + E32 * (N * k)[:, :, None], "dv")
        tg = 8 * E32 * N * (D * k + M)
        if self.delta:
            _near(got["dbeta"], w["dbeta"], E32 * N * k * (v + M), "dbeta")
            _near(got["dlog_g"], w["dg"], tg, "dlog_g")
        elif self.decay == "token":
            _near(got["dlog_decay"], w["dg"], tg, "dlog_decay")
        elif self.decay == "head":
            _near(got["dlog_decay"], w["dg"].sum(0), tg.sum(0), "dlog_decay")
        else:
            assert got["dlog_decay"] is None
        if self.initial:
            _near(got["dinitial_state"], w["dinit"] * _np(self.has)[:, None, None, None],
                  E32 * w["size"][:, :, None, None], "dinitial_state")
        else:
            assert got["dinitial_state"] is None


LENS = [[1], [0], [3, 0, 1, 63, 64, 65, 0], [130], [257, 1, 0, 200]]
LINEAR = [dict(HK=2, HV=4, K=64, V=128, decay="head"), dict(HK=3, HV=3, K=128, V=64, decay="token"),
          dict(HK=1, HV=5, K=128, V=128, decay="none"), dict(HK=1, HV=1, K=64, V=64, decay="token")]
DELTA = [dict(HK=2, HV=4, K=64, V=64), dict(HK=3, HV=3, K=128, V=128), dict(HK=1, HV=5, K=128, V=128),
         dict(HK=9, HV=9, K=64, V=64)]
_ID = "HK{HK}HV{HV}K{K}V{V}".format


def _both(lens, shape, delta, io):
    m = Mix(lens, delta=delta, io=io, wide=lens == [130], seed=len(lens), **shape)
    final = torch.full_like(m.pool, 7.0)
    o = m.forward(final_state=final)
    m.check_forward(o, final)
    other = torch.ones(m.slots, dtype=torch.bool)
    other[m.slot.cpu().long()] = False
    assert (final[other.cuda()] == 7.0).all()          # no other slot is written
    m.check_backward(m.backward())


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", LINEAR, ids=lambda s: _ID(**s))
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_linear_attention(lens, shape, io):
    _both(lens, shape, False, io)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", DELTA, ids=lambda s: _ID(**s))
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_delta_rule(lens, shape, io):
    _both(lens, shape, True, io)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", [dict(delta=False, **LINEAR[0]), dict(delta=False, **LINEAR[1]),
                                   dict(delta=True, **DELTA[0]), dict(delta=True, **DELTA[1])],
                         ids=lambda s: ("delta" if s["delta"] else "linear") + _ID(**s))
@pytest.mark.parametrize("lens", [[1300], [513, 2, 0, 1025, 512]], ids=str)
def test_segments(lens, shape, io):
    """Sequences of more than 512 tokens are worked on in segments; the pool that they
    start from may be the one that they store to."""
    m = Mix(lens, io=io, seed=23, **shape)
    pool = m.pool.clone()
    m.check_forward(m.forward(initial_state=pool, final_state=pool), pool)
    m.check_backward(m.backward())


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("io", [F32, BF16])
def test_bare(io, delta):
    """No table, slots or states; a scale of the caller's."""
    m = Mix([100], delta=delta, io=io, initial=False, scale=0.25)
    bare = dict(cu_seqlens=None, slot_idx=None)
    m.check_forward(m.forward(**bare), None)
    m.check_backward(m.backward(dfinal_state=None, **bare), dlast=False)


@pytest.mark.parametrize("delta", [False, True])
def test_no_tokens(delta):
    """Empty sequences pass their states through, and their gradients back."""
    m = Mix([0, 0, 0, 0], delta=delta, decay="token" if delta else "head")
    final = torch.full_like(m.pool, 7.0)
    assert m.forward(final_state=final).shape == (0, 4, 64)
    has = m.has[:, None, None, None].float()
    assert torch.equal(final[m.slot.long()], m.pool[m.slot.long()] * has)
    g = m.backward()
    assert torch.equal(g["dinitial_state"], m.dlast * has)
    if not delta:
        assert (g["dlog_decay"] == 0).all()


@pytest.mark.parametrize("delta", [False, True])
def test_in_place_and_continued(delta):
    """The final states over the initial ones; and 200 tokens in two calls are the
    200 in one."""
    m = Mix([200, 90], HK=2, HV=2, K=128, V=128, delta=delta, seed=3)
    pool = m.pool.clone()
    final = torch.empty_like(pool)
    o = m.forward(final_state=final)
    o2 = m.forward(initial_state=pool, final_state=pool)
    at = m.slot.long()
    assert torch.equal(o, o2) and torch.equal(final[at], pool[at])
    fn = R.gdn_scan_forward if delta else R.linear_attention_forward
    state, parts = m.pool.clone(), []
    for a, b in ((0, 128), (128, 200)):   # the first sequence: its chunks are the same
        gates = [m.g[a:b], m.beta[a:b]] if delta else [m.g[a:b]]
        parts.append(fn(m.q[a:b], m.k[a:b], m.v[a:b], *gates, initial_state=state, final_state=state,
                        slot_idx=m.slot[:1]))
    a = m.oracle()
    want, last, size = X.mix_forward(**a)
    tol = HALF[m.io] * abs(want[:200]) + E32 * (a["scale"] * size[0])[None, :, None]
    _near(torch.cat(parts), want[:200], tol, "continued")
    _near(state[m.slot[:1].long()], last[:1], E32 * size[:1, :, None, None], "continued state")


def test_prefill_then_decode():
    """The pools that the prefill leaves are the decode step's."""
    m = Mix([70, 5, 64], HK=2, HV=4, K=128, V=128, io=F32, seed=5)
    pool = m.pool.clone()
    m.forward(initial_state=pool, final_state=pool)
    a = m.oracle()
    _, last, size = X.mix_forward(**a)
    n = Mix([1, 1, 1], HK=2, HV=4, K=128, V=128, io=F32, seed=6)
    o = R.gdn_standard_decode(pool, m.slot, n.q, n.k, n.v, n.g.exp(), n.beta)
    b = n.oracle()
    b["init"] = last
    want, last2, size2 = X.mix_forward(**b)
    size = np.maximum(size, size2)
    _near(o, want, E32 * (b["scale"] * size)[:, :, None], "decoded")
    _near(pool[m.slot.long()], last2, E32 * size[:, :, None, None], "state")


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", LINEAR, ids=lambda s: _ID(**s))
def test_decode(shape, io):
    """One token of every row, to another pool, in place, and by slots 0..n-1."""
    m = Mix([1] * 7, delta=False, io=io, wide=True, seed=9, **shape)
    m.has[:] = 1
    g = m.g
    new = torch.full_like(m.pool, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = R.linear_attention_decode(m.pool, m.slot, m.q, m.k, m.v, g, new_state=new, status=status)
    m.check_forward(o, new)
    other = torch.ones(m.slots, dtype=torch.bool)
    other[m.slot.cpu().long()] = False
    assert (new[other.cuda()] == 7.0).all() and int(status) == 0
    pool = m.pool.clone()
    assert torch.equal(R.linear_attention_decode(pool, m.slot, m.q, m.k, m.v, g), o)
    assert torch.equal(pool[m.slot.long()], new[m.slot.long()])
    rows = m.pool[m.slot.long()].contiguous()
    assert torch.equal(R.linear_attention_decode(rows, None, m.q, m.k, m.v, g), o)
    assert torch.equal(rows, new[m.slot.long()])


def test_decode_bad_slots():
    m = Mix([1] * 4, delta=False, initial=True, seed=2)
    m.has[:] = 1
    slot = m.slot.clone()
    slot[1], slot[3] = -1, m.slots
    pool, status = m.pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = R.linear_attention_decode(m.pool.clone(), m.slot, m.q, m.k, m.v, m.g)
    o = R.linear_attention_decode(pool, slot, m.q, m.k, m.v, m.g, status=status)
    assert int(status) == R.ST_BAD_SLOT
    assert torch.equal(o[::2], want[::2]) and torch.isnan(o[1::2]).all()
    keep = torch.ones(m.slots, dtype=torch.bool)
    keep[m.slot[::2].cpu().long()] = False
    assert torch.equal(pool[keep.cuda()], m.pool[keep.cuda()])


@pytest.mark.parametrize("delta", [False, True])
def test_status(delta):
    """A bad slot starts from zeros and stores nothing; a bad table is reported."""
    m = Mix([70, 3, 66], delta=delta, seed=4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    final = torch.full_like(m.pool, 7.0)
    o = m.forward(final_state=final, status=status)
    assert int(status) == 0
    slot = m.slot.clone()
    slot[0] = m.slots
    f2 = torch.full_like(m.pool, 7.0)
    o2 = m.forward(final_state=f2, slot_idx=slot, status=status)
    assert int(status) == R.ST_BAD_SLOT
    assert torch.equal(o2[70:], o[70:]) and (f2[m.slot[0].long()] == 7.0).all()
    has = m.has.clone()
    has[0] = 0
    assert torch.equal(o2, m.forward(has_initial=has))
    status.zero_()
    g = m.backward(slot_idx=slot, status=status)
    assert int(status) == R.ST_BAD_SLOT and (g["dinitial_state"][0] == 0).all()
    for bad in ([0, 70, 60, 139], [1, 70, 73, 139], [0, 70, 73, 130], [0, 70, 73, 150], [0, -5, 73, 139]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda: m.forward(final_state=f2, cu_seqlens=cu, status=status),
                     lambda: m.backward(cu_seqlens=cu, status=status)):
            status.zero_()
            call()
            assert int(status) & R.ST_BAD_SEQ, bad


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("io", [F32, BF16])
def test_extreme_gates(io, delta):
    """Decays of -infinity, far below any exponent, and zero; beta of 0 and 1; a key
    that repeats; states that are forgotten while others are kept."""
    m = Mix([150, 70], delta=delta, io=io, seed=8)
    m.g[3] = m.g[64, :2] = -math.inf
    m.g[70:80] = -1e30
    m.g[90], m.g[130:] = -200.0, 0.0
    m.g[:, 3] = 0.0
    m.beta[::3], m.beta[1::5] = 0.0, 1.0
    m.k[100:120] = m.k[100:101].clone()
    final = torch.empty_like(m.pool)
    m.check_forward(m.forward(final_state=final), final)
    m.check_backward(m.backward())


@pytest.mark.parametrize("delta", [False, True])
def test_other_sequences_are_left_alone(delta):
    """NaN in one sequence, in its state and in unused slots: the others' results
    have the same bits, gradients too."""
    m = Mix([66, 40, 130], delta=delta, seed=11)
    final, f2 = torch.zeros_like(m.pool), torch.zeros_like(m.pool)
    o, g = m.forward(final_state=final), m.backward()
    at = slice(66, 106)
    for t in (m.q, m.k, m.v, m.do, m.beta):
        t[at] = math.nan
    used = m.slot[[0, 2]].long()
    keep = m.pool[used].clone()
    m.pool[:] = math.nan
    m.pool[used] = keep
    o2, g2 = m.forward(final_state=f2), m.backward()
    for a, b in [(o, o2)] + [(g[k], g2[k]) for k in g if g[k] is not None and k != "dinitial_state"]:
        assert torch.equal(a[:66], b[:66]) and torch.equal(a[106:], b[106:])
    assert torch.equal(final[used], f2[used])
    assert torch.equal(g["dinitial_state"][[0, 2]], g2["dinitial_state"][[0, 2]])
    assert torch.isnan(o2[at]).all()


@pytest.mark.parametrize("delta", [False, True])
def test_gradients_are_differences(delta):
    """Directional derivatives of the fp32 forward, by central differences: their
    error is h^2 (h = 2^-7 relative steps) of the third derivative, which for these
    sizes is of the gradient's order: 2^-12; and the sums' roundings over h, 2^-17."""
    m = Mix([80, 33], delta=delta, io=F32, seed=13, initial=True)
    g = m.backward()
    gen = torch.Generator().manual_seed(1)
    names = dict(q="dq", k="dk", v="dv", g="dlog_g" if delta else "dlog_decay", pool="dinitial_state")
    if delta:
        names["beta"] = "dbeta"

    def loss():
        final = torch.zeros_like(m.pool)
        o = m.forward(final_state=final)
        return float((m.do.double() * o).sum() + (m.dlast.double() * final[m.slot.long()]).sum())
    for name, grad in names.items():
        x = getattr(m, name)
        way = torch.randn(x.shape, generator=gen).cuda() * x.abs().mean()
        dot = (g[grad].double() * (way[m.slot.long()] if name == "pool" else way)).sum()
        size = (g[grad].double().norm() * way.norm()).item()
        old, h = x.clone(), 2.0 ** -7
        x.copy_(old + h * way)
        up = loss()
        x.copy_(old - h * way)
        down = loss()
        x.copy_(old)
        assert abs((up - down) / (2 * h) - float(dot)) <= 2.0 ** -10 * size, name


@pytest.mark.parametrize("delta", [False, True])
def test_same_bits_streams_and_graphs(delta):
    """Two calls, a side stream, and a captured pass replayed between other work all
    give the same bits."""
    m = Mix([200, 7, 64], HK=2, HV=4, K=128, V=128, delta=delta, decay="token" if delta else "head", seed=17)

    def both(stream=None):
        final = torch.zeros_like(m.pool)
        o = m.forward(final_state=final, stream=stream)
        g = m.backward(stream=stream)
        return [o, final] + [t for t in g.values() if t is not None]
    want = both()
    for a, b in zip(want, both()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    v = m.v.clone()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        m.v.copy_(v * (i + 1))
        graph.replay()
        (torch.randn(256, 256, device="cuda") @ torch.randn(256, 256, device="cuda")).sum().item()
        kept = [t.clone() for t in got]
        for a, b in zip(both(), kept):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements, and rows 2^30 elements apart."""
    HV, K, slots = 32, 128, 4200
    pool = torch.empty((slots, HV, K, K), device="cuda")
    m = Mix([3, 2], HK=2, HV=HV, K=K, V=K, seed=19)
    at = [4150, 4199]
    for i, s in enumerate(at):
        pool[s] = m.pool[m.slot[i].long()]
    slot = torch.tensor(at, dtype=torch.int32, device="cuda")
    far = {}
    for name in ("q", "k", "v", "do"):
        x = getattr(m, name)
        big = torch.empty(4 * 2 ** 30 + x[0].numel(), dtype=x.dtype, device="cuda")
        far[name] = big.as_strided(x.shape, (2 ** 30, x.shape[2], 1))
        far[name].copy_(x)
    want, final = [], torch.empty_like(m.pool)
    want = [m.forward(final_state=final)] + list(m.backward().values())
    near = {n: getattr(m, n) for n in far}
    for n, x in far.items():
        setattr(m, n, x)
    got = [m.forward(initial_state=pool, final_state=pool, slot_idx=slot)]
    assert torch.equal(pool[at], final[m.slot.long()])
    for i, s in enumerate(at):
        pool[s] = m.pool[m.slot[i].long()]
    got += list(m.backward(initial_state=pool, slot_idx=slot).values())
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    step = [x[:2] for x in (far["q"], far["k"], far["v"])]
    plain = [near[n][:2] for n in ("q", "k", "v")]
    o = R.linear_attention_decode(pool, slot, *step, m.g[:2].contiguous())
    small = m.pool[m.slot.long()].contiguous()
    assert torch.equal(o, R.linear_attention_decode(small, None, *plain, m.g[:2].contiguous()))
    assert torch.equal(pool[at], small)


@pytest.mark.parametrize("delta", [False, True])
def test_segments_bits_streams_and_graphs(delta):
    """The same with sequences of several segments, whose order of work is made by
    atomic counters: two calls at once on two streams, and a captured pass replayed
    between others, give the same bits."""
    m = Mix([700, 64, 0, 1300, 1, 513, 520, 2], HK=2, HV=8, K=64, V=64, delta=delta,
            decay="token" if delta else "head", seed=23)

    def both(stream=None):
        final = torch.zeros_like(m.pool)
        o = m.forward(final_state=final, stream=stream)
        g = m.backward(stream=stream)
        return [o, final] + [t for t in g.values() if t is not None]
    want = both()
    m.check_forward(want[0], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        here = both()
        with torch.cuda.stream(side):
            there = both(stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(want, here, there):
            assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    v, cu = m.v.clone(), m.cu.clone()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        m.v.copy_(v * (i + 1))
        if i == 2:      # other lengths in the same graph: the order of work follows
            m.cu.copy_(torch.tensor([0, 1, 2000, 2001, 2001, 2500, 2900, 3099, 3100], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(both(), kept):
            assert torch.equal(a, b)
    m.cu.copy_(cu)


@pytest.mark.parametrize("delta", [False, True])
def test_segments_and_a_bad_table(delta):
    """A table that is not one is reported, and the rows of sequences that it gives
    right have the values they have without it."""
    m = Mix([600, 700, 40], delta=delta, initial=False, seed=29)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = m.forward()
    for bad in ([0, 600, 500, 1340], [0, 600, 1300, 1400], [-3, 600, 1300, 1340], [0, 600, 2 ** 31 - 1, 1340]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda: m.forward(cu_seqlens=cu, status=status), lambda: m.backward(cu_seqlens=cu, status=status)):
            status.zero_()
            call()
            assert int(status) & R.ST_BAD_SEQ, bad
    # the last row behind the last sequence keeps what was there
    cu = torch.tensor([0, 600, 1300, 1339], dtype=torch.int32, device="cuda")
    o = torch.full_like(want, 5.0)
    m.forward(cu_seqlens=cu, o=o)
    assert torch.equal(o[:1300], want[:1300]) and (o[1339] == 5.0).all()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("delta", [False, True])
def test_many_heads(delta, io):
    """More heads and sequences than compute units: a workgroup then takes all 128
    columns of a head forward, and otherwise half of them."""
    m = Mix([70, 3, 66, 1, 5], HK=16, HV=32, K=128, V=128, delta=delta, io=io, seed=37)
    final = torch.full_like(m.pool, 7.0)
    m.check_forward(m.forward(final_state=final), final)


def test_one_key_head_for_all():
    """Sixteen value heads on one key head, whose gradients add up over them."""
    for delta in (False, True):
        m = Mix([150, 20], HK=1, HV=16, K=64, V=64, delta=delta, decay="token", seed=31)
        m.check_forward(m.forward(), None)
        m.check_backward(m.backward())


# ------------------------------------------------------------------- positions

ROT = [(1, 1, 64, 64), (7, 3, 40, 40), (5, 2, 128, 14), (9, 5, 24, 2), (300, 4, 128, 128), (3, 2, 1024, 1024),
       (33, 70, 66, 62), (4, 1, 36, 34)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ROT, ids=str)
def test_rotary(shape, interleaved, io):
    """Each of the two products and their sum is off by 2^-24 of its size, the sine
    by 2^-25 of it: 2^-22 (|a| + |b|) covers them; then the io type's rounding."""
    T, H, D, rot = shape
    g = torch.Generator().manual_seed(T + rot)
    x = torch.randn(T, H, D, generator=g).to(io).cuda()
    pos = torch.randint(0, 1 << 20, (T,), generator=g).cuda()
    f = R.rotary_frequencies(rot)[0]
    keep = x.clone()
    for back in (False, True):
        fn = R.rotary_backward if back else R.rotary_forward
        want = X.rotary(_np(x), _np(pos), _np(f), interleaved, 1.25, back)
        size = np.abs(_np(x)).max(axis=2, keepdims=True) * 2.5
        tol = HALF[io] * abs(want) + 2.0 ** -22 * size
        y = fn(x, pos, f, interleaved=interleaved, amplitude=1.25)
        _near(y, want, tol, "rotary")
        assert torch.equal(y[..., rot:], x[..., rot:]) and torch.equal(x, keep)
        assert torch.equal(fn(x, pos.int(), f, interleaved=interleaved, amplitude=1.25), y)
        # a slice of wider rows, in place and into another slice of the same rows
        row = torch.full((T, 2 * H * D + 3), 7.0, dtype=io, device="cuda")
        a, b = row[:, 1:1 + H * D].unflatten(1, (H, D)), row[:, 2 + H * D:2 + 2 * H * D].unflatten(1, (H, D))
        a.copy_(x)
        assert fn(a, pos, f, interleaved=interleaved, amplitude=1.25, out=b) is b
        assert torch.equal(b, y) and torch.equal(a, x)
        fn(a, pos, f, interleaved=interleaved, amplitude=1.25, out=a)
        assert torch.equal(a, y) and torch.equal(b, y)
        assert (row[:, 0] == 7).all() and (row[:, 1 + H * D] == 7).all() and (row[:, -1] == 7).all()


def test_rotary_far_positions_and_none():
    """Positions near 2^31 and past 2^32, where an fp32 angle has no digits left;
    and no tokens."""
    f = R.rotary_frequencies(64)[0]
    x = torch.randn(4, 2, 64, device="cuda")
    pos = torch.tensor([2 ** 31 - 1, 2 ** 33 + 7, 0, 123456789], device="cuda")
    want = X.rotary(_np(x), _np(pos), _np(f))
    # the angle, up to 2^34, is exact to 2^-53 of itself: 2^-18 in both sides' sines
    _near(R.rotary_forward(x, pos, f), want, 2.0 ** -17 * float(x.abs().max()), "far")
    assert R.rotary_forward(x[:0], pos[:0], f).shape == (0, 2, 64)


def test_rotary_turns_back_and_replays():
    x = torch.randn(50, 3, 64, device="cuda")
    pos, f = torch.arange(50, device="cuda"), R.rotary_frequencies(64, scaling="yarn", factor=4.0,
                                                                  original_length=64)[0]
    y = R.rotary_forward(x, pos, f)
    size = float(x.abs().max())
    assert float((R.rotary_backward(y, pos, f) - x).abs().max()) <= 2.0 ** -20 * size
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        R.rotary_forward(x, pos, f, out=out)
    for i in range(3):
        pos += 1
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, R.rotary_forward(x, pos, f))


# ------------------------------------------------------------------- refusals

def test_binding_refusals():
    m = Mix([5, 4], delta=True)
    ok = dict(q=m.q, k=m.k, v=m.v, log_g=m.g, beta=m.beta, cu_seqlens=m.cu)
    R.gdn_scan_forward(**ok)
    far = torch.zeros(9, 2, 64, dtype=BF16)
    for bad in (dict(q=far), dict(k=far), dict(q=m.q.float()), dict(q=m.q[:, :, :32]), dict(k=m.k[:8]),
                dict(v=m.v[:, :3].contiguous()), dict(v=m.v.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(log_g=None), dict(log_g=m.g[0].contiguous()), dict(log_g=m.g.double()), dict(beta=None),
                dict(beta=m.beta[:, :2].contiguous()), dict(beta=m.beta.to(BF16)), dict(scale=0.0),
                dict(scale=-1.0), dict(cu_seqlens=m.cu.long()), dict(cu_seqlens=m.cu[None]),
                dict(initial_state=m.pool.to(BF16)), dict(initial_state=m.pool[:, :2].contiguous()),
                dict(initial_state=m.pool, final_state=m.pool[:3].contiguous()), dict(slot_idx=m.slot.long()),
                dict(has_initial=m.has.bool()), dict(o=torch.empty(9, 4, 64, device="cuda")),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, R.RssmError)):
            R.gdn_scan_forward(**{**ok, **bad})
    lin = dict(q=m.q, k=m.k, v=m.v)
    for bad in (dict(log_decay=m.g[:, :2].contiguous()), dict(log_decay=m.g[0, :3].contiguous()),
                dict(log_decay=m.g[:8].contiguous())):
        with pytest.raises(ValueError):
            R.linear_attention_forward(**{**lin, **bad})
    with pytest.raises(ValueError):
        R.linear_attention_decode(None, None, m.q, m.k, m.v)
    with pytest.raises(ValueError):
        R.gdn_scan_backward(m.do.float(), m.q, m.k, m.v, m.g, m.beta)
    with pytest.raises(ValueError):
        R.gdn_scan_backward(m.do, m.q, m.k, m.v, m.g, m.beta, cu_seqlens=m.cu, dfinal_state=m.dlast[:1])
    x, pos, f = m.v, torch.arange(9, device="cuda"), R.rotary_frequencies(64)[0]
    for bad in (dict(positions=pos[:8]), dict(positions=pos.float()), dict(positions=None), dict(freqs=f.double()),
                dict(freqs=torch.ones(33, device="cuda")), dict(freqs=f[:0]), dict(freqs=None),
                dict(out=x[:8]), dict(out=x.float()), dict(x=x[:, :, ::2])):
        with pytest.raises(ValueError):
            R.rotary_forward(**{**dict(x=x, positions=pos, freqs=f), **bad})
    whole = torch.zeros(10, 4, 64, dtype=BF16, device="cuda")
    with pytest.raises(R.RssmError):   # rows over other rows
        R.rotary_forward(whole[:9], pos, f, out=whole[1:])


def test_differentiating_a_result_raises():
    m = Mix([5, 4], delta=True)
    q = m.q.detach().requires_grad_()
    st = m.pool.clone()
    for o in (R.gdn_scan_forward(q, m.k, m.v, m.g, m.beta), R.linear_attention_forward(q, m.k, m.v, m.g),
              R.linear_attention_decode(torch.zeros(9, 4, 64, 64, device="cuda"), None, q, m.k, m.v, m.g),
              R.rotary_forward(q, torch.arange(9, device="cuda"), R.rotary_frequencies(64)[0])):
        with pytest.raises(RuntimeError, match="backward pass"):
            o.float().sum().backward()
    assert torch.equal(st, m.pool)
