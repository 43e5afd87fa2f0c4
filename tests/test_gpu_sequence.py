"""Sequence operators on the GPU against the 64-bit oracle.

Tolerances are element by element.  With u = 2^-8 (bf16's half step) for
bf16 inputs and outputs and m the size of the terms a result adds up:

* an fp32 result, or an fp32 part of one: E32 * m with E32 = 2^-16.  A sum of
  up to N + 64 terms is off by at most (N + 64) 2^-24 m <= 2^-15.6 m if every
  rounding went one way; they do not, and the decays' exponents (relative
  error 2^-22, entering as |g| e^-|g| 2^-22) and hardware exp2, exp and
  reciprocal (2^-22 each) stay below 2^-18.
* a bf16 result of the scan: u |v| for its rounding and u m for the one factor
  of each product that is rounded to bf16 (decay times C.B, decay times
  dy.x, or the state).
* a bf16 result of the convolution or the norm: u |v| + E32 m.
* e4m3: 2^-4 of the value (2^-10 absolute below its smallest normal number),
  plus what the scale's and y's fp32 error shift it by (2^-18 of the value).
"""

import math

import numpy as np
import pytest
import torch

import linear_recurrence_amd as R
from oracle import sequence as Q

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
    bad = ~(off <= tol + 1e-30)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, off by up to " \
        f"{np.nanmax(off[bad] / (np.broadcast_to(tol, off.shape)[bad] + 1e-30)):.3g} tolerances"


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


class Scan:
    """Inputs of a scan; x, B, C and dt are slices of one wide row, as a
    projection's output is, or tensors of their own."""

    def __init__(self, lens, H=4, P=64, N=32, G=2, io=BF16, state=F32, initial=True, wide=False,
                 seed=0):
        g = torch.Generator().manual_seed(seed)
        T, n = sum(lens), len(lens)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lens, self.starts, self.io, self.n = lens, _starts(lens), io, n
        x, B, C = rnd(T, H, P).to(io), (rnd(T, G, N) / 4).to(io), (rnd(T, G, N) / 4).to(io)
        dt = rnd(T, H).to(io)
        if wide:
            pad = torch.full((T, 8), float("nan"), dtype=io)
            row = torch.cat([pad, x.flatten(1), pad, B.flatten(1), C.flatten(1), dt, pad], 1)
            row = torch.cat([row, torch.full((T, -row.shape[1] % 8), float("nan"), dtype=io)], 1).cuda()
            at = 8
            self.x = row[:, at:at + H * P].unflatten(1, (H, P))
            at += H * P + 8
            self.B = row[:, at:at + G * N].unflatten(1, (G, N))
            at += G * N
            self.C = row[:, at:at + G * N].unflatten(1, (G, N))
            at += G * N
            self.dt = row[:, at:at + H]
        else:
            self.x, self.B, self.C, self.dt = x.cuda(), B.cuda(), C.cuda(), dt.cuda()
        self.A = -torch.exp(torch.rand(H, generator=g) * math.log(16.0)).cuda()
        self.D = rnd(H).cuda()
        self.bias = torch.log(torch.expm1(torch.rand(H, generator=g) * 0.099 + 0.001)).cuda()
        self.z, self.dy = rnd(T, H, P).to(io).cuda(), rnd(T, H, P).to(io).cuda()
        self.slots = n + 3
        self.pool = (rnd(self.slots, H, P, N) * 0.1).to(state).cuda()
        self.slot = torch.randperm(self.slots, generator=g)[:n].to(torch.int32).cuda()
        self.has = torch.tensor([i % 3 != 2 for i in range(n)], dtype=torch.uint8).cuda()
        self.initial = initial
        self.dlast = (rnd(n, H, P, N) * 0.1).cuda()
        self.cu = torch.tensor(self.starts, dtype=torch.int32).cuda()

    def oracle_inputs(self):
        init = np.zeros((self.n,) + tuple(self.pool.shape[1:]))
        if self.initial:
            init = _np(self.pool[self.slot.long()]) * _np(self.has)[:, None, None, None]
        dt = Q.scan_dt(_np(self.dt), _np(self.bias))
        return dict(x=_np(self.x), dt=dt, A=_np(self.A), B=_np(self.B), C=_np(self.C),
                    D=_np(self.D), starts=self.starts, init=init)

    def forward(self, **over):
        a = dict(D=self.D, dt_bias=self.bias, cu_seqlens=self.cu, slot_idx=self.slot,
                 initial_state=self.pool if self.initial else None,
                 has_initial=self.has if self.initial else None)
        a.update(over)
        return R.ssu_scan_forward(self.x, self.dt, self.A, self.B, self.C, **a)

    def backward(self, **over):
        a = dict(D=self.D, dt_bias=self.bias, cu_seqlens=self.cu, slot_idx=self.slot,
                 initial_state=self.pool if self.initial else None,
                 has_initial=self.has if self.initial else None, dfinal_state=self.dlast)
        a.update(over)
        return R.ssu_scan_backward(self.dy, self.x, self.dt, self.A, self.B, self.C, **a)

    def check_forward(self, y, final, z=False):
        a = self.oracle_inputs()
        want, last = Q.scan_forward(**a)
        mag, mlast = Q.scan_magnitude(**a)
        u = HALF[self.io]
        if z:
            gate = _np(self.z) * Q.sigmoid(_np(self.z))
            want, mag = want * gate, mag * abs(gate)
        _near(y, want, u * (abs(want) + mag) + E32 * mag, "y")
        if final is not None:
            _near(final[self.slot.long()], last, HALF[final.dtype] * abs(last) + E32 * mlast, "final")

    def check_backward(self, got, dlast=True):
        a = self.oracle_inputs()
        a["dlast"] = _np(self.dlast) if dlast else np.zeros(a["init"].shape)
        want = Q.scan_backward(_np(self.dy), **a)
        mag = Q.scan_backward(_np(self.dy), **a, magnitude=True)
        raw = _np(self.dt) + _np(self.bias)
        sig = Q.sigmoid(raw)
        for d in (want, mag):
            d["ddt"] = d["ddt"] * sig
            d["ddt_bias"] = d["ddt"].sum(0)
            d["dinitial_state"] = d["dinit"] * _np(self.has)[:, None, None, None]
        mag["dD"] = (abs(_np(self.dy)) * abs(_np(self.x))).sum((0, 2))
        u = HALF[self.io]
        for k in ("dx", "dB", "dC"):
            _near(got[k], want[k], u * (abs(want[k]) + mag[k]) + E32 * mag[k], k)
        _near(got["ddt"], want["ddt"], u * abs(want["ddt"]) + E32 * mag["ddt"], "ddt")
        for k in ("dA", "dD", "ddt_bias"):
            _near(got[k], want[k], E32 * mag[k], k)
        if self.initial:
            _near(got["dinitial_state"], want["dinitial_state"], E32 * mag["dinitial_state"], "dinit")


LENS = [[1], [0], [3, 0, 1, 63, 64, 65, 0], [130], [257, 1, 0, 300]]
SHAPES = [dict(H=4, P=64, N=128, G=1), dict(H=6, P=32, N=16, G=2), dict(H=3, P=128, N=64, G=3),
          dict(H=10, P=64, N=256, G=2), dict(H=5, P=128, N=256, G=1), dict(H=2, P=32, N=32, G=1)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "H{H}P{P}N{N}G{G}".format(**s))
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_scan(lens, shape, io):
    s = Scan(lens, io=io, state=io, wide=lens == [130], seed=len(lens), **shape)
    final = torch.full_like(s.pool, 7.0)
    y = s.forward(final_state=final)
    s.check_forward(y, final)
    other = torch.ones(s.slots, dtype=torch.bool)
    other[s.slot.cpu().long()] = False
    assert (final[other.cuda()] == 7.0).all()          # no other slot is written
    s.check_forward(s.forward(z=s.z), None, z=True)
    s.check_backward(s.backward())


@pytest.mark.parametrize("io", [F32, BF16])
def test_scan_bare(io):
    """No D, dt_bias, table, slots or states; dt taken as it is."""
    s = Scan([100], io=io, initial=False)
    dt = torch.rand(100, 4, generator=torch.Generator().manual_seed(3)).to(io).cuda() * 0.2
    y = R.ssu_scan_forward(s.x, dt, s.A, s.B, s.C, dt_softplus=False)
    a = s.oracle_inputs()
    a.update(dt=_np(dt), D=None)
    want, _ = Q.scan_forward(**a)
    mag, _ = Q.scan_magnitude(**a)
    _near(y, want, HALF[io] * (abs(want) + mag) + E32 * mag, "y")
    got = R.ssu_scan_backward(s.dy, s.x, dt, s.A, s.B, s.C, dt_softplus=False)
    assert got["dD"] is None and got["ddt_bias"] is None and got["dinitial_state"] is None
    a["dlast"] = np.zeros(a["init"].shape)
    want = Q.scan_backward(_np(s.dy), **a)
    mag = Q.scan_backward(_np(s.dy), **a, magnitude=True)
    for k in ("dx", "dB", "dC", "ddt"):
        _near(got[k], want[k], HALF[io] * (abs(want[k]) + mag[k]) + E32 * mag[k], k)
    _near(got["dA"], want["dA"], E32 * mag["dA"], "dA")


@pytest.mark.parametrize("state", [F32, BF16])
def test_scan_in_place_over_many_segments(state):
    """The final states over the initial ones, sequences of many segments."""
    s = Scan([1500, 2, 700], H=2, P=32, N=16, G=1, state=state)
    old = s.pool.clone()
    ref = torch.empty_like(s.pool)
    y = s.forward(final_state=ref)
    s.check_forward(y, ref)
    y2 = s.forward(final_state=s.pool)
    assert torch.equal(y, y2)
    assert torch.equal(s.pool[s.slot.long()], ref[s.slot.long()])
    s.pool = old
    s.check_backward(s.backward())


def test_scan_no_tokens():
    s = Scan([0, 0], io=BF16)
    final = torch.zeros_like(s.pool)
    assert s.forward(final_state=final).shape == (0, 4, 64)
    s.check_forward(s.forward(final_state=final), final)
    got = s.backward()
    assert float(got["dA"].abs().sum()) == 0.0
    keep = s.has.bool()[:, None, None, None]
    assert torch.equal(got["dinitial_state"], torch.where(keep, s.dlast, torch.zeros_like(s.dlast)))


def test_scan_large_steps_and_far_decays():
    """Decays that underflow within a chunk, and none at all."""
    s = Scan([200, 70], H=4, P=32, N=32, G=1)
    s.dt.mul_(8.0)
    s.A = torch.tensor([-16.0, -1e-3, 0.0, -200.0]).cuda()
    final = torch.empty_like(s.pool)
    s.check_forward(s.forward(final_state=final), final)
    s.check_backward(s.backward())


def test_scan_status_and_nothing_out_of_range():
    s = Scan([40, 30], H=2, P=32, N=16, G=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.forward(status=status)
    s.backward(status=status)
    assert int(status) == 0
    bad = s.slot.clone()
    bad[1] = s.slots
    final = torch.full_like(s.pool, 3.0)
    s.forward(slot_idx=bad, final_state=final, status=status)
    assert int(status) == R.ST_BAD_SLOT
    rest = torch.ones(s.slots, dtype=torch.bool)
    rest[int(bad[0])] = False
    assert (final[rest.cuda()] == 3.0).all()
    for table in ([0, 40, 90], [0, -5, 70], [0, 50, 40], [4, 40, 70]):
        status.zero_()
        cu = torch.tensor(table, dtype=torch.int32, device="cuda")
        s.forward(cu_seqlens=cu, status=status)
        assert int(status) & R.ST_BAD_SEQ
        status.zero_()
        s.backward(cu_seqlens=cu, status=status)
        assert int(status) & R.ST_BAD_SEQ


def test_scan_other_sequences_do_not_see_a_nan():
    s = Scan([100, 64, 90], H=4, P=64, N=64, G=1)
    y0, g0 = s.forward(), s.backward()
    s.x[120, 1, 5] = float("nan")
    y1, g1 = s.forward(), s.backward()
    keep = [slice(0, 100), slice(164, 254)]
    for k in keep:
        assert torch.equal(y0[k], y1[k]) and torch.equal(g0["dx"][k], g1["dx"][k])
        assert torch.equal(g0["dB"][k], g1["dB"][k])
    assert y1[120, 1].isnan().any()


# ---------------------------------------------------------------- convolution

@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 33, 520])
@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("lens", [[1], [0, 2, 1, 40, 3, 0], [200, 5, 130]], ids=str)
def test_conv(lens, act, C, W, io):
    g = torch.Generator().manual_seed(W)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, n, starts = sum(lens), len(lens), _starts(lens)
    wide = rnd(T, 2 * C + 3).to(io).cuda()
    x, dy = wide[:, 1:1 + C], wide[:, C + 2:2 * C + 2]       # rows that start anywhere
    w, b = (rnd(C, W) / 2).cuda(), rnd(C).cuda()
    pool, slot = rnd(n + 2, W - 1, C).to(io).cuda(), torch.randperm(n + 2, generator=g)[:n].to(torch.int32).cuda()
    has = torch.tensor([i % 3 != 1 for i in range(n)], dtype=torch.uint8).cuda()
    cu = torch.tensor(starts, dtype=torch.int32).cuda()
    init = _np(pool[slot.long()]) * _np(has)[:, None, None]
    a = dict(cu_seqlens=cu, initial_state=pool, has_initial=has, slot_idx=slot, activation=act)
    u = HALF[io]
    want, last, _ = Q.conv_forward(_np(x), _np(w), _np(b), starts, init, act == "silu")
    mag = Q.conv_forward(abs(_np(x)), abs(_np(w)), abs(_np(b)), starts, abs(init), False)[0]
    final = pool.clone()
    y = R.causal_conv_forward(x, w, bias=b, final_state=final, **a)
    _near(y, want, u * abs(want) + E32 * mag, "y")
    assert np.array_equal(_np(final[slot.long()]), last)     # moved, not computed
    in_place = pool.clone()
    a["initial_state"] = in_place
    assert torch.equal(R.causal_conv_forward(x, w, bias=b, final_state=in_place, **a), y)
    assert torch.equal(in_place, final)
    a["initial_state"] = pool
    got = R.causal_conv_backward(dy, x, w, bias=b, **a)
    want = Q.conv_backward(_np(dy), _np(x), _np(w), _np(b), starts, init, act == "silu")
    m = Q.conv_backward(_np(dy), _np(x), _np(w), _np(b), starts, init, act == "silu", magnitude=True)
    # silu' multiplies a dv whose own relative error is that of v, |v| <= mag
    more = 1.0 + float(mag.max()) if T else 1.0
    _near(got["dx"], want["dx"], u * abs(want["dx"]) + E32 * m["dx"] * more, "dx")
    for k in ("dweight", "dbias"):
        _near(got[k], want[k], E32 * m[k] * more, k)
    di = want["dinit"] * _np(has)[:, None, None]
    _near(got["dinitial_state"][slot.long()], di, u * abs(di) + E32 * m["dinit"] * more, "dinit")
    rest = torch.ones(n + 2, dtype=torch.bool)
    rest[slot.cpu().long()] = False
    assert float(got["dinitial_state"][rest.cuda()].abs().sum()) == 0.0


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_steps_continue_a_prefill(W, io):
    """Prefill, then token by token in place: the same bits as the whole."""
    g = torch.Generator().manual_seed(1)
    C, T = 77, 9
    x, w = torch.randn(T, C, generator=g).to(io).cuda(), torch.randn(C, W, generator=g).cuda()
    whole = R.causal_conv_forward(x, w)
    state = torch.zeros(3, W - 1, C, dtype=io, device="cuda")
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    y = [R.causal_conv_forward(x[:4], w, final_state=state, slot_idx=slot)]
    for t in range(4, T):
        y.append(R.causal_conv_decode(x[t:t + 1], state, w, slot_idx=slot))
    assert torch.equal(torch.cat(y), whole)
    assert float(state[:2].abs().sum()) == 0.0


def test_conv_status():
    x, w = torch.randn(4, 16, device="cuda"), torch.randn(16, 4, device="cuda")
    st = torch.zeros(2, 3, 16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([0, 5, 1, -1], dtype=torch.int32, device="cuda")
    y = R.causal_conv_decode(x, st, w, slot_idx=slot, status=status)
    assert int(status) == R.ST_BAD_SLOT
    assert y[1].isnan().all() and y[3].isnan().all() and not y[[0, 2]].isnan().any()
    for table in ([0, 9, 4], [0, 3, 2], [1, 2, 4]):
        status.zero_()
        cu = torch.tensor(table, dtype=torch.int32, device="cuda")
        R.causal_conv_forward(x, w, cu_seqlens=cu, status=status)
        assert int(status) & R.ST_BAD_SEQ
        R.causal_conv_backward(x, x, w, cu_seqlens=cu)


def test_conv_slots_past_32_bits():
    """A pool of more than 2^31 elements: its last slot."""
    C, slots = 4096, (1 << 31) // (3 * 4096) + 2
    pool = torch.empty(slots, 3, C, dtype=BF16, device="cuda")
    pool[-1] = 1.0
    x, w = torch.ones(1, C, dtype=BF16, device="cuda"), torch.ones(C, 4, device="cuda")
    slot = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    y = R.causal_conv_decode(x, pool, w, slot_idx=slot, activation=None)
    assert (y == 4.0).all() and (pool[-1] == 1.0).all()
    y = R.causal_conv_forward(x, w, initial_state=pool, slot_idx=slot, activation=None)
    assert (y == 4.0).all()


# ------------------------------------------------------------------- the norm

NORMS = [(1, 8, 8), (3, 40, 40), (5, 130, 65), (2, 512, 128), (4, 1031, 1031), (3, 5120, 5120),
         (2, 8192, 1024), (2, 16384, 16384), (1, 32768, 32768), (3, 24, 3)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("size", NORMS, ids=str)
def test_norm(size, gate, io):
    rows, dim, group = size
    g = torch.Generator().manual_seed(dim)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wide = rnd(rows, 3 * dim + 1).to(io).cuda()
    x, z, dy = wide[:, :dim], wide[:, dim:2 * dim] if gate else None, wide[:, 2 * dim:3 * dim]
    w = (1.0 + 0.2 * rnd(dim)).cuda()
    u, nz = HALF[io], None if z is None else _np(z)
    for res in (None, F32, io):
        r = None if res is None else (3.0 * rnd(rows, dim)).to(res).cuda()
        h = _np(x)
        got = R.rms_norm_forward(x, w, z=z, residual=r, group_size=group)
        if r is not None:
            h = h + _np(r)
            _near(got["residual"], h, HALF[res] * abs(h) + 2.0 ** -24 * abs(h), "residual")
            h = _np(got["residual"])
            again = r.clone()
            same = R.rms_norm_forward(x, w, z=z, residual=again, group_size=group, residual_out=again)
            assert torch.equal(again, got["residual"]) and torch.equal(same["out"], got["out"])
        want = Q.norm_forward(h, _np(w), nz, group, 1e-5)
        _near(got["out"], want, u * abs(want) + E32 * abs(want), "out")
    got = R.rms_norm_backward(dy, x, w, z=z, group_size=group)
    want, mag = Q.norm_backward(_np(dy), _np(x), _np(w), nz, group, 1e-5)
    for k in want:
        half = HALF[F32] if k == "dweight" else u
        # dz: 1 + z (1 - s) may cancel: its error is relative to 1 + |z|
        more = 8.0 if k == "dz" else 1.0
        extra = 2.0 ** -20 * np.abs(_np(dy)).max() * np.abs(_np(x)).max() * 8 if k == "dz" else 0.0
        _near(got[k], want[k], half * abs(want[k]) + E32 * mag[k] * more + extra, k)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("size", [(3, 128, 128), (5, 1280, 640), (2, 5120, 5120), (4, 8192, 1024)], ids=str)
def test_norm_8bit(size, block, io):
    rows, dim, group = size
    g = torch.Generator().manual_seed(dim)
    x, w = torch.randn(rows, dim, generator=g).to(io).cuda(), torch.randn(dim, generator=g).cuda()
    x[0] = 0.0                                     # a row of zeros has scale 1
    got = R.rms_norm_forward(x, w, group_size=group, out_dtype=torch.float8_e4m3fn, scale_block=block)
    want = Q.norm_forward(_np(x), _np(w), None, group, 1e-5)
    b = block or dim
    top = abs(want).reshape(rows, -1, b).max(-1)
    scale = np.where(top > 0, top / 448.0, 1.0)
    _near(got["scale"], scale, E32 * scale, "scale")
    q = want / np.repeat(scale, b, 1)
    # half a step of e4m3, or of its subnormal numbers, and the next step's where the error crosses
    _near(got["out"].float(), q, abs(q) * (2.0 ** -4 + 2.0 ** -14) + 2.0 ** -10 * (1 + 2.0 ** -8), "out")


def test_norm_odd_rows_8bit():
    x, w = torch.randn(3, 37, device="cuda").to(BF16), torch.ones(37, device="cuda")
    got = R.rms_norm_forward(x, w, out_dtype=torch.float8_e4m3fn)
    want = Q.norm_forward(_np(x), _np(w), None, 37, 1e-5)
    back = _np(got["out"].float()) * _np(got["scale"])
    assert (abs(back - want) <= abs(want) * (2.0 ** -4 + 2.0 ** -14) + 2.0 ** -9 * _np(got["scale"])).all()


def test_norm_keeps_non_finite_rows_apart():
    x = torch.randn(4, 600, device="cuda")
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    w = torch.ones(600, device="cuda")
    clean = R.rms_norm_forward(x[[0, 3]], w, out_dtype=torch.float8_e4m3fn)
    got = R.rms_norm_forward(x, w, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(got["out"][[0, 3]].view(torch.uint8), clean["out"].view(torch.uint8))
    assert got["out"][1].float().isnan().all()
    assert got["out"][2, 9].float().isnan()
    zero = R.rms_norm_forward(torch.zeros(1, 8, device="cuda"), torch.ones(8, device="cuda"), eps=0.0)
    assert zero["out"].isnan().all()              # 0 * rsqrt(0), as the formula has it


def test_norm_rows_past_32_bits():
    stride, rows, dim = 1 << 22, 520, 64
    flat = torch.empty(stride * rows, dtype=BF16, device="cuda")
    x = flat.view(rows, stride)[:, :dim]
    x.copy_(torch.randn(rows, dim, device="cuda"))
    w = torch.ones(dim, device="cuda")
    a, b = R.rms_norm_forward(x, w), R.rms_norm_forward(x.contiguous(), w)
    assert torch.equal(a["out"], b["out"])
    a, b = R.rms_norm_backward(x, x, w), R.rms_norm_backward(x.contiguous(), x.contiguous(), w)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])


def test_norm_no_rows():
    x, w = torch.zeros(0, 16, device="cuda"), torch.ones(16, device="cuda")
    assert R.rms_norm_forward(x, w)["out"].shape == (0, 16)
    assert float(R.rms_norm_backward(x, x, w)["dweight"].abs().sum()) == 0.0


# ------------------------------------------------------------- streams, graphs

def _all(s, w, b, nw):
    out = [s.forward(z=s.z), R.causal_conv_forward(s.x.flatten(1), w, bias=b, cu_seqlens=s.cu)]
    out += [v for v in s.backward().values()]
    out += [v for v in R.causal_conv_backward(s.dy.flatten(1), s.x.flatten(1), w, bias=b,
                                              cu_seqlens=s.cu).values() if v is not None]
    out += [v for v in R.rms_norm_forward(s.x.flatten(1), nw, z=s.z.flatten(1),
                                          residual=s.dy.flatten(1)).values() if v is not None]
    out += [v for v in R.rms_norm_backward(s.dy.flatten(1), s.x.flatten(1), nw,
                                           z=s.z.flatten(1)).values()]
    return out


def _setup():
    s = Scan([700, 20, 0, 333], H=4, P=64, N=128, G=2)
    C = 256
    return s, torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda"), torch.ones(C, device="cuda")


def _same(a, b):
    return all(torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))
               for p, q in zip(a, b))


def test_same_bits_every_time_and_on_another_stream():
    args = _setup()
    ref = _all(*args)
    for _ in range(3):
        assert _same(ref, _all(*args))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = _all(*args)
    st.synchronize()
    assert _same(ref, got)
    y = args[0].forward(z=args[0].z, stream=st)
    st.synchronize()
    assert torch.equal(y, ref[0])


def test_graph_replays():
    args = _setup()
    ref = _all(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _all(*args)
    x = args[0].x.clone()
    for k in range(3):
        for o in out:
            o.fill_(0)
        args[0].x.copy_(x * (k + 1))
        g.replay()
        torch.cuda.synchronize()
        a = torch.randn(256, 256, device="cuda")
        (a @ a).sum().item()
        assert _same(out, _all(*args) if k else ref)


def test_binding_refusals():
    s = Scan([8], H=2, P=32, N=16, G=1)
    ok = dict(D=s.D, dt_bias=s.bias)
    with pytest.raises(ValueError, match="dt has"):
        R.ssu_scan_forward(s.x, s.dt.float(), s.A, s.B, s.C, **ok)
    with pytest.raises(ValueError, match="A has"):
        R.ssu_scan_forward(s.x, s.dt, s.A[:1], s.B, s.C, **ok)
    with pytest.raises(ValueError, match="final_state"):
        R.ssu_scan_forward(s.x, s.dt, s.A, s.B, s.C, initial_state=s.pool, final_state=s.pool.to(BF16), **ok)
    with pytest.raises(ValueError, match="contiguous"):
        R.ssu_scan_forward(s.x.transpose(1, 2).contiguous().transpose(1, 2), s.dt, s.A, s.B, s.C, **ok)
    with pytest.raises(ValueError, match="cu_seqlens"):
        R.ssu_scan_forward(s.x, s.dt, s.A, s.B, s.C, cu_seqlens=s.cu.long(), **ok)
    with pytest.raises(R.RssmError, match="shape"):
        R.ssu_scan_forward(torch.zeros(8, 2, 48, device="cuda"), torch.zeros(8, 2, device="cuda"), s.A,
                           torch.zeros(8, 1, 16, device="cuda"), torch.zeros(8, 1, 16, device="cuda"))
    with pytest.raises(R.RssmError):
        R.causal_conv_forward(torch.zeros(3, 8, device="cuda"), torch.zeros(8, 5, device="cuda"))
    with pytest.raises(ValueError, match="activation"):
        R.causal_conv_forward(torch.zeros(3, 8, device="cuda"), torch.zeros(8, 4, device="cuda"), activation="gelu")
    with pytest.raises(ValueError, match="scale_block"):
        R.rms_norm_forward(torch.zeros(3, 128, device="cuda"), torch.ones(128, device="cuda"), scale_block=128)
    with pytest.raises(ValueError, match="out_dtype"):
        R.rms_norm_forward(torch.zeros(3, 128, device="cuda"), torch.ones(128, device="cuda"), out_dtype=BF16)
