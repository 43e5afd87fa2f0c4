"""The sequence operators at the sizes where their host rules pick another kernel,
or where a kernel's loops take a second round.

Each case states the rule it is chosen by and checks that it still holds.  The
tolerances are those of test_gpu_sequence.py; the scan's bf16 results get only
their own rounding and the fp32 part, as in test_gpu_scan_rounding.py.
"""

import numpy as np
import pytest
import torch

import linear_recurrence_amd as R
from oracle import sequence as Q
from test_gpu_sequence import BF16, E32, F32, HALF, Scan, _near, _np, _starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- the scan

def _check_scan(s, y, final, got):
    """All of a scan's results."""
    a, u = s.oracle_inputs(), HALF[s.io]
    want, last = Q.scan_forward(**a)
    mag, mlast = Q.scan_magnitude(**a)
    _near(y, want, u * abs(want) + E32 * mag, "y")
    _near(final[s.slot.long()], last, HALF[final.dtype] * abs(last) + E32 * mlast, "final")
    a["dlast"] = _np(s.dlast)
    want = Q.scan_backward(_np(s.dy), **a)
    mag = Q.scan_backward(_np(s.dy), **a, magnitude=True)
    mag["dD"] = (abs(_np(s.dy)) * abs(_np(s.x))).sum((0, 2))
    sig = Q.sigmoid(_np(s.dt) + _np(s.bias))
    for d in (want, mag):
        d["ddt"] = d["ddt"] * sig
        d["ddt_bias"] = d["ddt"].sum(0)
        d["dinitial_state"] = d["dinit"] * _np(s.has)[:, None, None, None]
    for k in ("dx", "dB", "dC", "ddt"):
        _near(got[k], want[k], u * abs(want[k]) + E32 * mag[k], k)
    for k in ("dA", "dD", "ddt_bias", "dinitial_state"):
        _near(got[k], want[k], E32 * mag[k], k)


# heads, headdim, dstate, type, waves of the backward's workgroup, empty sequences
UNITS = [(17, 64, 128, BF16, 8, 250), (17, 64, 64, BF16, 4, 510), (9, 128, 32, BF16, 4, 510),
         (17, 32, 256, BF16, 8, 250), (17, 64, 16, BF16, 4, 510), (9, 64, 128, F32, 4, 510),
         (9, 64, 16, F32, 4, 510)]


@pytest.mark.parametrize("case", UNITS, ids=lambda c: "H{}P{}N{}-{}".format(c[0], c[1], c[2], str(c[3])[6:]))
def test_scan_with_many_units_a_workgroup(case):
    """17 or 18 units (a head's 32 or 64 state rows) a group: workgroups of 16 and of
    the rest, in the forward's output launch and the backward's main one.  Both
    take 16 where that leaves enough workgroups, which empty sequences, each with
    a chunk's place, make up for here."""
    H, P, N, io, waves, empty = case
    lens = [70, 1] + [0] * empty + [130, 64, 3]
    T, n = sum(lens), len(lens)
    chunks = T // 64 + n
    rows = 32 if io is F32 or P == 32 or N == 256 else 64
    bwd, fwd = H * (P // rows), H * max(1, P // 64)
    assert bwd > 16 and chunks * _up(bwd, 16) >= (512 if waves == 8 else 1024)
    assert T > 128 and fwd > 8 and chunks * _up(fwd, 16) >= 256
    s = Scan(lens, H=H, P=P, N=N, G=1, io=io, seed=N)
    final = torch.empty_like(s.pool)
    y = s.forward(final_state=final)
    _check_scan(s, y, final, s.backward())


@pytest.mark.parametrize("io", [F32, BF16])
def test_scan_groups_with_many_units(io):
    """Two groups of 17 or 34 units each: 16, 16 and 2 of one group never mix with the other's."""
    lens = [70] + [0] * 260 + [130]
    assert (sum(lens) // 64 + len(lens)) * 2 * _up(17, 16) >= 1024
    s = Scan(lens, H=34, P=64 if io is F32 else 32, N=16, G=2, io=io, seed=8)
    final = torch.empty_like(s.pool)
    y = s.forward(final_state=final)
    _check_scan(s, y, final, s.backward())


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("state", [F32, BF16])
def test_scan_over_many_segments(io, state):
    """11 and 17 segments of 256 tokens: the combining launches take eight at a time."""
    lens = [2700, 5, 4300]
    s = Scan(lens, H=2, P=32, N=16, G=1, io=io, state=state, seed=9)
    for waves in (2048, 1024):                        # forward, backward
        assert max(256, _up(sum(lens) * 2, waves) + 63 & ~63) == 256
    final = torch.empty_like(s.pool)
    y = s.forward(final_state=final)
    _check_scan(s, y, final, s.backward())
    assert torch.equal(s.forward(final_state=s.pool), y)          # over the initial states
    assert torch.equal(s.pool[s.slot.long()], final[s.slot.long()])


# ---------------------------------------------------------------- convolution

def _run(T, blocks):
    run = 32
    while run > 8 and _up(T, run) * blocks < 2048:
        run >>= 1
    return run


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T, C, run", [(65600, 33, 32), (33000, 33, 16), (17000, 520, 16)])
def test_conv_runs(T, C, run, W, io):
    assert _run(T, _up(C, 512)) == run and _run(T, _up(C, 256)) == run
    g = torch.Generator().manual_seed(T + W)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lens = [T // 3, 0, 1, 5, T // 7, 31]
    lens.append(T - sum(lens))
    n, starts = len(lens), _starts(lens)
    x, dy = rnd(T, C).to(io).cuda(), rnd(T, C).to(io).cuda()
    w, b, pool = (rnd(C, W) / 2).cuda(), rnd(C).cuda(), rnd(n, W - 1, C).to(io).cuda()
    cu, u = torch.tensor(starts, dtype=torch.int32).cuda(), HALF[io]
    p = [_np(v) for v in (x, w, b, pool, dy)]
    want, last, _ = Q.conv_forward(*p[:3], starts, p[3])
    mag = Q.conv_forward(*[abs(v) for v in p[:3]], starts, abs(p[3]), False)[0]
    final = pool.clone()
    y = R.causal_conv_forward(x, w, bias=b, cu_seqlens=cu, initial_state=final, final_state=final)
    _near(y, want, u * abs(want) + E32 * mag, "y")
    assert np.array_equal(_np(final), last)
    got = R.causal_conv_backward(dy, x, w, bias=b, cu_seqlens=cu, initial_state=pool)
    want = Q.conv_backward(p[4], *p[:3], starts, p[3])
    m = Q.conv_backward(p[4], *p[:3], starts, p[3], magnitude=True)
    more = 1.0 + float(mag.max())
    _near(got["dx"], want["dx"], u * abs(want["dx"]) + E32 * m["dx"] * more, "dx")
    for k in ("dweight", "dbias"):
        _near(got[k], want[k], E32 * m[k] * more, k)
    _near(got["dinitial_state"], want["dinit"], u * abs(want["dinit"]) + E32 * m["dinit"] * more, "dinit")


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("nb, C", [(4099, 40), (4097, 33), (2050, 520), (4095, 40)])
def test_conv_step_of_many_rows(nb, C, W, io):
    """From 4096 waves' worth of rows on a wave takes four; the last takes the rest."""
    assert (nb * _up(C, 512) >= 4096) == (nb != 4095) and nb % 4
    g = torch.Generator().manual_seed(nb + W)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w, b = rnd(nb, C).to(io).cuda(), rnd(C, W).cuda(), rnd(C).cuda()
    pool, slot = rnd(nb + 5, W - 1, C).to(io).cuda(), torch.randperm(nb + 5, generator=g)[:nb].to(torch.int32)
    bad = torch.tensor([0, 6, nb - 2, nb - 1])
    slot[bad] = torch.tensor([-1, nb + 5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    ok = torch.ones(nb, dtype=torch.bool)
    ok[bad] = False
    status, old = torch.zeros(1, dtype=torch.int32, device="cuda"), pool.clone()
    y = R.causal_conv_decode(x, pool, w, bias=b, slot_idx=slot.cuda(), status=status)
    assert int(status) == R.ST_BAD_SLOT
    assert y[bad.cuda()].isnan().all()
    at = slot[ok].long().cuda()
    win = torch.cat([old[at], x[ok.cuda()][:, None]], 1)              # [rows, W, C]
    v = (_np(win) * _np(w).T[None]).sum(1) + _np(b)
    mag = (abs(_np(win)) * abs(_np(w)).T[None]).sum(1) + abs(_np(b))
    want = v * Q.sigmoid(v)
    _near(y[ok.cuda()], want, HALF[io] * abs(want) + E32 * mag, "y")
    assert torch.equal(pool[at], win[:, 1:])
    rest = torch.ones(nb + 5, dtype=torch.bool)
    rest[at.cpu()] = False
    assert torch.equal(pool[rest.cuda()], old[rest.cuda()])           # no other slot is written


# ------------------------------------------------------------------- the norm

# rows, dim, group, threads and vectors a lane forward and backward
NORMS = [(2100, 40, 40, (64, 1), (64, 1)), (2100, 1000, 500, (64, 2), (64, 2)), (1100, 1500, 1500, (256, 1), (256, 1)),
         (1030, 2560, 2560, (256, 2), (256, 2)), (1030, 2560, 640, (256, 2), (256, 2)),
         (1027, 3001, 3001, (256, 2), (256, 2)), (600, 5120, 5120, (256, 4), (512, 2)),
         (520, 8192, 1024, (256, 4), (512, 2)), (300, 10001, 10001, (1024, 2), (1024, 2)),
         (260, 20000, 5000, (1024, 4), (1024, 4))]


def _shape(nvec, rows, backward):
    if not backward and rows <= 256 and 256 < nvec <= 1024:
        return (1024, 1)
    for most, sh in ((64, (64, 1)), (128, (64, 2)), (256, (256, 1)), (512, (256, 2)),
                     (1024, (512, 2) if backward else (256, 4)), (2048, (1024, 2))):
        if nvec <= most:
            return sh
    return (1024, 4)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("case", NORMS, ids=lambda c: "{}x{}g{}".format(*c))
def test_norm_of_many_rows(case, gate, io):
    """More rows than the backward has workgroups: each takes several."""
    rows, dim, group, fwd, bwd = case
    nvec = dim // group * _up(group, 8)
    assert _shape(nvec, rows, False) == fwd and _shape(nvec, rows, True) == bwd
    assert rows > min(2048, 256 * 1024 // bwd[0])
    g = torch.Generator().manual_seed(dim + rows)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, dy = rnd(rows, dim).to(io).cuda(), rnd(rows, dim).to(io).cuda()
    z = rnd(rows, dim).to(io).cuda() if gate else None
    w, r = (1.0 + 0.2 * rnd(dim)).cuda(), (3.0 * rnd(rows, dim)).cuda()
    u, nz = HALF[io], None if z is None else _np(z)
    got = R.rms_norm_forward(x, w, z=z, residual=r, group_size=group)
    h = _np(x) + _np(r)
    _near(got["residual"], h, 2.0 ** -24 * abs(h), "residual")
    want = Q.norm_forward(_np(got["residual"]), _np(w), nz, group, 1e-5)
    _near(got["out"], want, u * abs(want) + E32 * abs(want), "out")
    got = R.rms_norm_backward(dy, x, w, z=z, group_size=group)
    want, mag = Q.norm_backward(_np(dy), _np(x), _np(w), nz, group, 1e-5)
    for k in want:
        half = 0.0 if k == "dweight" else u
        more = 8.0 if k == "dz" else 1.0
        extra = 2.0 ** -20 * np.abs(_np(dy)).max() * np.abs(_np(x)).max() * 8 if k == "dz" else 0.0
        _near(got[k], want[k], half * abs(want[k]) + E32 * mag[k] * more + extra, k)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows, dim, group", [(300, 2560, 2560), (300, 5120, 640), (257, 8192, 8192)])
def test_norm_8bit_of_many_rows(rows, dim, group, block, io):
    g = torch.Generator().manual_seed(dim)
    x, w = torch.randn(rows, dim, generator=g).to(io).cuda(), torch.randn(dim, generator=g).cuda()
    got = R.rms_norm_forward(x, w, group_size=group, out_dtype=torch.float8_e4m3fn, scale_block=block)
    want = Q.norm_forward(_np(x), _np(w), None, group, 1e-5)
    b = block or dim
    scale = abs(want).reshape(rows, -1, b).max(-1) / 448.0
    _near(got["scale"], scale, E32 * scale, "scale")
    q = want / np.repeat(scale, b, 1)
    _near(got["out"].float(), q, abs(q) * (2.0 ** -4 + 2.0 ** -14) + 2.0 ** -10 * (1 + 2.0 ** -8), "out")
