"""What the linear-attention operators refuse, and what they do not, at the ends of
their ranges: on the host, before any HIP call."""

import pytest

import linear_recurrence_amd as R
from test_mixer_refusals import EINVAL, ESHAPE, NAMES, OK, SEQ, V, _mix, _rot


@pytest.fixture(scope="module")
def lib():
    return R.load()


def test_a_heads_decay_always_has_a_gradient(lib):
    """Its shape has no token in it: it is written for an empty batch too."""
    for seqs in (0, 2):
        assert _mix(lib, "linear_attention_backward", decay=1, tokens=0, seqs=seqs, gg=None) == EINVAL
    assert _mix(lib, "linear_attention_backward", decay=2, tokens=0, seqs=0, gg=None) == OK


@pytest.mark.parametrize("fn", SEQ)
def test_launches_of_2_32_threads_are_refused(lib, fn):
    """Where only one kind of launch would be too large, and where the number of
    segment slots passes 32 bits."""
    for dims in (dict(tokens=8, seqs=1 << 23), dict(tokens=8, seqs=1 << 22, dk=64 if "linear" in fn else 128, dv=128),
                 dict(tokens=4096, seqs=(1 << 31) - 1), dict(tokens=(1 << 31) - 1, seqs=(1 << 31) - 1),
                 dict(tokens=(1 << 31) - 1, k_heads=256, v_heads=1 << 20), dict(tokens=8, v_heads=1 << 20, seqs=1 << 6)):
        assert _mix(lib, fn, **dims, ws=1 << 62) == ESHAPE, dims


@pytest.mark.parametrize("fn", ["rotary_forward", "rotary_backward"])
@pytest.mark.parametrize("heads", [(1 << 30) + 1, (1 << 31) - 1])
def test_rotary_heads_are_counted_in_32_bits(lib, fn, heads):
    """A thread steps past the last of them: past 2^31 it would begin at -2^31 again."""
    assert _rot(lib, fn, y=V(1 << 50), tokens=1, heads=heads, dim=2, rotary_dim=2) == ESHAPE


FAR = {n: V((i + 2) << 40) for i, n in enumerate(
    "q k v do g beta cu has slot init final state new o gq gk gv gg gbeta dfinal dinit ws".split())}


@pytest.mark.parametrize("fn", list(NAMES))
def test_results_over_inputs_are_refused(lib, fn):
    """Only refused calls: the pointers are made up.  8 tokens of bf16, 2 key and 4 value
    heads of 64: rows of 256 and 512 bytes."""
    names, back = NAMES[fn].split(), "backward" in fn

    def call(out, over, at, **dims):
        base = FAR[over].value
        return _mix(lib, fn, **{**{n: FAR[n] for n in names if n != "ws"}, **dims, out: V(base + at)})
    for out, row in (("gq", 256), ("gk", 256), ("gv", 512)) if back else (("o", 512),):
        for over, width in (("q", 256), ("k", 256), ("v", 512)) + ((("do", 512),) if back else ()):
            for at in (0, 16, 8 * width - 16, 16 - 8 * row):
                if (out, over, at) == ("o", "v", 0):
                    continue   # in place
                assert call(out, over, at) == EINVAL, (out, over, at)
            if over == "do":
                continue
            # rows of wider ones: over the last, and up to the second
            for at in (7 * 2048 + width - 16, 2048 - 8 * row + 16):
                assert call(out, over, at, **{over + "_stride": 1024}) == EINVAL, (out, over, at)
    pool = 4 * 64 * 64 * 4   # bytes of a slot: two of them
    pairs = dict(linear_attention_decode=("new", "state")).get(fn, ("dinit", "init") if back else ("final", "init"))
    for at in (16, 2 * pool - 16, 16 - 2 * pool) + ((0,) if back else ()):
        assert call(*pairs, at) == EINVAL, at
