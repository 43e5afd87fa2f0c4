"""Where segments of long sequences keep their states: the index arithmetic on the
host, and the workspaces' sizes."""

import os
import subprocess

import pytest

import linear_recurrence_amd as R
from linear_recurrence_amd import mixer as S

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_place_is_inside_its_buffer(tmp_path):
    exe = str(tmp_path / "check")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-ftrapv",
                        os.path.join(HERE, "mixer_index_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


@pytest.mark.parametrize("fn", ["linear_attention_forward", "linear_attention_backward", "gdn_scan_forward",
                                "gdn_scan_backward"])
@pytest.mark.parametrize("tokens, seqs", [(2048, 256), (16384, 256), (65536, 4096), (16384, 8), (1 << 20, 1)])
def test_short_sequences_take_no_segment(fn, tokens, seqs):
    """What a call holds beside its chunks: states and, for the delta rule, matrices of
    at most 4 tokens / 512 segments, however many sequences there are; and 4 bytes a
    segment slot."""
    HV, K, both = 32, 128, fn.endswith("backward")
    size = getattr(R.load(), fn + "_workspace")(S.MixerDims(tokens, seqs, 16, HV, K, K, seqs, 1, 2, 0.0))
    delta, chunks = fn.startswith("gdn"), tokens // 64 + seqs
    chunk = (delta * (2 if both else 1) * 6 * 64 * 48 + both * (8 * K * K + 4 + delta * 8 * 64 * K)) * HV
    state = (2 if both else 1) * 4 * K * K
    matrix = delta * (2 if both else 1) * 6 * K * K
    most = chunks * chunk + 4 * tokens / 512 * (state + matrix + 4) * HV + 4 * (tokens / 512 + seqs) + 8 * 16
    assert size <= most, (size, most)
