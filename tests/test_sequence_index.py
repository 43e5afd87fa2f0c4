"""The sequence kernels' index arithmetic, compiled for the host: every token,
workspace place and LDS element that it gives, against what it is an index of."""

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_index_is_inside_its_buffer(tmp_path):
    exe = str(tmp_path / "check")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-ftrapv",
                        os.path.join(HERE, "seq_index_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
