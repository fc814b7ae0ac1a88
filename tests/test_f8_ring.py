"""The load producer of the 8-bit product (csrc/f8_ring.h), compiled for the host and run against a model of its barriers
(f8_ring_check.cc): blocks and stages in order, and, where any one wait runs out, every stage's last load and no phase
that cannot complete waited for."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "compressed_sparse_attention_09_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_ring_fills_and_their_drain(tmp_path):
    exe = str(tmp_path / "ring")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wno-unknown-pragmas", "-I", CSRC, "-o", exe, os.path.join(HERE, "f8_ring_check.cc")],
                   check=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
