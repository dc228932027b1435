"""The order of the waits by which a stage of the policy loss's ring changes
hands, against a model of its barrier (ring_model.cpp), on the CPU."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "second_order_optimisation_gb300", "csrc")


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
def test_every_order_of_a_stages_events(tmp_path):
    exe = str(tmp_path / "ring_model")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, os.path.join(HERE, "ring_model.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
