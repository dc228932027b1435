"""How the tiles of checkpoints' products are dealt out to the pairs of CTAs (csrc/mx_plan.h),
gone through on the CPU (mx_plan_model.cpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "second_order_optimisation_gb300", "csrc")


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
def test_every_stage_is_taken_once_and_pieces_meet(tmp_path):
    exe = str(tmp_path / "mx_plan_model")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", CSRC, os.path.join(HERE, "mx_plan_model.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
