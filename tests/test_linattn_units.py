"""The cut into units of the linear attention, compiled for the host with g++: no run adds up summaries
that its workspace does not hold, whatever the offsets in device memory say."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gated_delta_rule_82_b200", "csrc")


def test_runs_add_up_only_what_the_workspace_holds(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "linattn_units_check")
    subprocess.run([gxx, "-O2", "-std=c++17", "-I", CSRC, os.path.join(HERE, "linattn_units_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "bad 0" in r.stdout, r.stdout + r.stderr
