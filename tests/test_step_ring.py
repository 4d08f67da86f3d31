"""A ring of steps as a warp of the attention over 4-bit pages walks it, on the host: after a wait that ran
out, the copies that are still on their way are the ones that are waited for."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_late_steps_are_drained(tmp_path):
    exe = tmp_path / "step_ring_model"
    build = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror",
                            "-I", os.path.join(ROOT, "prefill_only_cascade_gb300", "csrc"),
                            os.path.join(ROOT, "tests", "c", "step_ring_model.cpp"), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
