"""Every launch of the linear and gated calls stays within what a launch can hold, over
the whole range of sizes that the checks accept (CPU; with address and
undefined-behaviour checks where the compiler has them)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_launches_hold_every_valid_size(tmp_path):
    exe = str(tmp_path / "driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "linear_launch_driver.cpp"),
           *(os.path.join(CSRC, f) for f in ("linear_plan.cpp", "conv_plan.cpp")), "-o", exe]
    checks = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    built = subprocess.run(cmd + checks, capture_output=True, text=True)
    if built.returncode and "cannot find -l" in built.stderr:
        built = subprocess.run(cmd, capture_output=True, text=True)
    assert built.returncode == 0, built.stderr[-2000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout[-500:] + run.stderr[-2000:]
