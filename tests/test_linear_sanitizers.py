"""The linear, gated and clipping planners under address and undefined-behaviour
checks, on the CPU, over random problems of the whole range of sizes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_planners_under_sanitizers(tmp_path):
    exe = str(tmp_path / "driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "linear_sanitize_driver.cpp"),
           *(os.path.join(CSRC, f) for f in ("linear_plan.cpp", "grad_clip_plan.cpp", "conv_plan.cpp")),
           "-o", exe]
    built = subprocess.run(cmd, capture_output=True, text=True)
    if built.returncode and "cannot find -l" in built.stderr:
        pytest.skip("no sanitizer runtime")
    assert built.returncode == 0, built.stderr[-2000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout[-500:] + run.stderr[-2000:]
