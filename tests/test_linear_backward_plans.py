"""CPU tests of the plans of the linear and gated gradients (include/linear.h)."""
import os
import shutil
import subprocess

import pytest

import convolution_forward_amd as cf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_a_product_of_a_pair_alone(tmp_path):
    exe = str(tmp_path / "driver")
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                           os.path.join(ROOT, "tests", "linear_pair_driver.cpp"),
                           *(os.path.join(CSRC, f) for f in ("linear_plan.cpp", "conv_plan.cpp")), "-o", exe])
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,name", [
    (2048, 2048, 1024, "dx.tile64x64.dw.tile64x64.both"), (2000, 2056, 1000, "both.tile256x128"),
    (4096, 4096, 2048, "both.tile256x256"), (4000, 1992, 1992, "both.tile256x128"),
    (2001, 2003, 1031, "both.tile256x128.pack"),
    (520, 1032, 72, "dx.tile64x64.split6.dw.tile64x64.split3.both"),
    (1001, 65, 2000, "dx.tile64x64.dw.tile64x64.split8.both.pack")])
def test_linear_gradients(m, n, k, name, dtype):
    for layout in ("nk", "kn"):
        p = cf.make_linear_problem(m, n, k, w_layout=layout)
        assert cf.linear_backward_describe_variant(p, dtype) == f"linear_backward.{dtype}.{name}"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,f,k,name", [
    (2048, 1408, 1024, "both.tile256x128"), (2000, 1401, 1000, "both.tile256x128"),
    (1501, 1003, 1031, "dx.tile64x64.dw.tile64x64.both.pack"), (4096, 5632, 2048, "both.tile256x256")])
def test_gated_gradients(m, f, k, name, dtype):
    p = cf.make_gated_problem(m, f, k)
    assert cf.gated_backward_describe_variant(p, dtype) == f"gated_backward.{dtype}.{name}"
