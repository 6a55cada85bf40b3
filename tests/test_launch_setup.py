"""What launches look up once (no GPU): csrc/launch_setup.h compiled against a runtime
made for the test (tests/launch_setup.cpp)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_matrix_multiply_gb300", "csrc")


def test_launch_setup(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if shutil.which("g++") is None or not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("g++ and CUDA's headers")
    exe = tmp_path / "launch_setup"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", include, "-I", CSRC,
                        os.path.join(ROOT, "tests", "launch_setup.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
