"""Host-side logic of the paged cache's kernels, compiled with nvcc as host programs (no GPU needed)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["paged_parts_check"])
def test_host_program(name, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / name)
    build = subprocess.run([nvcc, "-std=c++17", "-O1", "-Wno-deprecated-gpu-targets",
                            "-I", os.path.join(ROOT, "exact_io_aware_91_b200", "csrc"),
                            "-I", os.path.join(ROOT, "include"),
                            os.path.join(ROOT, "tests", "host", name + ".cu"), "-o", exe],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert run.stdout.startswith("ok ")
