"""What the launching code keeps between calls (shared memory limits, answers of the
runtime), against a runtime whose calls fail when told to.  Host code only: compiled
here with nvcc, linked without the CUDA runtime."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_launch_state(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("needs nvcc")
    exe = str(tmp_path / "launch_state")
    subprocess.run([nvcc, "-std=c++17", "-x", "c++", "-cudart", "none", "-o", exe,
                    os.path.join(HERE, "native", "launch_state.cu")], check=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout + run.stderr
