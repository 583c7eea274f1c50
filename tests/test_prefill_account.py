"""The account of copies under way of the prefill's copy warps, with copies that land as late as the waits
allow: compiles tests/prefill_account_check.cu with nvcc and runs it (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_tiles_are_announced_once_they_are_there(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "prefill_account_check")
    subprocess.run([nvcc, "-O2", "-std=c++17", "-o", exe,
                    os.path.join(HERE, "prefill_account_check.cu")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    assert r.stdout.rstrip().endswith("bad 0")
