"""Index arithmetic of the paged cache and of the decode's work split against
brute force, on the host: compiles tests/paged_index_check.cu with nvcc and runs
it (no GPU needed)."""
import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_paged_index_arithmetic():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "paged_index_check")
        subprocess.run([nvcc, "-O2", "-std=c++17", "-o", exe,
                        os.path.join(HERE, "paged_index_check.cu")], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    assert r.stdout.rstrip().endswith("bad 0")


def test_prefill_work_split():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "prefill_index_check")
        subprocess.run([nvcc, "-O2", "-std=c++17", "-o", exe,
                        os.path.join(HERE, "prefill_index_check.cu")], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    assert r.stdout.rstrip().endswith("bad 0")
