"""A CTA of the forward that gives up takes over those that have not started, so that a call whose waits
run out ends after one wait's limit (compiles and runs tests/clc_drop_check.cu)."""
import os
import shutil
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "attention_backward_flashattention_gb300", "csrc")


def test_no_cta_starts_behind_one_that_gives_up(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / "clc_drop_check")
    subprocess.run([nvcc, "-O2", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-o", exe,
                    os.path.join(HERE, "clc_drop_check.cu")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    rows = [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    assert len(rows) == 16
    for mode, grid, sms, started in rows:
        # (without taking over, all of them start)
        assert started == grid if mode == 0 else 1 <= started <= min(grid, sms), (mode, grid, started)


def test_the_forward_takes_the_rest_over():
    text = open(os.path.join(CSRC, "attn_fwd.cu")).read()
    give_up = text[text.index("      if (!ok) {"):]
    assert "clc_drop_rest(answer, clc, asked, sh.n_items);" in give_up[:200]
