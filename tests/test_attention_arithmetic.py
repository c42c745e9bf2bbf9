"""The paged attention's quotients and shares, on the CPU: the same functions
run in the kernels."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not installed")
def test_quotients_and_shares(tmp_path):
    exe = str(tmp_path / "attention_arithmetic_check")
    r = subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-x", "cu",
                        "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "gated_deltanet_linear_chunk_gb300", "csrc"),
                        "-I", os.path.join(ROOT, "include"),
                        os.path.join(HERE, "csrc", "attention_arithmetic_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    quotients, tiles = map(int, r.stdout.split())
    assert quotients > 1000000 and tiles > 500000
