"""The block operators' copies of single 16-bit elements read nothing outside
their tensors, on the CPU: the same function places the kernels' copies."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not installed")
def test_element_reads_stay_inside_their_tensor(tmp_path):
    exe = str(tmp_path / "element_word_check")
    r = subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-x", "cu",
                        "-I", os.path.join(ROOT, "gated_deltanet_linear_chunk_gb300", "csrc"),
                        "-I", os.path.join(ROOT, "include"),
                        os.path.join(HERE, "csrc", "element_word_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) == 8 * 24 * 25 // 2
