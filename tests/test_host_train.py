"""Host-side checks of the channels-last training kernels' planners (no GPU).

Each program under tests/host/ includes the planner's own file and replays its
arithmetic; it prints its failures and exits non-zero on any:
  * check_nhwc_bwd.cu: the layer backward's workspace holds the sums and the
    aligned copies of a call from any source (the input, its codes), over
    images of up to 70000 rows; rows whose scales lie 2^32 bytes apart are
    left to the kernel that steps over them in 64 bits; the aligned copies
    bring every byte of a pixel and read none outside the tensor; a lane of
    the generic filter gradient adds up at most 1024 pixels;
  * check_norm.cu: the group norm's threads add up at most 4096 rows each as
    long as the kernels take more chunks, and every family's sums lie inside
    the workspace and the shared memory.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "depthwise_convolution_dwconv2d_gb300", "csrc")


@pytest.mark.parametrize("name", ["check_nhwc_bwd", "check_norm"])
def test_planner(tmp_path, name):
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / name)
    r = subprocess.run([nvcc, "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "host", name + ".cu"),
                        "-o", exe], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    tail = r.stdout.strip().splitlines()[-1] if r.stdout.strip() else ""
    assert r.returncode == 0 and "fails: 0" in tail, "\n".join(r.stdout.splitlines()[-20:])
