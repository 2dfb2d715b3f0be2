"""The entry points around a block's layers on the host: which kernel a call maps to on both sides of each bound."""
import os
import shutil
import subprocess

import pytest

from block_pairs import PAIRS
from depthwise_convolution_dwconv2d_gb300 import binding as B
from depthwise_convolution_dwconv2d_gb300 import build as BLD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "depthwise_convolution_dwconv2d_gb300", "csrc")


@pytest.fixture(scope="module", autouse=True)
def lib():
    BLD.build()
    return B.load()


def plans(C, dtype, rows=5, **kw):
    d = B.make_rms_desc(rows, C, dtype=dtype, **kw)
    return tuple(B.dwconv_rms_norm_plan_name(d, k) for k in (0, 1))


@pytest.mark.parametrize("dtype,V", [("bf16", 8), ("f16", 8), ("f32", 4)])
def test_rms_plans_on_both_sides_of_each_bound(dtype, V):
    """Forward: 2048 vectors of 16 bytes to a row, or 8192 elements where its tensors do not begin alike. Backward: 8192
    channels; never without rows that begin alike."""
    for rows in (1, 5, 100_000):
        assert plans(2048 * V, dtype, rows)[0] == "row" and plans(2049 * V, dtype, rows)[0] == "wide"
        assert plans(8192, dtype, rows)[1] == "row" and plans(8192 + V, dtype, rows)[1] == "wide"
        # off 16 bytes a row may reach over V - 1 elements in front of it
        assert plans(2047 * V + 1, dtype, rows)[0] == "row" and plans(2048 * V + 1, dtype, rows)[0] == "wide"
        assert plans(8192 - V + 1, dtype, rows)[1] == "row" and plans(8193, dtype, rows)[1] == "wide"
        # x and y do not begin alike: slices of other widths, other offsets
        for kw in (dict(x_c_total=20_001, y_c_total=20_000), dict(x_c_offset=1, x_c_total=20_000, y_c_total=20_000)):
            assert plans(8192, dtype, rows, **kw) == ("row", "wide")
            assert plans(8193, dtype, rows, **kw) == plans(8200, dtype, rows, **kw) == ("wide", "wide")
            assert plans(64, dtype, rows, **kw) == ("row", "wide")
    # off 16 bytes but alike
    kw = dict(x_c_offset=3, x_c_total=20_001, y_c_offset=3, y_c_total=20_001)
    assert plans(8000, dtype, **kw) == ("row", "row")


def test_rms_plan_of_a_wider_slice():
    """12000 channels of rows 12001 apart into rows of their own: no kernel holds such a row."""
    assert plans(12000, "bf16", x_c_total=12001) == ("wide", "wide")
    assert plans(12000, "bf16", x_c_total=12001, y_c_total=12001) == ("row", "wide")


def test_weights_too_small_for_their_sizes_are_refused():
    """Kernels write and read whole rows of 128 codes: rows of cin codes, the natural shape, end before those do."""
    torch = pytest.importorskip("torch")
    codes = lambda *s, t=torch.float8_e4m3fn: torch.empty(*s, dtype=t)  # noqa: E731
    scales = torch.empty(2, 3)
    for good in (codes(200, 384), codes(200, 384, t=torch.uint8), codes(200 * 384 + 5), codes(1, 200, 384)):
        w8 = B.make_weight8(200, 300, good, scales)
        assert w8.codes == good.data_ptr() and w8.scales == scales.data_ptr() and w8.tensors[0] is good
    for bad in (codes(200, 300), codes(199, 384), codes(200 * 384 - 1), codes(200, 512), codes(384, 200), codes(200, 384, t=torch.bfloat16)):
        with pytest.raises(ValueError, match="codes"):
            B.make_weight8(200, 300, bad, scales)
    for bad in (torch.empty(2, 2), torch.empty(5), torch.empty(2, 3, dtype=torch.float64), torch.empty(2, 3, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="scales"):
            B.make_weight8(200, 300, codes(200, 384), bad)
    B.make_weight8(200, 300, 0x1000, 0x2000)  # addresses: nothing to look at
    B.make_weight8(200, 300, codes(200, 384), torch.empty(3, 3))


def test_products_that_pairs_take(tmp_path):
    """The GPU tests' products by pairs of thread blocks are that (the plan's name does not tell them from tiles)."""
    nvcc = shutil.which("nvcc") or ("/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "check_pointwise8")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "host", "check_pointwise8.cu"),
                        os.path.join(CSRC, "tma.cu"), "-o", exe, "-lcuda"], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe] + [str(n) for c in PAIRS for n in c[:3]], capture_output=True, text=True, timeout=60)
    got = [line.split() for line in r.stdout.splitlines()]
    assert got == [["pair", str(c[5]), str(-(-c[1] // 128))] for c in PAIRS]
    assert any(c[5] > 1 and -(-c[1] // 128) % 2 for c in PAIRS) and any(c[5] > 1 and -(-c[1] // 128) % 2 == 0 for c in PAIRS)
    assert all(B.dwconv2d_pointwise8_plan_name(*c[:3]) == "tile" for c in PAIRS)
