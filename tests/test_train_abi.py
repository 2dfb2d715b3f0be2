"""The channels-last training entry points on the host: struct layouts and refusals (nothing is enqueued)."""
import ctypes

import pytest

from depthwise_convolution_dwconv2d_gb300 import binding as B
from depthwise_convolution_dwconv2d_gb300 import build as BLD

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4
P = 0x10000  # a well-aligned fake address: validation fails before any use
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    BLD.build()
    return B.load()


def status_of(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except B.DwconvError as e:
        return e.status
    return 0


def act8(rows=16, C=40, kind="i8", block=32, codes=P, scales=P):
    return B.make_act8(kind, block, codes, scales, rows, C)


def norm(**kw):
    return B.make_norm_desc(**{**dict(N=2, H=4, W=4, C=40, groups=4, act="silu", dtype="bf16"), **kw})


def test_layouts():
    assert ctypes.sizeof(B.Act8) == 40 and B.Act8.codes.offset == 24
    assert ctypes.sizeof(B.NormDesc) == 80 and B.NormDesc.eps.offset == 44 and B.NormDesc.x_c_offset.offset == 48


@pytest.mark.parametrize("t,total,dtype,want", [
    (act8(rows=-1), 0, "bf16", INVALID), (act8(C=0), 0, "bf16", INVALID), (act8(kind=2), 0, "bf16", UNSUPPORTED),
    (act8(kind=-1), 0, "bf16", UNSUPPORTED), (act8(block=0), 0, "bf16", INVALID), (act8(block=48), 0, "bf16", UNSUPPORTED),
    (act8(block=256), 0, "bf16", UNSUPPORTED), (act8(), 39, "bf16", INVALID), (act8(), -1, "bf16", INVALID),
    (act8(), 0, 3, UNSUPPORTED), (act8(codes=None), 0, "bf16", INVALID), (act8(scales=None), 0, "bf16", INVALID),
    (act8(scales=P + 2), 0, "bf16", MISALIGNED), (act8(rows=1 << 45), 0, "bf16", UNSUPPORTED), (None, 0, "bf16", INVALID),
    (act8(rows=1, C=(1 << 20) + 1), 0, "f32", UNSUPPORTED)])
def test_act8_refusals(t, total, dtype, want):
    assert status_of(B.dwconv_act8_encode, P, t, total, dtype, 0) == want
    assert status_of(B.dwconv_act8_decode, t, P, total, dtype, 0) == want


def test_act8_pointers():
    assert status_of(B.dwconv_act8_encode, None, act8(), 0, "bf16", 0) == INVALID
    assert status_of(B.dwconv_act8_decode, act8(), P + 1, 0, "f16", 0) == MISALIGNED
    assert status_of(B.dwconv_act8_encode, P + 2, act8(), 0, "f32", 0) == MISALIGNED
    empty = act8(rows=0, codes=None, scales=None)
    assert status_of(B.dwconv_act8_encode, None, empty, 0, "bf16", 0) == 0
    assert status_of(B.dwconv_act8_decode, empty, None, 0, "bf16", 0) == 0


@pytest.mark.parametrize("d,want", [
    (norm(N=-1), INVALID), (norm(H=0), INVALID), (norm(W=0), INVALID), (norm(C=0), INVALID), (norm(groups=0), INVALID),
    (norm(groups=3), INVALID), (norm(groups=80), INVALID), (norm(act=5), INVALID), (norm(act=-1), INVALID),
    (norm(eps=-1e-5), INVALID), (norm(eps=float("nan")), INVALID), (norm(eps=float("inf")), INVALID),
    (norm(dtype=3), UNSUPPORTED), (norm(x_c_offset=1), INVALID), (norm(x_c_total=39), INVALID),
    (norm(y_c_offset=8, y_c_total=47), INVALID), (norm(y_c_offset=-1, y_c_total=64), INVALID), (norm(x_c_total=-8), INVALID),
    (norm(C=1 << 21, groups=1), UNSUPPORTED), (norm(H=1 << 30, W=1 << 30), UNSUPPORTED), (norm(N=1 << 40), UNSUPPORTED),
    (norm(x_c_offset=1 << 62, x_c_total=1 << 62), INVALID), (norm(x_c_total=1 << 62), UNSUPPORTED)])
def test_norm_descriptors(d, want):
    assert status_of(B.dwconv2d_group_norm_nhwc, d, P, P, P, P, P, P, P, BIG, stream=0) == want
    assert status_of(B.dwconv2d_group_norm_nhwc_bwd, d, P, P, P, P, P, P, P, P, P, P, BIG, stream=0) == want
    for p in (0, 1):
        assert B.dwconv2d_group_norm_nhwc_workspace_size(d, p) == 0
        assert B.dwconv2d_group_norm_nhwc_plan_name(d, p) == "invalid"


def test_norm_arguments():
    d, f, b = norm(), B.dwconv2d_group_norm_nhwc, B.dwconv2d_group_norm_nhwc_bwd
    assert B.dwconv2d_group_norm_nhwc_workspace_size(d, 2) == 0 and B.dwconv2d_group_norm_nhwc_plan_name(d, -1) == "invalid"
    need = [B.dwconv2d_group_norm_nhwc_workspace_size(d, p) for p in (0, 1)]
    assert status_of(f, d, None, P, P, P, P, P, P, BIG, stream=0) == INVALID
    assert status_of(f, d, P, P, P, None, P, P, P, BIG, stream=0) == INVALID
    assert status_of(f, d, P + 1, P, P, P, P, P, P, BIG, stream=0) == MISALIGNED
    assert status_of(f, d, P, P + 1, P, P, P, P, P, BIG, stream=0) == MISALIGNED
    assert status_of(f, d, P, P, P, P, P + 2, P, P, BIG, stream=0) == MISALIGNED
    if need[0]:
        assert status_of(f, d, P, P, P, P, P, P, None, 0, stream=0) == WORKSPACE
        assert status_of(f, d, P, P, P, P, P, P, P, need[0] - 1, stream=0) == WORKSPACE
        assert status_of(f, d, P, P, P, P, P, P, P + 8, BIG, stream=0) == MISALIGNED
    # a checkpoint of other rows or channels, or of no kind
    for t in (act8(rows=31), act8(rows=32, C=41), act8(rows=32, block=31)):
        assert status_of(f, d, P, P, P, P, P, P, P, BIG, t, 0) in (INVALID, UNSUPPORTED)
        assert status_of(b, d, None, P, P, P, P, P, P, P, P, P, BIG, t, 0) in (INVALID, UNSUPPORTED)
    t = act8(rows=32)
    assert status_of(b, d, P, P, P, P, P, P, P, P, P, P, BIG, t, 0) == INVALID       # x and x8
    assert status_of(b, d, None, P, P, P, P, P, P, P, P, P, BIG, None, 0) == INVALID  # neither
    assert status_of(b, d, P, None, P, P, P, P, P, P, P, P, BIG, None, 0) == INVALID
    assert status_of(b, d, P, P, P, P, None, P, P, P, P, P, BIG, None, 0) == INVALID
    assert status_of(b, d, P, P, P, P, P, None, P, P, P, P, BIG, None, 0) == INVALID
    assert status_of(b, d, P, P, P, P, P, P, P + 1, P, P, P, BIG, None, 0) == MISALIGNED
    assert status_of(b, d, P, P, P, P, P, P, P, P, P, P, need[1] - 1, None, 0) == WORKSPACE
    assert status_of(b, d, P, P, P, P, P, P, None, None, None, None, 0, None, 0) == 0  # nothing asked for


def test_epilogue_keeps_to_its_own_activations():
    d = B.make_desc(2, 3, 8, 8, 3, 1, 1)
    for a in ("silu", "gelu"):
        assert status_of(B.dwconv2d_fwd_epilogue, d, P, P, None, None, None, a, P, 0) == INVALID
        assert status_of(B.dwconv2d_fwd_nhwc, d, P, P, None, P, None, None, a, 0) == INVALID


def test_conv_backward_refusals():
    f = B.dwconv2d_bwd_nhwc
    d = B.make_desc(2, 40, 4, 4, 3, 1, 1, dtype="bf16")
    for bad, want in ((B.make_desc(2, 0, 4, 4), INVALID), (B.make_desc(2, 4, 4, 4, dtype=9), UNSUPPORTED),
                      (B.make_desc(1, 3, 2, 2, 5, 1, 0), INVALID)):
        assert status_of(f, bad, P, P, P, P, P, P, P, BIG, stream=0) == want
        assert B.dwconv2d_bwd_nhwc_workspace_size(bad) == 0 and B.dwconv2d_bwd_nhwc_plan_name(bad) == "invalid"
    need = B.dwconv2d_bwd_nhwc_workspace_size(d)
    assert need > 0
    assert status_of(f, d, P, P, P, P, P, P, P, need - 1, stream=0) == WORKSPACE
    assert status_of(f, d, P, P, P, P, P, P, None, 0, stream=0) == WORKSPACE
    assert status_of(f, d, P, P, P, P, P, P, P + 8, BIG, stream=0) == MISALIGNED
    assert status_of(f, d, P, P, None, P, P, P, P, BIG, stream=0) == INVALID       # gx without w
    assert status_of(f, d, P, None, P, P, P, P, P, BIG, stream=0) == INVALID
    assert status_of(f, d, None, P, P, P, P, P, P, BIG, stream=0) == INVALID       # gw without an input
    assert status_of(f, d, P, P, P, P, P, P, P, BIG, act8(rows=32), stream=0) == INVALID
    assert status_of(f, d, None, P, P, P, P, P, P, BIG, act8(rows=30), stream=0) == INVALID
    assert status_of(f, d, P, P, P, P, P, P, P, BIG, None, 2, 0) == INVALID         # accumulate
    assert status_of(f, d, P, P + 1, P, P, P, P, P, BIG, stream=0) == MISALIGNED
    assert status_of(f, d, P, P, P, P, P + 1, P, P, BIG, stream=0) == MISALIGNED
    assert status_of(f, d, None, P, None, None, None, None, None, 0, stream=0) == 0  # nothing asked for


def test_plan_names():
    """Slabs that a cluster holds, slabs that it does not, and slices wider than a thread block."""
    name = B.dwconv2d_group_norm_nhwc_plan_name
    assert [name(norm(N=64, H=56, W=56, C=128, groups=32), p) for p in (0, 1)] == ["slab", "slab"]
    assert [name(norm(N=2, H=256, W=256, C=64, groups=8, dtype="f32"), p) for p in (0, 1)] == ["stream", "stream"]
    assert [name(norm(N=1, H=9, W=9, C=4110, groups=1), p) for p in (0, 1)] == ["split", "split"]
    assert name(norm(N=0), 0) in ("slab", "stream", "split")
    conv = B.dwconv2d_bwd_nhwc_plan_name
    for k, s, pad in ((3, 1, 1), (3, 2, 0), (5, 1, 2), (7, 2, 3)):
        assert conv(B.make_desc(2, 40, 20, 20, k, s, pad)) == "nhwc"
    for kw in (dict(kernel=4, pad=1), dict(kernel=3, pad=2), dict(kernel=3, pad=2, dilation=2), dict(kernel=3, pad=1, stride=3),
               dict(kernel=3, pad=1, multiplier=2), dict(kernel=(3, 5), pad=(1, 2))):
        assert conv(B.make_desc(2, 40, 20, 20, **kw)) == "generic"


def test_workspaces_cover_aligned_copies():
    """Channels that are no multiple of 16 bytes: room for gy and x (or its codes) on aligned pixels beside the sums."""
    size = B.dwconv2d_bwd_nhwc_workspace_size
    assert size(B.make_desc(4, 65, 20, 20, 3, 1, 1, dtype="bf16")) > 2 * 4 * 400 * 72 * 2
    # a channel slice off 16 bytes needs gy's copy alone
    a = size(B.make_desc(4, 64, 20, 20, 3, 1, 1, dtype="bf16", out_c_offset=8, out_c_total=80))
    b = size(B.make_desc(4, 64, 20, 20, 3, 1, 1, dtype="bf16", out_c_offset=3, out_c_total=80))
    assert b - a == 4 * 400 * 64 * 2
