"""The entry points around a block's layers on the host: struct layouts, refusals (nothing is enqueued), plans."""
import ctypes

import pytest

from depthwise_convolution_dwconv2d_gb300 import binding as B
from depthwise_convolution_dwconv2d_gb300 import build as BLD

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
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


def act8(rows=16, C=40, kind="e4m3", block=128, codes=P, scales=P):
    return B.make_act8(kind, block, codes, scales, rows, C)


def rms(**kw):
    return B.make_rms_desc(**{**dict(rows=16, C=40, eps=1e-6, dtype="bf16"), **kw})


def grads(*ts):
    return (B.Grad * len(ts))(*[B.Grad(*t) for t in ts])


def test_layouts():
    assert ctypes.sizeof(B.RmsDesc) == 56 and B.RmsDesc.eps.offset == 20 and B.RmsDesc.x_c_offset.offset == 24
    assert ctypes.sizeof(B.Weight8) == 32 and B.Weight8.codes.offset == 16
    assert ctypes.sizeof(B.Grad) == 32 and B.Grad.n.offset == 16 and B.Grad.dtype.offset == 24


@pytest.mark.parametrize("d,want", [
    (rms(rows=-1), INVALID), (rms(C=0), INVALID), (rms(eps=-1e-6), INVALID), (rms(eps=float("nan")), INVALID),
    (rms(eps=float("inf")), INVALID), (rms(dtype=3), UNSUPPORTED), (rms(C=(1 << 20) + 1), UNSUPPORTED),
    (rms(x_c_offset=1), INVALID), (rms(x_c_total=39), INVALID), (rms(y_c_offset=-1, y_c_total=64), INVALID),
    (rms(y_c_offset=8, y_c_total=47), INVALID), (rms(x_c_total=-8), INVALID), (rms(rows=1 << 40), UNSUPPORTED),
    (rms(x_c_total=1 << 62), UNSUPPORTED), (rms(x_c_offset=1 << 62, x_c_total=1 << 62), INVALID)])
def test_rms_descriptors(d, want):
    assert status_of(B.dwconv_rms_norm, d, P, P, P, P, P, P, stream=0) == want
    assert status_of(B.dwconv_rms_norm_bwd, d, P, P, P, P, P, P, P, P, BIG, 0) == want
    assert B.dwconv_rms_norm_bwd_workspace_size(d) == 0
    assert B.dwconv_rms_norm_plan_name(d, 0) == B.dwconv_rms_norm_plan_name(d, 1) == "invalid"


def test_rms_arguments():
    d, f, b = rms(), B.dwconv_rms_norm, B.dwconv_rms_norm_bwd
    assert status_of(f, d, None, P, P, P, P, P, stream=0) == INVALID
    assert status_of(f, d, P, P, P, P, None, P, stream=0) == INVALID  # no output
    for k in range(5):  # x, residual, gamma, h, y
        a = [P] * 5
        a[k] = P + 1
        assert status_of(f, d, *a, P, stream=0) == MISALIGNED
    assert status_of(f, d, P, P, P, P, P, P + 2, stream=0) == MISALIGNED
    for t, want in ((act8(rows=15), INVALID), (act8(C=41), INVALID), (act8(kind=2), UNSUPPORTED), (act8(block=16), UNSUPPORTED),
                    (act8(codes=None), INVALID), (act8(scales=P + 2), MISALIGNED)):
        assert status_of(f, d, P, P, P, P, P, P, t, 0) == want
    need = B.dwconv_rms_norm_bwd_workspace_size(d)
    assert need >= 40 * 4 and B.dwconv_rms_norm_plan_name(d, 2) == "invalid"
    assert status_of(b, d, P, P, P, P, P, P, P, P, need - 1, 0) == WORKSPACE
    assert status_of(b, d, P, P, P, P, P, P, P, None, 0, 0) == WORKSPACE
    assert status_of(b, d, P, P, P, P, P, P, P, P + 8, BIG, 0) == MISALIGNED
    for k in (0, 1, 3):  # h, gy, rstd
        a = [P] * 7
        a[k] = None
        assert status_of(b, d, *a, P, BIG, 0) == INVALID
    for k in range(7):
        a = [P] * 7
        a[k] = P + 1
        assert status_of(b, d, *a, P, BIG, 0) == MISALIGNED
    assert status_of(b, d, None, None, None, None, None, None, None, None, 0, 0) == OK  # nothing asked for
    assert status_of(f, rms(rows=0), None, None, None, None, None, stream=0) == OK


def weight8(cout=24, cin=40, codes=P, scales=P):
    return B.make_weight8(cout, cin, codes, scales)


@pytest.mark.parametrize("w8,want", [
    (None, INVALID), (weight8(cout=0), INVALID), (weight8(cin=-1), INVALID), (weight8(cout=(1 << 20) + 1), UNSUPPORTED),
    (weight8(codes=None), INVALID), (weight8(scales=None), INVALID), (weight8(scales=P + 2), MISALIGNED)])
def test_weights(w8, want):
    assert status_of(B.dwconv_weight8_encode, P, w8, 0, "bf16", 0) == want
    assert status_of(B.dwconv2d_pointwise8, act8(), w8, P, 0, P, P, BIG, dtype="bf16", stream=0) == want


def test_weight_arguments():
    f = B.dwconv_weight8_encode
    assert status_of(f, None, weight8(), 0, "bf16", 0) == INVALID
    assert status_of(f, P + 1, weight8(), 0, "bf16", 0) == MISALIGNED
    assert status_of(f, P, weight8(), 2, "bf16", 0) == INVALID
    assert status_of(f, P, weight8(), 0, 3, 0) == UNSUPPORTED


def test_pointwise8_arguments():
    f, w8 = B.dwconv2d_pointwise8, weight8()
    go = lambda x8=None, w=w8, bias=P, act=0, y=P, ws=P, n=BIG, off=0, total=0, dtype="bf16": status_of(  # noqa: E731
        f, act8() if x8 is None else x8, w, bias, act, y, ws, n, off, total, dtype, 0)
    assert status_of(f, None, w8, P, 0, P, P, BIG, dtype="bf16", stream=0) == INVALID
    for x8, want in ((act8(rows=-1), INVALID), (act8(C=41), INVALID), (act8(kind="i8"), UNSUPPORTED), (act8(kind=7), UNSUPPORTED),
                     (act8(block=64), UNSUPPORTED), (act8(block=0), INVALID), (act8(codes=None), INVALID),
                     (act8(scales=None), INVALID), (act8(scales=P + 1), MISALIGNED), (act8(rows=1 << 40), UNSUPPORTED)):
        assert go(x8) == want
    assert go(act=5) == INVALID and go(act=-1) == INVALID and go(dtype=3) == UNSUPPORTED
    assert go(y=None) == INVALID and go(y=P + 1) == MISALIGNED and go(bias=P + 1) == MISALIGNED
    assert go(off=1) == INVALID and go(off=-1, total=64) == INVALID and go(total=23) == INVALID and go(off=2, total=25) == INVALID
    assert go(total=1 << 62) == UNSUPPORTED
    size = B.dwconv2d_pointwise8_workspace_size
    assert size(16, 40, 24) == 16 * 128 and size(16, 48, 24) == 0 and size(-1, 40, 24) == 0 and size(16, 0, 24) == 0
    assert go(ws=None, n=0) == WORKSPACE and go(n=16 * 128 - 1) == WORKSPACE and go(ws=P + 8) == MISALIGNED
    assert go(act8(rows=0, codes=None, scales=None), y=None, ws=None, n=0) == OK


def test_pointwise8_plans():
    name = B.dwconv2d_pointwise8_plan_name
    assert name(1, 4096, 4096) == name(32, 64, 64) == name(128, 4096, 4096) == "row"
    assert name(33, 64, 64) == name(196, 512, 512) == name(12544, 512, 512) == name(4096, 4096, 4096) == "tile"
    assert name(1, 1 << 20, 64) in ("row", "tile")
    assert name(-1, 64, 64) == name(1, 0, 64) == name(1, 64, (1 << 20) + 1) == "invalid"


def test_clip_arguments():
    f, size = B.dwconv_grad_norm_clip, B.dwconv_grad_norm_clip_workspace_size
    good = grads((P, P, 100, 0, 0), (P + 4096, None, 7, 2, 0))
    need = size(good)
    assert need >= 8 and size(grads((P, P, 0, 0, 0))) == 0
    assert status_of(f, good, 1.0, P, P, need - 1, 0) == WORKSPACE and status_of(f, good, 1.0, P, None, 0, 0) == WORKSPACE
    assert status_of(f, good, 1.0, P, P + 8, BIG, 0) == MISALIGNED
    for most in (0.0, -1.0, float("nan")):
        assert status_of(f, good, most, P, P, BIG, 0) == INVALID
    assert status_of(f, good, 1.0, P + 2, P, BIG, 0) == MISALIGNED
    for bad, want in (((P, P, -1, 0, 0), INVALID), ((P, P, 5, 3, 0), UNSUPPORTED), ((None, P, 5, 0, 0), INVALID),
                      ((P + 2, P, 5, 0, 0), MISALIGNED), ((P, P + 1, 5, 1, 0), MISALIGNED), ((P, P, 1 << 41, 1, 0), UNSUPPORTED)):
        assert status_of(f, grads((P, P, 100, 0, 0), bad), 1.0, P, P, BIG, 0) == want
    assert status_of(f, grads((P, P, 1 << 40, 0, 0), (P, P, 1 << 40, 0, 0)), 1.0, P, P, BIG, 0) == UNSUPPORTED
    assert B.load().dwconv_grad_norm_clip(-1, good, 1.0, P, P, BIG, None) == INVALID
    assert B.load().dwconv_grad_norm_clip(1, None, 1.0, P, P, BIG, None) == INVALID
    assert B.load().dwconv_grad_norm_clip(0, None, 1.0, None, None, 0, None) == OK


def test_lists_of_gradients():
    torch = pytest.importorskip("torch")
    a, b = torch.zeros(5), torch.zeros(6)
    with pytest.raises(ValueError):
        B.make_grads([a, b], [a])
    with pytest.raises(ValueError):
        B.make_grads([a], [b])
    with pytest.raises(ValueError):
        B.make_grads([a], [a.half()])
    with pytest.raises(ValueError):
        B.make_grads([torch.zeros(4, 4).t()])
    lst = B.make_grads([a, b])
    assert lst[0].out == lst[0].g == a.data_ptr() and lst[1].n == 6
