"""Channels-last training operators at the edges of their plans: tall images,
long chains of additions, checkpoints at any byte, and gradients whose group
sums weigh as much as their other terms. 64-bit forms are train_ref.py's."""
import pytest

torch = pytest.importorskip("torch")

import train_bounds as T
import train_ref as R
from depthwise_convolution_dwconv2d_gb300 import binding as B
from test_gpu_train_nhwc import NORMS, conv_inputs, filled, gen, new_act8, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from depthwise_convolution_dwconv2d_gb300 import build
    build.build()
    B.load()


class Guarded:
    """`nbytes` of workspace with 64 KB behind it that a call must leave as they are."""

    def __init__(self, nbytes):
        self.buf = torch.full((nbytes + (1 << 16),), 0x7f, dtype=torch.uint8, device="cuda")
        self.ws, self.behind = self.buf[:nbytes], self.buf[nbytes:]

    def check(self):
        assert bool((self.behind == 0x7f).all()), "written behind the workspace"


def conv_backward(d, x, gy, w, dtype, x8=None):
    gx, gw, gb = filled(d.N, d.H, d.W, d.C, dtype=dtype), filled(*w.shape, dtype=dtype), filled(w.shape[0], dtype=dtype)
    room = Guarded(B.dwconv2d_bwd_nhwc_workspace_size(d))
    B.dwconv2d_bwd_nhwc(d, x, gy, w, gx, gw, gb, room.ws, x8=x8)
    room.check()
    return gx, gw, gb


def check_conv(out, d, x, gy, w, dtype, chain, what):
    """chain: the most additions behind a value of gw or gb."""
    rgx, rgw, rgb, sx, sw, sb = R.conv_bwd(x.double(), gy.double(), w.double(), d)
    R.within(out[0], rgx, R.EPS32 * (d.kh * d.kw + 2) * sx, dtype, what + " gx")
    R.within(out[1], rgw, R.EPS32 * chain * sw, dtype, what + " gw")
    R.within(out[2], rgb, R.EPS32 * chain * sb, dtype, what + " gb")


# ---- layer backward: tall images -------------------------------------------


@pytest.mark.parametrize("dtype,C,H,W,k,s", [("f32", 17, 10000, 32, 5, 1), ("f32", 17, 8300, 32, 5, 1), ("bf16", 35, 17000, 9, 5, 1),
                                             ("f16", 17, 17000, 32, 7, 2), ("f32", 17, 10000, 32, 3, 1)])
@pytest.mark.parametrize("kind", ["none", "i8", "e4m3"])
def test_conv_backward_of_tall_images(dtype, C, H, W, k, s, kind):
    """Channels off 16 bytes: aligned copies of gy and of x or its codes, whichever of them the call's plan makes, stay
    inside the workspace that the descriptor alone decides. A thread adds at most 4096 products, then lanes and blocks."""
    d, x, w, gy = conv_inputs(1, C, H, W, k, s, k // 2, 1, 1, dtype, H + k)
    x8 = None
    if kind != "none":
        codes, scales = R.encode(x, kind, 32)
        x8 = B.make_act8(kind, 32, codes, scales)
    out = conv_backward(d, None if x8 else x, gy, w, dtype, x8)
    check_conv(out, d, R.decode(codes, scales, 32) if x8 else x, gy, w, dtype, 4096 + 256, f"{kind} {C}x{H}x{W} k{k}")


# ---- layer backward: codes at any byte -------------------------------------


def at_byte(t, by):
    """A contiguous copy of a one-byte tensor that starts `by` bytes after an allocation."""
    buf = torch.empty(t.numel() + by, dtype=torch.uint8, device="cuda")
    v = buf[by:].view(t.shape)
    v.copy_(t.view(torch.uint8))
    return v.view(t.dtype)


@pytest.mark.parametrize("by", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("N,C,H,W,k,s", [(2, 33, 9, 12, 3, 1), (2, 64, 13, 11, 3, 2), (3, 17, 12, 10, 5, 1), (1, 20, 15, 16, 5, 2),
                                         (1, 287, 8, 21, 7, 1), (2, 48, 19, 18, 7, 2), (2, 6, 9, 8, 3, 1)])
def test_conv_backward_from_codes_at_any_byte(N, C, H, W, k, s, by):
    """Copied to aligned pixels where channels are off 16 bytes, read by the direct kernels where only the pointer is."""
    for dtype, kind in (("bf16", "i8"), ("f32", "e4m3")):
        d, x, w, gy = conv_inputs(N, C, H, W, k, s, k // 2, 1, 1, dtype, C + by)
        codes, scales = R.encode(x, kind, 32)
        out = conv_backward(d, None, gy, w, dtype, B.make_act8(kind, 32, at_byte(codes, by), scales))
        check_conv(out, d, R.decode(codes, scales, 32), gy, w, dtype, 512, f"{dtype} {kind} at {by}")


# ---- long sums -------------------------------------------------------------


def test_conv_backward_filter_gradient_of_many_pixels():
    """131072 pixels of constant terms, a 9x9 filter (1024 channels and 82 sums of them fill the GPU with one chunk): 1024
    additions of a lane, 8 lanes, 16 chunks. One chain of 16384 is off by up to 4000 * 2^-24."""
    C, H, W, k = 1024, 264, 520, 9
    d = B.make_desc(1, C, H, W, k, 1, 0, 1, 1, "f32")
    g = gen(41)
    vx, vg = (torch.rand(C, generator=g, device="cuda") * 0.3 + 0.2 for _ in range(2))
    x, gy = vx.expand(1, H, W, C).contiguous(), vg.expand(1, H - 8, W - 8, C).contiguous()
    gw, gb = filled(C, k, k), filled(C)
    room = Guarded(B.dwconv2d_bwd_nhwc_workspace_size(d))
    B.dwconv2d_bwd_nhwc(d, x, gy, None, None, gw, gb, room.ws)
    room.check()
    n = (H - 8) * (W - 8)
    rgw, rgb = (n * vx.double() * vg.double())[:, None, None].expand(C, k, k), n * vg.double()
    R.within(gw, rgw, R.EPS32 * 1056 * rgw, "f32", "gw")
    R.within(gb, rgb, R.EPS32 * 1056 * rgb, "f32", "gb")


def test_norm_parameter_gradients_of_many_samples():
    """131075 samples of one pixel, a sum of each: 1024 additions in a run, 17 runs, 8 lanes."""
    N, C, G = 131075, 32, 4
    d = B.make_norm_desc(N, 1, 1, C, G, "none", 1e-5, "f32")
    g = gen(42)
    vx, vg = (torch.rand(C, generator=g, device="cuda") * 0.3 + 0.2 for _ in range(2))
    x, gy = vx.expand(N, 1, 1, C).contiguous(), vg.expand(N, 1, 1, C).contiguous()
    mean, rstd = torch.zeros(N, G, device="cuda"), torch.ones(N, G, device="cuda")
    gg, gb = filled(C), filled(C)
    room = Guarded(B.dwconv2d_group_norm_nhwc_workspace_size(d, 1))
    B.dwconv2d_group_norm_nhwc_bwd(d, x, gy, None, None, mean, rstd, None, gg, gb, room.ws)
    room.check()
    rgg, rgb = N * vx.double() * vg.double(), N * vg.double()
    R.within(gg, rgg, R.EPS32 * 1056 * rgg, "f32", "ggamma")
    R.within(gb, rgb, R.EPS32 * 1056 * rgb, "f32", "gbeta")


# ---- group norm: sums about a value that is not an outlier's ----------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,W,C,G", [(456, 256, 256, 8, 8), (152, 40, 40, 32, 32), (2, 56, 56, 128, 64), (456, 67, 61, 9, 3)])
def test_norm_moments_with_the_first_pixel_far_off(N, H, W, C, G, dtype):
    """All pixels of a channel alike but the first, 1000 away. About any value near the others the sums hold next to
    nothing but the outlier's own square, so what is left are the roundings of chained additions: 512 rows, 128 row lanes
    and 8 blocks or less, then channels. About the outlier each of a block's r rows brings its square, up to r / 4 chained
    roundings of r times the variance."""
    level = normal(gen(N + C), C, std=0.25).to(R.DT[dtype])
    x = level.expand(N, H, W, C).contiguous()
    x[:, 0, 0] = (level.float() + 1000).to(x.dtype)
    d = B.make_norm_desc(N, H, W, C, G, "none", 1e-5, dtype)
    y, mean, rstd = torch.empty_like(x), filled(N, G), filled(N, G)
    room = Guarded(B.dwconv2d_group_norm_nhwc_workspace_size(d, 0))
    B.dwconv2d_group_norm_nhwc(d, x, None, None, y, mean, rstd, room.ws)
    room.check()
    rmean, rrstd = R.moments(x[:1].double(), G, 1e-5)
    R.within(mean, rmean.expand(N, G), R.EPS32 * 768 * (1 + rmean.abs()).expand(N, G), "f32", "mean")
    R.within(rstd, rrstd.expand(N, G), R.EPS32 * 768 * rrstd.expand(N, G), "f32", "rstd")


# ---- group norm: every term of the gradients, from any source ---------------


def norm_pass(d, x, gamma, beta, shape, G, dtype, x8=None):
    y, mean, rstd = filled(*shape, dtype=dtype), filled(shape[0], G), filled(shape[0], G)
    room = Guarded(B.dwconv2d_group_norm_nhwc_workspace_size(d, 0))
    B.dwconv2d_group_norm_nhwc(d, x, gamma, beta, y, mean, rstd, room.ws, x8=x8)
    room.check()
    return y, mean, rstd


def norm_back(d, x, gy, gamma, beta, mean, rstd, dtype, x8=None):
    out = filled(*gy.shape, dtype=dtype), filled(gy.shape[-1], dtype=dtype), filled(gy.shape[-1], dtype=dtype)
    room = Guarded(B.dwconv2d_group_norm_nhwc_workspace_size(d, 1))
    B.dwconv2d_group_norm_nhwc_bwd(d, x, gy, gamma, beta, mean, rstd, *out, room.ws, x8=x8)
    room.check()
    return out


def check_gradients(out, x, gy, gamma, beta, mean, rstd, act, dtype, what):
    want, slack = T.backward(*(t.double() for t in (x, gy, gamma, beta, mean, rstd)), act)
    for name, o, w, s in zip(("gx", "ggamma", "gbeta"), out, want, slack):
        R.within(o, w, s, dtype, f"{what} {name}")


def away_from_kinks(gy, x, gamma, beta, mean, rstd, act):
    """gy, with no part where rounding may decide the slope."""
    if act not in ("relu", "relu6"):
        return gy
    C = x.shape[-1]
    u = (x.double() - R.per_channel(mean, C)) * R.per_channel(rstd, C) * gamma.double() + beta.double()
    return torch.where(u.abs() * (u - 6).abs() < 1e-4, torch.zeros_like(gy), gy)


@pytest.mark.parametrize("act", ["none", "relu", "relu6", "silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_norm_to_its_roundings(dtype, act):
    """y from the kernel's own moments, and gradients of a gy that gives both sums of a group the size of the term beside
    them: slabs, streams and slices wider than a block."""
    for i, (N, H, W, C, G) in enumerate(NORMS):
        what = f"{N}x{H}x{W}x{C} G{G}"
        x, gamma, beta, gy = T.inputs(N, H, W, C, G, dtype, i, "cuda")
        d = B.make_norm_desc(N, H, W, C, G, act, 1e-5, dtype)
        y, mean, rstd = norm_pass(d, x, gamma, beta, (N, H, W, C), G, dtype)
        ry, ey = T.forward(*(t.double() for t in (x, gamma, beta, mean, rstd)), act)
        R.within(y, ry, ey, dtype, what + " y")
        gy = away_from_kinks(gy, x, gamma, beta, mean, rstd, act)
        check_gradients(norm_back(d, x, gy, gamma, beta, mean, rstd, dtype), x, gy, gamma, beta, mean, rstd, act, dtype, what)


@pytest.mark.parametrize("by", [0, 1, 2, 4])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_norm_from_codes_at_any_byte(dtype, by):
    """The forward writes its checkpoint, and the backward reads it, at any byte."""
    for i, (N, H, W, C, G) in enumerate(NORMS):
        kind, block = (("i8", 32), ("e4m3", 64), ("i8", 128))[i % 3]
        what = f"{N}x{H}x{W}x{C} G{G} {kind} at {by}"
        x, gamma, beta, gy = T.inputs(N, H, W, C, G, dtype, 40 + i, "cuda")
        d = B.make_norm_desc(N, H, W, C, G, "silu", 1e-5, dtype)
        fresh = new_act8((N, H, W, C), kind, block)
        codes, scales = at_byte(fresh.tensors[0], by), fresh.tensors[1]
        x8 = B.make_act8(kind, block, codes, scales)
        y, mean, rstd = norm_pass(d, x, gamma, beta, (N, H, W, C), G, dtype, x8)
        ry, ey = T.forward(*(t.double() for t in (x, gamma, beta, mean, rstd)), "silu")
        R.within(y, ry, ey, dtype, what + " y")
        want, wscales = R.encode(x, kind, block)
        assert torch.equal(codes.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales, wscales), what
        out = norm_back(d, None, gy, gamma, beta, mean, rstd, dtype, x8)
        check_gradients(out, R.decode(want, wscales, block), gy, gamma, beta, mean, rstd, "silu", dtype, what)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("by", [1, 2, 4, 12])
def test_act8_codes_at_any_byte(kind, by):
    """Bit for bit the definition's codes and values; the bytes before and behind them stay."""
    for dtype, rows, C, block in (("bf16", 33, 64, 32), ("f32", 7, 40, 32), ("f16", 257, 8, 64), ("bf16", 5, 200, 128), ("f32", 3, 33, 32)):
        x = normal(gen(by + C), rows, C, dtype=dtype)
        buf = torch.full((by + rows * C + 32,), 0x55, dtype=torch.uint8, device="cuda")
        codes = buf[by:by + rows * C].view(rows, C)
        scales = torch.empty(rows, -(-C // block), device="cuda")
        x8 = B.make_act8(kind, block, codes, scales)
        B.dwconv_act8_encode(x, x8)
        want, wscales = R.encode(x, kind, block)
        assert torch.equal(codes, want.view(torch.uint8)) and torch.equal(scales, wscales), (dtype, rows, C)
        assert bool((buf[:by] == 0x55).all()) and bool((buf[by + rows * C:] == 0x55).all())
        y = filled(rows, C, dtype=dtype)
        B.dwconv_act8_decode(x8, y)
        assert torch.equal(y, R.decode(want, wscales, block).float().to(R.DT[dtype])), (dtype, rows, C)
