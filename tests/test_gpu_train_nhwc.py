"""Channels-last training operators on the GPU: 8-bit activation checkpoints,
group norm with an activation (forward and backward) and the depthwise
backward, against plain 64-bit forms (train_ref.py)."""
import pytest

torch = pytest.importorskip("torch")

import train_ref as R
from depthwise_convolution_dwconv2d_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from depthwise_convolution_dwconv2d_gb300 import build
    build.build()
    B.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype="f32", std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(R.DT[dtype])


def filled(*shape, dtype="f32", value=-7.0):
    return torch.full(shape, value, dtype=R.DT[dtype], device="cuda")


def room(nbytes):
    return torch.full((max(nbytes, 16),), 0x7f, dtype=torch.uint8, device="cuda")


def new_act8(shape, kind, block):
    codes = torch.full(shape, 0x55, dtype=torch.uint8, device="cuda").view(
        torch.int8 if kind == "i8" else torch.float8_e4m3fn)
    scales = torch.full((*shape[:-1], -(-shape[-1] // block)), -1.0, device="cuda")
    return B.make_act8(kind, block, codes, scales)


def offset_view(t, by=1):
    """A contiguous copy of t that starts `by` elements after an allocation: not 16-byte aligned."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


# ---- 8-bit checkpoints -----------------------------------------------------

ROWS = [(1, 1), (1, 31), (3, 32), (5, 33), (7, 64), (2, 65), (9, 96), (4, 127), (33, 128), (3, 200), (257, 8),
        (130, 24), (1, 1024), (6, 1000)]


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_act8_codes_are_the_definition_bit_for_bit(dtype, kind, block):
    for i, (rows, C) in enumerate(ROWS):
        g = gen(i)
        x = normal(g, rows, C, dtype=dtype)
        x *= torch.exp2(torch.randint(-9, 6, (rows, 1), generator=g, device="cuda").float()).to(x.dtype)
        x[rows // 2] = 0
        x8 = new_act8((rows, C), kind, block)
        B.dwconv_act8_encode(x, x8)
        y = filled(rows, C, dtype=dtype)
        B.dwconv_act8_decode(x8, y)
        codes, scales = x8.tensors
        want, wscales = R.encode(x, kind, block)
        assert torch.equal(scales, wscales), (rows, C)
        assert torch.equal(codes.view(torch.uint8), want.view(torch.uint8)), (rows, C)
        assert torch.equal(y, R.decode(want, wscales, block).to(torch.float32).to(R.DT[dtype])), (rows, C)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_act8_slices_and_unaligned_pointers(kind):
    """Rows further apart than C, and pointers at an odd element: the values between rows stay."""
    for dtype, C, total, off in (("bf16", 64, 96, 0), ("f16", 64, 100, 3), ("f32", 40, 44, 4), ("bf16", 48, 48, 1)):
        g = gen(C + total)
        buf = normal(g, 11 * total + off, dtype=dtype)
        x = buf[off:].view(11, total)
        x8 = new_act8((11, C), kind, 32)
        B.dwconv_act8_encode(x.data_ptr(), x8, total, dtype)
        want, wscales = R.encode(x[:, :C], kind, 32)
        assert torch.equal(x8.tensors[0].view(torch.uint8), want.view(torch.uint8))
        out = filled(11 * total + off, dtype=dtype)
        v = out[off:].view(11, total)
        B.dwconv_act8_decode(x8, v.data_ptr(), total, dtype)
        assert torch.equal(v[:, :C], R.decode(want, wscales, 32).float().to(R.DT[dtype]))
        assert bool((v[:, C:] == -7).all()) and bool((out[:off] == -7).all())


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("C", [64, 63])
def test_act8_keeps_overflow_visible_and_zeros_exact(dtype, kind, C):
    """A block with an infinity or a NaN decodes to NaN throughout, its neighbours do not; zeros, negative zeros and
    values too small for a normal scale decode to zero."""
    x = normal(gen(5), 6, C, dtype=dtype)
    x[0, 3] = float("inf")
    x[1, 40] = float("-inf")
    x[2, 33] = float("nan")
    x[3] = 0
    x[4] = -0.0
    if dtype != "f16":
        x[5, :32] = 2.0 ** -126
    x8 = new_act8((6, C), kind, 32)
    y = filled(6, C, dtype=dtype)
    B.dwconv_act8_encode(x, x8)
    B.dwconv_act8_decode(x8, y)
    assert bool(y[0, :32].isnan().all()) and bool(y[0, 32:].isfinite().all())
    assert bool(y[1, 32:].isnan().all()) and bool(y[1, :32].isfinite().all())
    assert bool(y[2, 32:].isnan().all()) and bool(y[2, :32].isfinite().all())
    assert bool((y[3:5] == 0).all())
    if dtype != "f16":
        assert bool((y[5, :32] == 0).all()) and bool((y[5, 32:] != 0).any())


def test_act8_beyond_32_bit_offsets():
    rows, C = (1 << 25) + 5, 64  # 2^31 elements and more
    x = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    tail = normal(gen(1), 9, C, dtype="bf16")
    x[-9:] = tail
    x8 = B.make_act8("i8", 64, torch.empty(rows, C, dtype=torch.int8, device="cuda"),
                     torch.empty(rows, 1, device="cuda"))
    B.dwconv_act8_encode(x, x8)
    want, ws = R.encode(tail, "i8", 64)
    assert torch.equal(x8.tensors[0][-9:], want) and torch.equal(x8.tensors[1][-9:], ws)
    assert int(x8.tensors[0][:-9].count_nonzero()) == 0
    x.fill_(3)
    B.dwconv_act8_decode(x8, x)
    assert torch.equal(x[-9:], R.decode(want, ws, 64).to(torch.bfloat16))
    assert int(x[:-9].count_nonzero()) == 0


# ---- group norm ------------------------------------------------------------

EPS = 1e-5

# N, H, W, C, G: one pixel, one channel per group, one group, odd sizes, groups that are no multiple of a vector, groups
# wider than a vector's slice, planes that one block holds and that it does not, fewer pixels than thread blocks
NORMS = [(1, 1, 1, 8, 2), (2, 1, 1, 7, 7), (1, 2, 3, 5, 1), (3, 7, 7, 64, 32), (2, 5, 9, 30, 3), (1, 14, 14, 512, 32),
         (2, 19, 23, 40, 4), (2, 37, 29, 320, 32), (4, 28, 28, 128, 1), (1, 64, 65, 24, 3), (1, 128, 128, 16, 2),
         (2, 3, 3, 1024, 8), (1, 9, 9, 2056, 1), (5, 11, 3, 33, 11), (1, 200, 150, 8, 1), (2, 56, 56, 128, 32), (1, 5, 4, 1031, 1), (2, 4, 5, 1044, 2)]


def norm_inputs(N, H, W, C, dtype, seed, level=0.5):
    g = gen(seed)
    x = (torch.randn(N, H, W, C, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(C, generator=g, device="cuda"))
         + level * torch.randn(C, generator=g, device="cuda")).to(R.DT[dtype])
    gamma, beta = normal(g, C, dtype=dtype, std=0.3, mean=1.0), normal(g, C, dtype=dtype, std=0.4)
    return x, gamma, beta, normal(g, N, H, W, C, dtype=dtype, std=0.05)


def run_fwd(d, x, gamma, beta, N, G, shape, dtype, x8=None, stream=None):
    y = filled(*shape, dtype=dtype)
    mean, rstd = filled(N, G), filled(N, G)
    B.dwconv2d_group_norm_nhwc(d, x, gamma, beta, y, mean, rstd, room(B.dwconv2d_group_norm_nhwc_workspace_size(d, 0)),
                               x8=x8, stream=stream)
    return y, mean, rstd


def run_bwd(d, x, gy, gamma, beta, mean, rstd, shape, C, dtype, x8=None, stream=None):
    gx, gg, gb = filled(*shape, dtype=dtype), filled(C, dtype=dtype), filled(C, dtype=dtype)
    B.dwconv2d_group_norm_nhwc_bwd(d, x, gy, gamma, beta, mean, rstd, gx, gg, gb,
                                   room(B.dwconv2d_group_norm_nhwc_workspace_size(d, 1)), x8=x8, stream=stream)
    return gx, gg, gb


def check_fwd(y, mean, rstd, x, gamma, beta, G, act, dtype, what):
    x, gamma, beta = x.double(), gamma.double(), beta.double()
    ry, rmean, rrstd = R.norm_fwd(x, gamma, beta, G, EPS, act)
    C = x.shape[-1]
    size = R.per_channel((x.abs().reshape(x.shape[0], -1, G, C // G)).mean((1, 3)), C)  # what the mean's error goes by
    slack = R.EPS32 * (16 * (x.abs() + R.CHAIN * size) * R.per_channel(rrstd, C) * gamma.abs() + 64 * ry.abs() + 4 * beta.abs())
    R.within(y, ry, slack, dtype, what + " y")
    R.within(mean, rmean, R.CHAIN * R.EPS32 * size[:, 0, 0, ::C // G], "f32", what + " mean")
    cond = 1 + (size[:, 0, 0, ::C // G] * rrstd) ** 2  # deviations from a mean that is off by a rounding
    R.within(rstd, rrstd, R.CHAIN * R.EPS32 * rrstd * cond, "f32", what + " rstd")


def check_bwd(gx, gg, gb, x, gy, gamma, beta, mean, rstd, act, dtype, what):
    a = [t.double() for t in (x, gy, gamma, beta, mean, rstd)]
    rgx, rgg, rgb, size, sg, sb = R.norm_bwd(*a, act)
    N, G = mean.shape
    C = x.shape[-1]
    off = 1 + (R.per_channel(a[4].abs(), C) * R.per_channel(a[5], C))  # (x - mean): a rounding of the larger one
    far = 8 * (1 + a[0].abs().max() * a[5].max())  # how steep the slopes are times that
    R.within(gx, rgx, R.EPS32 * far * off * (8 * size), dtype, what + " gx")
    R.within(gg, rgg, R.EPS32 * (R.CHAIN * sg + far * float(off.max()) * (sg + sb)), dtype, what + " ggamma")
    R.within(gb, rgb, R.EPS32 * (R.CHAIN * sb + far * float(off.max()) * (sg + sb)), dtype, what + " gbeta")


@pytest.mark.parametrize("act", ["none", "relu", "relu6", "silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_norm_forward_and_backward(dtype, act):
    for i, (N, H, W, C, G) in enumerate(NORMS):
        what = f"{N}x{H}x{W}x{C} G{G}"
        x, gamma, beta, gy = norm_inputs(N, H, W, C, dtype, i)
        d = B.make_norm_desc(N, H, W, C, G, act, EPS, dtype)
        y, mean, rstd = run_fwd(d, x, gamma, beta, N, G, (N, H, W, C), dtype)
        check_fwd(y, mean, rstd, x, gamma, beta, G, act, dtype, what)
        if act in ("relu", "relu6"):  # slopes at the kink follow the forward's own arithmetic
            u = (x.float() - R.per_channel(mean, C)) * R.per_channel(rstd, C) * gamma.float() + beta.float()
            gy = torch.where(u.abs() * (u - 6).abs() < 1e-4, torch.zeros_like(gy), gy)
        out = run_bwd(d, x, gy, gamma, beta, mean, rstd, (N, H, W, C), C, dtype)
        check_bwd(*out, x, gy, gamma, beta, mean, rstd, act, dtype, what)


@pytest.mark.parametrize("kind,block", [("i8", 32), ("i8", 64), ("e4m3", 32), ("e4m3", 128)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_norm_writes_and_reads_checkpoints(dtype, kind, block):
    """The forward's checkpoint is the encoder's, bit for bit; the backward from it is the formula on its values."""
    for i, (N, H, W, C, G) in enumerate(NORMS):
        what = f"{N}x{H}x{W}x{C} G{G}"
        x, gamma, beta, gy = norm_inputs(N, H, W, C, dtype, 50 + i)
        d = B.make_norm_desc(N, H, W, C, G, "silu", EPS, dtype)
        x8 = new_act8((N, H, W, C), kind, block)
        y, mean, rstd = run_fwd(d, x, gamma, beta, N, G, (N, H, W, C), dtype, x8)
        check_fwd(y, mean, rstd, x, gamma, beta, G, "silu", dtype, what)
        codes, scales = R.encode(x, kind, block)
        assert torch.equal(x8.tensors[0].view(torch.uint8), codes.view(torch.uint8)), what
        assert torch.equal(x8.tensors[1], scales), what
        out = run_bwd(d, None, gy, gamma, beta, mean, rstd, (N, H, W, C), C, dtype, x8)
        check_bwd(*out, R.decode(codes, scales, block), gy, gamma, beta, mean, rstd, "silu", dtype, what)


@pytest.mark.parametrize("dtype,C,G,xs,xo,ys,yo", [("bf16", 64, 8, 192, 64, 96, 32), ("f32", 24, 3, 31, 5, 24, 0),
                                                     ("f16", 40, 5, 48, 8, 43, 3), ("f32", 32, 32, 64, 32, 40, 4)])
def test_norm_channel_slices(dtype, C, G, xs, xo, ys, yo):
    """Slices of wider buffers (concatenated branches): nothing outside them is written."""
    N, H, W = 2, 13, 11
    g = gen(9)
    xb, gyb = normal(g, N, H, W, xs, dtype=dtype), normal(g, N, H, W, ys, dtype=dtype, std=0.1)
    gamma, beta = normal(g, C, dtype=dtype, mean=1.0, std=0.2), normal(g, C, dtype=dtype)
    d = B.make_norm_desc(N, H, W, C, G, "gelu", EPS, dtype, xo, xs, yo, ys)
    x, gy = xb[..., xo:xo + C], gyb[..., yo:yo + C]
    x8 = new_act8((N, H, W, C), "i8", 32)
    y, mean, rstd = run_fwd(d, xb, gamma, beta, N, G, (N, H, W, ys), dtype, x8)
    check_fwd(y[..., yo:yo + C], mean, rstd, x, gamma, beta, G, "gelu", dtype, "slice")
    assert bool((y[..., :yo] == -7).all()) and bool((y[..., yo + C:] == -7).all())
    codes, scales = R.encode(x.contiguous(), "i8", 32)
    assert torch.equal(x8.tensors[0], codes) and torch.equal(x8.tensors[1], scales)
    gx, gg, gb = run_bwd(d, xb, gyb, gamma, beta, mean, rstd, (N, H, W, xs), C, dtype)
    check_bwd(gx[..., xo:xo + C], gg, gb, x, gy, gamma, beta, mean, rstd, "gelu", dtype, "slice")
    assert bool((gx[..., :xo] == -7).all()) and bool((gx[..., xo + C:] == -7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_unaligned_pointers_optional_operands_and_streams(dtype):
    """Odd pointers give the results of aligned ones within tolerance; NULL gamma and beta are 1 and 0; NULL outputs are
    skipped; a call on another stream runs there; repeated calls are bitwise equal."""
    N, H, W, C, G = 2, 17, 15, 64, 4
    x, gamma, beta, gy = norm_inputs(N, H, W, C, dtype, 77)
    d = B.make_norm_desc(N, H, W, C, G, "silu", EPS, dtype)
    one, zero = torch.ones_like(gamma), torch.zeros_like(beta)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, mean, rstd = run_fwd(d, offset_view(x), None, None, N, G, (N, H, W, C), dtype)
        out = run_bwd(d, offset_view(x), offset_view(gy), None, None, mean, rstd, (N, H, W, C), C, dtype)
        again = run_bwd(d, offset_view(x), offset_view(gy), None, None, mean, rstd, (N, H, W, C), C, dtype)
    side.synchronize()
    check_fwd(y, mean, rstd, x, one, zero, G, "silu", dtype, "unaligned")
    check_bwd(*out, x, gy, one, zero, mean, rstd, "silu", dtype, "unaligned")
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    y2 = filled(N, H, W, C, dtype=dtype)
    B.dwconv2d_group_norm_nhwc(d, x, gamma, beta, y2, None, None, room(B.dwconv2d_group_norm_nhwc_workspace_size(d, 0)))
    y3, mean, rstd = run_fwd(d, x, gamma, beta, N, G, (N, H, W, C), dtype)
    assert torch.equal(y2, y3)
    whole = run_bwd(d, x, gy, gamma, beta, mean, rstd, (N, H, W, C), C, dtype)
    ws = room(B.dwconv2d_group_norm_nhwc_workspace_size(d, 1))
    for k in range(3):
        part = [filled(*t.shape, dtype=dtype) if j == k else None for j, t in enumerate(whole)]
        B.dwconv2d_group_norm_nhwc_bwd(d, x, gy, gamma, beta, mean, rstd, *part, ws)
        assert torch.equal(part[k], whole[k])


@pytest.mark.parametrize("shape", [(1, 12, 12, 64, 4), (1, 200, 150, 8, 1)])
def test_norm_variance_of_a_far_level(shape):
    """Values around 1000 with a spread of 1: sums of squares of x would lose the variance."""
    N, H, W, C, G = shape
    x = normal(gen(3), N, H, W, C, mean=1000.0)
    d = B.make_norm_desc(N, H, W, C, G, "none", EPS, "f32")
    _, mean, rstd = run_fwd(d, x, None, None, N, G, (N, H, W, C), "f32")
    rmean, rrstd = R.moments(x.double(), G, EPS)
    R.within(mean, rmean, R.CHAIN * R.EPS32 * rmean.abs(), "f32", "mean")
    # deviations from a value within a few spreads of the mean: rounding of the mean enters squared
    R.within(rstd, rrstd, R.CHAIN * R.EPS32 * rrstd * (1 + (1000 * R.CHAIN * R.EPS32) ** 2), "f32", "rstd")


@pytest.mark.parametrize("shape", [(2, 40, 40, 64, 4), (1, 200, 150, 8, 1), (2, 21, 20, 33, 3)])
def test_norm_variance_beside_an_outlier(shape):
    """The first pixel, which the sums are taken about, a thousand spreads off: the outlier is part of the variance, and
    a block of r rows has at most r roundings of it."""
    N, H, W, C, G = shape
    x = normal(gen(3), N, H, W, C)
    x[:, 0, 0] += 1000
    d = B.make_norm_desc(N, H, W, C, G, "none", EPS, "f32")
    _, mean, rstd = run_fwd(d, x, None, None, N, G, (N, H, W, C), "f32")
    rmean, rrstd = R.moments(x.double(), G, EPS)
    R.within(mean, rmean, R.EPS32 * (1000 + R.CHAIN), "f32", "mean")
    R.within(rstd, rrstd, R.EPS32 * (H * W + R.CHAIN) * rrstd, "f32", "rstd")


@pytest.mark.parametrize("shape", [(2, 6, 6, 64, 2), (2, 5, 5, 33, 3)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_norm_keeps_nan_inside_its_group(shape, bad):
    N, H, W, C, G = shape
    x, gamma, beta, gy = norm_inputs(N, H, W, C, "f32", 4)
    x[1, 2, 3, 0] = bad
    D = C // G
    for act in ("none", "relu", "relu6", "silu", "gelu"):
        d = B.make_norm_desc(N, H, W, C, G, act, EPS, "f32")
        y, mean, rstd = run_fwd(d, x, gamma, beta, N, G, (N, H, W, C), "f32")
        assert bool(y[1, ..., :D].isnan().all()) and bool(y[0].isfinite().all()) and bool(y[1, ..., D:].isfinite().all())
        gx, gg, gb = run_bwd(d, x, gy, gamma, beta, mean, rstd, (N, H, W, C), C, "f32")
        assert bool(gx[1, ..., :D].isnan().all()) and bool(gx[0].isfinite().all())
        assert bool(gx[1, ..., D:].isfinite().all()) and bool(gg[D:].isfinite().all())
        assert bool(gg[:D].isnan().any())


def test_norm_constant_group_and_single_value_groups():
    """Variance 0: xh is 0 and y is act(beta), the gradient has no infinities (eps > 0)."""
    for N, H, W, C, G in ((1, 4, 4, 64, 8), (2, 1, 1, 16, 16)):
        x = torch.full((N, H, W, C), 5.0, device="cuda")
        beta = normal(gen(2), C)
        d = B.make_norm_desc(N, H, W, C, G, "none", EPS, "f32")
        y, mean, rstd = run_fwd(d, x, None, beta, N, G, (N, H, W, C), "f32")
        assert torch.equal(y, beta.expand(N, H, W, C))
        assert torch.equal(mean, torch.full_like(mean, 5.0))
        gx, gg, gb = run_bwd(d, x, normal(gen(3), N, H, W, C), None, beta, mean, rstd, (N, H, W, C), C, "f32")
        assert bool(gx.isfinite().all()) and bool((gg == 0).all())


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", [(2, 5, 7, 16, 4), (1, 30, 30, 64, 2), (2, 4, 3, 9, 3)])
def test_norm_gradient_against_differences(act, shape):
    """(L(p + h v) - L(p - h v)) / 2h with L = sum y * r, forward in fp32 and the sum in 64 bits. The second difference's
    error is h^2 L''' / 6; L's own error is about 2^-22 of sum |y r| at random signs."""
    N, H, W, C, G = shape
    x, gamma, beta, r = norm_inputs(N, H, W, C, "f32", 11)
    d = B.make_norm_desc(N, H, W, C, G, act, EPS, "f32")
    y, mean, rstd = run_fwd(d, x, gamma, beta, N, G, (N, H, W, C), "f32")
    grads = run_bwd(d, x, r, gamma, beta, mean, rstd, (N, H, W, C), C, "f32")
    L = lambda *a: float((run_fwd(d, *a, N, G, (N, H, W, C), "f32")[0].double() * r.double()).sum())  # noqa: E731
    h = 2.0 ** -7
    for k, t in enumerate((x, gamma, beta)):
        v = normal(gen(20 + k), *t.shape)
        lo, hi = [x, gamma, beta], [x, gamma, beta]
        lo[k], hi[k] = t - h * v, t + h * v
        diff = (L(*hi) - L(*lo)) / (2 * h)
        want = float((grads[k].double() * v.double()).sum())
        size = float((grads[k].double() * v.double()).square().sum().sqrt())
        noise = 2.0 ** -22 * float((y.double() * r.double()).square().sum().sqrt()) / h
        assert abs(diff - want) <= 4 * noise + 64 * h * h * max(size, float(r.double().square().sum().sqrt())), (k, diff, want)


def test_norm_empty_batch():
    d = B.make_norm_desc(0, 4, 4, 32, 4, "relu", EPS, "f32")
    assert B.dwconv2d_group_norm_nhwc_workspace_size(d, 0) == 0
    B.dwconv2d_group_norm_nhwc(d, None, None, None, None, None, None, None)
    gg, gb = filled(32), filled(32)
    B.dwconv2d_group_norm_nhwc_bwd(d, None, None, None, None, None, None, None, gg, gb, None)
    assert bool((gg == 0).all()) and bool((gb == 0).all())


def test_norm_beyond_32_bit_offsets():
    N, H, W, C, G = 3, 4096, 2800, 64, 8  # the last sample starts past 2^30 elements and ends past 2^31
    x = torch.zeros(N, H, W, C, dtype=torch.bfloat16, device="cuda")
    x[-1] = normal(gen(1), H, W, C, dtype="bf16", mean=0.5)
    d = B.make_norm_desc(N, H, W, C, G, "silu", EPS, "bf16")
    y, mean, rstd = run_fwd(d, x, None, None, N, G, (N, H, W, C), "bf16")
    rows = slice(H - 3, H)
    rmean, rrstd = R.moments(x[-1:].double(), G, EPS)
    assert float((mean[-1:] - rmean).abs().max()) < 1e-5 and float((rstd[-1:] / rrstd - 1).abs().max()) < 1e-5
    u = (x[-1, rows].double() - R.per_channel(rmean, C)[0]) * R.per_channel(rrstd, C)[0]
    R.within(y[-1, rows], R.act(u, "silu"), 1e-4, "bf16", "tail")
    assert bool((y[:-1] == 0).all())
    del u
    gx, gg, gb = run_bwd(d, x, y, None, None, mean, rstd, (N, H, W, C), C, "bf16")
    xh = (x[-1:].float() - R.per_channel(mean[-1:], C)) * R.per_channel(rstd[-1:], C)
    q = torch.sigmoid(xh)
    du = y[-1:].float() * (q * (1 + xh * (1 - q)))
    s1, s2 = (t.reshape(-1, G, C // G).double().mean((0, 2)).repeat_interleave(C // G) for t in (du, du * xh))
    want = R.per_channel(rstd[-1:].double(), C)[0] * (du[0, rows].double() - s1 - xh[0, rows].double() * s2)
    R.within(gx[-1, rows], want, 1e-4, "bf16", "gx tail")
    total = (du * xh).double().sum((0, 1, 2))
    assert float((gg.double() / total - 1).abs().max()) < 1e-2


# ---- depthwise backward ----------------------------------------------------

# N, C, H, W, k, stride, pad, dilation, multiplier: the row-walking kernel's shapes (odd and even sides, one pixel, sides
# below the filter, channels below and above one warp's, odd channels) and shapes that only the generic kernels serve
CONVS = [(1, 8, 1, 1, 3, 1, 1, 1, 1), (2, 64, 5, 6, 3, 1, 1, 1, 1), (3, 130, 7, 7, 3, 1, 1, 1, 1), (2, 33, 9, 12, 3, 1, 1, 1, 1),
         (1, 7, 20, 3, 3, 1, 0, 1, 1), (2, 66, 13, 11, 3, 2, 1, 1, 1), (2, 16, 14, 14, 3, 2, 0, 1, 1), (1, 5, 8, 9, 3, 2, 1, 1, 1),
         (2, 72, 12, 10, 5, 1, 2, 1, 1), (1, 20, 3, 4, 5, 1, 2, 1, 1), (2, 34, 15, 16, 5, 2, 2, 1, 1), (1, 40, 17, 9, 5, 2, 1, 1, 1),
         (2, 24, 11, 13, 7, 1, 3, 1, 1), (1, 9, 8, 21, 7, 1, 2, 1, 1), (1, 68, 19, 18, 7, 2, 3, 1, 1), (4, 256, 28, 28, 3, 1, 1, 1, 1),
         (1, 32, 60, 70, 3, 1, 1, 1, 1), (16, 12, 9, 9, 3, 2, 1, 1, 1),
         (3, 40, 6, 37, 3, 1, 1, 1, 1), (17, 48, 7, 7, 3, 1, 1, 1, 1), (9, 96, 7, 8, 3, 2, 1, 1, 1), (2, 64, 31, 45, 3, 2, 0, 1, 1),
         (5, 160, 4, 3, 3, 1, 0, 1, 1), (1, 80, 3, 130, 3, 2, 1, 1, 1), (2, 64, 70, 5, 3, 1, 1, 1, 1), (1, 32, 1, 1, 3, 2, 1, 1, 1),
         (2, 6, 9, 8, 3, 1, 2, 1, 1), (1, 10, 9, 9, 4, 1, 1, 1, 1), (2, 5, 11, 12, 3, 1, 2, 2, 1), (1, 6, 8, 7, 3, 1, 1, 1, 2),
         (1, 4, 9, 9, (3, 5), (2, 1), (1, 2), 1, 3), (1, 3, 12, 12, 9, 1, 4, 1, 1), (1, 5, 6, 6, 3, 3, 1, 1, 1)]


def conv_inputs(N, C, H, W, k, s, p, dil, m, dtype, seed):
    d = B.make_desc(N, C, H, W, k, s, p, dil, m, dtype)
    Ho, Wo = B.dwconv2d_output_shape(d)
    g = gen(seed)
    x = normal(g, N, H, W, C, dtype=dtype)
    w = normal(g, C * m, d.kh, d.kw, dtype=dtype, std=1.0 / d.kh)
    gy = normal(g, N, Ho, Wo, C * m, dtype=dtype)
    return d, x, w, gy


def run_conv(d, x, gy, w, dtype, x8=None, accumulate=0, gx=None, stream=None):
    gx = filled(d.N, d.H, d.W, d.C, dtype=dtype) if gx is None else gx
    gw, gb = filled(*w.shape, dtype=dtype), filled(w.shape[0], dtype=dtype)
    ws = room(B.dwconv2d_bwd_nhwc_workspace_size(d))
    B.dwconv2d_bwd_nhwc(d, x, gy, w, gx, gw, gb, ws, x8=x8, accumulate=accumulate, stream=stream)
    return gx, gw, gb


def check_conv(out, d, x, gy, w, dtype, what, onto=None):
    rgx, rgw, rgb, sx, sw, sb = R.conv_bwd(x.double(), gy.double(), w.double(), d)
    if onto is not None:
        rgx, sx = rgx + onto.double(), sx + onto.double().abs()
    taps = d.kh * d.kw * d.multiplier
    R.within(out[0], rgx, R.EPS32 * (taps + 2) * sx, dtype, what + " gx")
    R.within(out[1], rgw, R.EPS32 * R.CHAIN * sw, dtype, what + " gw")
    R.within(out[2], rgb, R.EPS32 * R.CHAIN * sb, dtype, what + " gb")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_conv_backward(dtype):
    for i, shape in enumerate(CONVS):
        d, x, w, gy = conv_inputs(*shape, dtype, i)
        check_conv(run_conv(d, x, gy, w, dtype), d, x, gy, w, dtype, str(shape))


@pytest.mark.parametrize("kind,block", [("i8", 32), ("i8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_conv_backward_from_a_checkpoint(dtype, kind, block):
    for i, shape in enumerate(CONVS):
        d, x, w, gy = conv_inputs(*shape, dtype, 100 + i)
        codes, scales = R.encode(x, kind, block)
        out = run_conv(d, None, gy, w, dtype, B.make_act8(kind, block, codes, scales))
        check_conv(out, d, R.decode(codes, scales, block), gy, w, dtype, str(shape))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_backward_parts_accumulation_slices_and_pointers(dtype):
    for i, (shape, off, total) in enumerate([(CONVS[2], 8, 144), (CONVS[3], 1, 40), (CONVS[5], 2, 70), (CONVS[8], 0, 75),
                                             (CONVS[12], 8, 40), (CONVS[-6], 3, 16), (CONVS[-3], 5, 20),
                                             (CONVS[18], 8, 56), (CONVS[20], 16, 128), (CONVS[21], 4, 72)]):
        d, x, w, _ = conv_inputs(*shape, dtype, 200 + i)
        d.out_c_offset, d.out_c_total = off, total
        OC = w.shape[0]
        Ho, Wo = B.dwconv2d_output_shape(d)
        buf = normal(gen(300 + i), d.N, Ho, Wo, total, dtype=dtype)
        gy = buf[..., off:off + OC]
        whole = run_conv(d, x, buf, w, dtype)
        check_conv(whole, d, x, gy, w, dtype, str(shape))
        ws = room(B.dwconv2d_bwd_nhwc_workspace_size(d))
        for k in range(3):
            part = [filled(*t.shape, dtype=dtype) if j == k else None for j, t in enumerate(whole)]
            B.dwconv2d_bwd_nhwc(d, x if k == 1 else None, buf, w if k == 0 else None, *part, None if k == 0 else ws)
            assert torch.equal(part[k], whole[k]), (shape, k)
        onto = normal(gen(400 + i), *x.shape, dtype=dtype)
        added = run_conv(d, x, buf, w, dtype, accumulate=1, gx=onto.clone())
        check_conv(added, d, x, gy, w, dtype, str(shape), onto)
        assert torch.equal(added[1], whole[1])
        odd = run_conv(d, offset_view(x), offset_view(buf), offset_view(w), dtype, gx=offset_view(onto))
        check_conv(odd, d, x, gy, w, dtype, str(shape) + " odd pointers")


def test_conv_backward_against_differences():
    """The layer is linear in x and in w: central differences of L = sum y * r with a step of 1 have no error of their own."""
    for shape in (CONVS[1], CONVS[5], CONVS[8], CONVS[14]):
        d, x, w, r = conv_inputs(*shape, "f32", 31)
        gx, gw, gb = run_conv(d, x, r, w, "f32")

        def L(x_, w_):
            y = torch.empty_like(r)
            B.dwconv2d_fwd_nhwc(d, x_, w_, None, y)
            return float((y.double() * r.double()).sum())

        for grad, v, lo, hi in ((gx, normal(gen(1), *x.shape), None, None), (gw, normal(gen(2), *w.shape), None, None)):
            diff = (L(x + v, w) - L(x - v, w)) / 2 if grad is gx else (L(x, w + v) - L(x, w - v)) / 2
            size = float((grad.double() * v.double()).abs().sum())
            noise = 2.0 ** -22 * float(r.double().square().sum().sqrt()) * d.kh * d.kw
            assert abs(diff - float((grad.double() * v.double()).sum())) <= 2.0 ** -20 * size + 8 * noise


def test_conv_backward_empty_batch_and_repeats():
    d = B.make_desc(0, 16, 8, 8, 3, 1, 1)
    gw, gb = filled(16, 3, 3), filled(16)
    B.dwconv2d_bwd_nhwc(d, None, None, None, None, gw, gb, room(B.dwconv2d_bwd_nhwc_workspace_size(d)))
    assert bool((gw == 0).all()) and bool((gb == 0).all())
    d, x, w, gy = conv_inputs(3, 70, 30, 31, 3, 1, 1, 1, 1, "bf16", 8)
    a, b = run_conv(d, x, gy, w, "bf16"), run_conv(d, x, gy, w, "bf16")
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_conv_backward_nan_stays_in_its_channel():
    d, x, w, gy = conv_inputs(2, 36, 9, 9, 3, 1, 1, 1, 1, "f32", 6)
    x[1, 4, 4, 3] = float("nan")
    gy[0, 2, 2, 5] = float("inf")
    gx, gw, gb = run_conv(d, x, gy, w, "f32")
    bad = torch.zeros(36, dtype=torch.bool, device="cuda")
    bad[[3, 5]] = True
    assert bool((~gw.isfinite()).any((1, 2)).eq(bad).all())
    assert bool(gx[..., [c for c in range(36) if c != 5]].isfinite().all()) and not bool(gb[5].isfinite())


def test_conv_backward_beyond_32_bit_offsets():
    d = B.make_desc(9, 64, 2048, 1824, 3, 1, 1, 1, 1, "bf16")  # 2^31 elements and more, the last sample past 2^30 * 1.7
    x = torch.zeros(9, 2048, 1824, 64, dtype=torch.bfloat16, device="cuda")
    gy = torch.zeros_like(x)
    w = normal(gen(1), 64, 3, 3, dtype="bf16")
    x[-1, -6:] = normal(gen(2), 6, 1824, 64, dtype="bf16")
    gy[-1, -6:] = normal(gen(3), 6, 1824, 64, dtype="bf16", std=0.1)
    gx, gw, gb = run_conv(d, x, gy, w, "bf16")
    t = B.make_desc(1, 64, 8, 1824, 3, 1, 1, 1, 1, "bf16")
    rgx, rgw, rgb, sx, sw, sb = R.conv_bwd(x[-1:, -8:].double(), gy[-1:, -8:].double(), w.double(), t)
    R.within(gx[-1:, -6:], rgx[:, 2:], R.EPS32 * 16 * sx[:, 2:], "bf16", "gx tail")
    R.within(gw, rgw, R.EPS32 * 4096 * sw, "bf16", "gw")
    R.within(gb, rgb, R.EPS32 * 4096 * sb, "bf16", "gb")
    assert bool((gx[:-1] == 0).all())


# ---- capture ---------------------------------------------------------------


def test_a_step_replays_from_a_graph():
    """Forward, norm with a checkpoint, norm backward and layer backward, captured once: bitwise the eager results."""
    N, H, W, C, G = 2, 28, 28, 64, 8
    dc = B.make_desc(N, C, H, W, 3, 1, 1, 1, 1, "bf16")
    dn = B.make_norm_desc(N, H, W, C, G, "silu", EPS, "bf16")
    _, x, w, gy = conv_inputs(N, C, H, W, 3, 1, 1, 1, 1, "bf16", 3)
    gamma, beta = normal(gen(5), C, dtype="bf16", mean=1.0, std=0.2), normal(gen(6), C, dtype="bf16")
    z, y, dz, gx = (filled(N, H, W, C, dtype="bf16") for _ in range(4))
    mean, rstd = filled(N, G), filled(N, G)
    gg, gb, gw, gcb = filled(C, dtype="bf16"), filled(C, dtype="bf16"), filled(C, 3, 3, dtype="bf16"), filled(C, dtype="bf16")
    x8, z8 = new_act8((N, H, W, C), "i8", 64), new_act8((N, H, W, C), "e4m3", 32)
    wf, wb = (room(B.dwconv2d_group_norm_nhwc_workspace_size(dn, p)) for p in (0, 1))
    wc = room(B.dwconv2d_bwd_nhwc_workspace_size(dc))
    outs = (z, y, dz, gx, mean, rstd, gg, gb, gw, gcb, x8.tensors[1], z8.tensors[1])

    def step(s):
        B.dwconv_act8_encode(x, x8, stream=s)
        B.dwconv2d_fwd_nhwc(dc, x, w, None, z, stream=s)
        B.dwconv2d_group_norm_nhwc(dn, z, gamma, beta, y, mean, rstd, wf, x8=z8, stream=s)
        B.dwconv2d_group_norm_nhwc_bwd(dn, None, gy, gamma, beta, mean, rstd, dz, gg, gb, wb, x8=z8, stream=s)
        B.dwconv2d_bwd_nhwc(dc, None, dz, w, gx, gw, gcb, wc, x8=x8, stream=s)

    step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for t in outs:
        t.fill_(-3)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, eager))
