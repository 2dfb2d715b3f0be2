"""RMS norm, 8-bit 1x1 product and clipping on the GPU against plain 64-bit forms (block_ref.py)."""
import pytest

torch = pytest.importorskip("torch")

import block_ref as K
import train_ref as R
from depthwise_convolution_dwconv2d_gb300 import binding as B

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from depthwise_convolution_dwconv2d_gb300 import build
    build.build()
    B.load()


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    before = B.dwconv_device_timeouts()
    yield
    torch.cuda.synchronize()
    assert B.dwconv_device_timeouts() == before


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype="f32", std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(R.DT[dtype])


def filled(*shape, dtype="f32", value=-7.0):
    return torch.full(shape, value, dtype=R.DT[dtype], device="cuda")


def room(nbytes, guard=64):
    """A workspace with guard bytes behind it, and a check of them."""
    buf = torch.full((nbytes + guard,), 0x7f, dtype=torch.uint8, device="cuda")
    return buf[:nbytes], lambda: bool((buf[nbytes:] == 0x7f).all())


def new_act8(rows, C, block, kind="e4m3"):
    codes = torch.full((rows, C), 0x55, dtype=torch.uint8, device="cuda").view(torch.int8 if kind == "i8" else torch.float8_e4m3fn)
    return B.make_act8(kind, block, codes, torch.full((rows, -(-C // block)), -1.0, device="cuda"))


def act8_of(x, block=128):
    codes, scales = R.encode(x, "e4m3", block)
    return B.make_act8("e4m3", block, codes, scales)


def weight8_of(w):
    codes, scales = K.encode_weights(w)
    return B.make_weight8(*w.shape, codes, scales)


def offset_view(t, by=1):
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


# ---- RMS norm ---------------------------------------------------------------

# one channel, rows that end inside a vector, a warp, a block of codes; several warps to a row; rows read twice
SHAPES = [(1, 1), (3, 5), (7, 16), (1, 31), (5, 33), (33, 64), (9, 96), (2, 100), (4, 127), (257, 128), (6, 200), (3, 264),
          (130, 24), (2, 1000), (5, 1024), (2, 1030), (3, 2048), (1, 4096), (400, 4096), (2, 4100), (3, 5000), (2, 8192)]
WIDE = [(2, 9001), (3, 16400), (2, 40000)]


def check_fwd(rows, C, dtype, residual, want_h, want_y, kind, block, gamma=True, seed=0, eps=EPS, off=0):
    g = gen(seed + rows * 7919 + C)
    x = normal(g, rows, C, dtype=dtype)
    x *= torch.exp2(torch.randint(-6, 6, (rows, 1), generator=g, device="cuda").float()).to(x.dtype)
    res = normal(g, rows, C, dtype=dtype, std=3.0) if residual else None
    gm = normal(g, C, dtype=dtype, std=0.2, mean=1.0) if gamma else None
    if off:
        x, res, gm = (t if t is None else offset_view(t, off) for t in (x, res, gm))
    h = filled(rows, C, dtype=dtype) if want_h else None
    y = filled(rows, C, dtype=dtype) if want_y else None
    rstd = filled(rows)
    y8 = new_act8(rows, C, block, kind) if kind else None
    B.dwconv_rms_norm(B.make_rms_desc(rows, C, eps, dtype), x, res, gm, h, y, rstd, y8)
    wh, wr, wy = K.rms_fwd(x, res, gm, eps, dtype)
    if want_h:
        assert torch.equal(h, wh), (rows, C)
    assert bool(((rstd.double() - wr).abs() <= K.slack_rstd(wr)).all()), (rows, C)
    if want_y:
        R.within(y, wy, K.slack_y(wy), dtype, f"y {rows}x{C}")
    if kind:
        check_codes(y8, wy, kind, block, (rows, C))


def check_codes(y8, wy, kind, block, what):
    """Scales are the blocks' maxima, codes the nearest: half an e4m3 step of the value (2^-4, below the smallest exponent
    half of 2^-9 of the scale), or half an integer step."""
    codes, scales = y8.tensors
    C = wy.shape[-1]
    nb = -(-C // block)
    amax = torch.nn.functional.pad(wy.abs(), (0, nb * block - C)).reshape(-1, nb, block).amax(-1)
    want = amax / R.CODE_MAX[kind]
    assert bool(((scales.double() - want).abs() <= K.slack_y(want) + 2 * K.U * want).all()), what
    s = scales.double().repeat_interleave(block, -1)[:, :C]
    v = codes.double() * s
    half = 0.5 * s if kind == "i8" else torch.maximum(2.0 ** -4 * wy.abs(), 2.0 ** -10 * s)
    over = (v - wy).abs() - half * (1 + 2 ** -10) - 2 * K.slack_y(s * R.CODE_MAX[kind])
    assert float(over.max()) <= 0, what


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rms_norm(dtype, residual):
    for rows, C in SHAPES + WIDE:
        check_fwd(rows, C, dtype, residual, want_h=residual, want_y=True, kind=None, block=0)


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rms_norm_to_codes(dtype, kind, block):
    for i, (rows, C) in enumerate(SHAPES + WIDE):
        check_fwd(rows, C, dtype, residual=i % 2 == 0, want_h=i % 3 == 0, want_y=i % 4 == 0, kind=kind, block=block, gamma=i % 5 != 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rms_norm_pointers_off_16_bytes(dtype):
    for rows, C in ((5, 64), (3, 128), (2, 1024), (2, 4096), (2, 16384)):
        check_fwd(rows, C, dtype, True, True, True, "e4m3", 128, off=1)


def test_rms_norm_many_narrow_rows():
    for C, dtype in ((8, "bf16"), (17, "f16"), (128, "bf16"), (96, "f32")):
        check_fwd(70001, C, dtype, True, True, True, None, 0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rms_norm_ragged_rows_in_several_rounds(dtype):
    """Rows off 16 bytes, more of them than blocks take at once: the tensor's first and last rows and those between."""
    for i, (rows, C) in enumerate(((17, 513), (900, 515), (701, 1030), (950, 2031), (640, 2047), (4001, 217), (70001, 3), (6000, 437))):
        check_fwd(rows, C, dtype, i % 2 == 0, want_h=i % 3 != 1, want_y=True, kind=None, block=0, gamma=i % 4 != 3, off=i % 3)


@pytest.mark.parametrize("kind,block", [("e4m3", 128), ("i8", 32)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rms_norm_ragged_rows_to_codes(dtype, kind, block):
    for i, (rows, C) in enumerate(((17, 130), (5000, 218), (3000, 505), (2500, 723), (2001, 1013), (300, 1031), (9000, 31), (40000, 5))):
        check_fwd(rows, C, dtype, i % 2 == 0, want_h=i % 3 != 1, want_y=i % 2 == 1, kind=kind, block=block, gamma=i % 4 != 3)


def test_rms_norm_slices_and_codes_at_any_byte():
    """Codes whose rows do not lie as x's do, or begin at an odd byte: no byte around them is written."""
    for rows, C, xo, xt, by, dtype, block in ((700, 205, 3, 219, 0, "bf16", 32), (700, 205, 0, 0, 3, "f16", 64), (1000, 131, 0, 133, 1, "f32", 128),
                                              (900, 128, 0, 0, 5, "bf16", 128), (650, 2100, 1, 2101, 2, "bf16", 32), (1, 7, 2, 9, 1, "f16", 32)):
        g = gen(C)
        x = torch.full((rows, xt or C), float("nan"), dtype=R.DT[dtype], device="cuda")
        x[:, xo:xo + C] = normal(g, rows, C, dtype=dtype)
        gm = normal(g, C, dtype=dtype)
        buf = torch.full((rows * C + by + 64,), 0x55, dtype=torch.uint8, device="cuda")
        codes = buf[by:by + rows * C].view(rows, C).view(torch.float8_e4m3fn)
        y8 = B.make_act8("e4m3", block, codes, torch.full((rows, -(-C // block)), -1.0, device="cuda"))
        B.dwconv_rms_norm(B.make_rms_desc(rows, C, EPS, dtype, xo, xt), x, None, gm, None, None, None, y8)
        check_codes(y8, K.rms_fwd(x[:, xo:xo + C], None, gm, EPS, dtype)[2], "e4m3", block, (rows, C))
        assert bool((buf[:by] == 0x55).all()) and bool((buf[by + rows * C:] == 0x55).all())


def test_rms_norm_special_values_in_ragged_rows():
    """Infinities, NaN and zeros stay in their rows and blocks where blocks begin inside a vector."""
    x = normal(gen(1), 40, 333, dtype="bf16")
    x[21] = 0
    x[22, 100] = float("inf")
    x[23, 332] = float("nan")
    y, rstd, y8 = filled(40, 333, dtype="bf16"), filled(40), new_act8(40, 333, 32)
    B.dwconv_rms_norm(B.make_rms_desc(40, 333, EPS, "bf16"), x, None, None, None, y, rstd, y8)
    codes, scales = y8.tensors
    assert bool((y[21] == 0).all()) and bool(scales[21].eq(0).all())
    assert float(rstd[22]) == 0 and bool(scales[22, 3].isnan()) and int(scales[22].isnan().sum()) == 1
    assert bool(y[23].isnan().all()) and bool(scales[23].isnan().all())
    rest = [r for r in range(40) if r not in (22, 23)]
    assert bool(y[rest].isfinite().all()) and bool(scales[rest].isfinite().all())
    B.dwconv_rms_norm(B.make_rms_desc(40, 333, 0.0, "bf16"), x, None, None, None, None, rstd, y8)
    assert bool(scales[21].isnan().all()) and bool(scales[[20, 24]].isfinite().all())


def test_rms_norm_in_place_ragged():
    """Reads that reach over a row's ends while the rows beside it are written: the same results."""
    for rows, C, dtype in ((5000, 77, "bf16"), (700, 2131, "f16"), (3000, 501, "f32")):
        g = gen(C)
        x, res, gm = normal(g, rows, C, dtype=dtype), normal(g, rows, C, dtype=dtype), normal(g, C, dtype=dtype)
        d = B.make_rms_desc(rows, C, EPS, dtype)
        h, y = filled(rows, C, dtype=dtype), filled(rows, C, dtype=dtype)
        B.dwconv_rms_norm(d, x, res, gm, h, y)
        for k in range(2):
            a, b, z = x.clone(), res.clone(), filled(rows, C, dtype=dtype)
            B.dwconv_rms_norm(d, a, b, gm, (a, b)[k], z)
            assert torch.equal((a, b)[k], h) and torch.equal(z, y)
        gx, rstd = filled(rows, C, dtype=dtype), filled(rows)
        B.dwconv_rms_norm(d, x, res, gm, None, y, rstd)
        B.dwconv_rms_norm_bwd(d, h, y, gm, rstd, res, gx, None, None)
        B.dwconv_rms_norm_bwd(d, h, y, gm, rstd, res, res, None, None)
        assert torch.equal(res, gx)


def test_rms_norm_in_place():
    """h over x or over the residual, rows kept in registers and rows read twice: the same results."""
    for rows, C, dtype in ((5, 200, "bf16"), (3, 4096, "f16"), (2, 40000, "bf16"), (2, 9001, "f32")):
        g = gen(C)
        x, res, gm = normal(g, rows, C, dtype=dtype), normal(g, rows, C, dtype=dtype), normal(g, C, dtype=dtype)
        d = B.make_rms_desc(rows, C, EPS, dtype)
        h, y = filled(rows, C, dtype=dtype), filled(rows, C, dtype=dtype)
        B.dwconv_rms_norm(d, x, res, gm, h, y)
        for k in range(2):
            a, b, z = x.clone(), res.clone(), filled(rows, C, dtype=dtype)
            B.dwconv_rms_norm(d, a, b, gm, (a, b)[k], z)
            assert torch.equal((a, b)[k], h) and torch.equal(z, y)


def test_rms_norm_slices():
    """Channels of wider rows: what lies between is neither read nor written."""
    for rows, C, xo, xt, yo, yt, dtype in ((5, 64, 8, 96, 16, 128, "bf16"), (4, 40, 3, 50, 1, 47, "f32"), (3, 200, 0, 201, 5, 300, "f16")):
        g = gen(C)
        x, res = (torch.full((rows, xt), float("nan"), dtype=R.DT[dtype], device="cuda") for _ in range(2))
        x[:, xo:xo + C], res[:, xo:xo + C] = normal(g, rows, C, dtype=dtype), normal(g, rows, C, dtype=dtype)
        gm = normal(g, C, dtype=dtype)
        h, y, rstd = filled(rows, xt, dtype=dtype), filled(rows, yt, dtype=dtype), filled(rows)
        d = B.make_rms_desc(rows, C, EPS, dtype, xo, xt, yo, yt)
        B.dwconv_rms_norm(d, x, res, gm, h, y, rstd)
        xc, rc = x[:, xo:xo + C], res[:, xo:xo + C]
        wh, wr, wy = K.rms_fwd(xc, rc, gm, EPS, dtype)
        assert torch.equal(h[:, xo:xo + C], wh)
        R.within(y[:, yo:yo + C], wy, K.slack_y(wy), dtype)
        h[:, xo:xo + C], y[:, yo:yo + C] = -7, -7
        assert bool((h == -7).all()) and bool((y == -7).all())
        gy = torch.full((rows, yt), float("nan"), dtype=R.DT[dtype], device="cuda")
        gy[:, yo:yo + C] = normal(g, rows, C, dtype=dtype)
        gx, gg = filled(rows, xt, dtype=dtype), filled(C, dtype=dtype)
        hs = x.clone()
        hs[:, xo:xo + C] = wh
        ws, intact = room(B.dwconv_rms_norm_bwd_workspace_size(d))
        B.dwconv_rms_norm_bwd(d, hs, gy, gm, rstd, res, gx, gg, ws)
        wx, wg, sx, sg = K.rms_bwd(wh, gy[:, yo:yo + C], gm, rstd, rc)
        R.within(gx[:, xo:xo + C], wx, sx, dtype)
        R.within(gg, wg, sg, dtype)
        gx[:, xo:xo + C] = -7
        assert bool((gx == -7).all()) and intact()


@pytest.mark.parametrize("gres", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rms_norm_bwd(dtype, gres):
    for i, (rows, C) in enumerate(SHAPES + WIDE + [(5001, 40), (3000, 128), (1500, 77)]):
        g = gen(rows * 31 + C)
        h, gy = normal(g, rows, C, dtype=dtype, std=2.0), normal(g, rows, C, dtype=dtype, std=0.1)
        gm = normal(g, C, dtype=dtype, std=0.3, mean=1.0) if i % 4 != 3 else None
        gr = normal(g, rows, C, dtype=dtype, std=0.1) if gres else None
        if i % 5 == 4:
            h, gy = offset_view(h), offset_view(gy)
        rstd = torch.rsqrt(h.float().square().mean(-1) + EPS)
        d = B.make_rms_desc(rows, C, EPS, dtype)
        gx, gg = filled(rows, C, dtype=dtype), filled(C, dtype=dtype)
        ws, intact = room(B.dwconv_rms_norm_bwd_workspace_size(d))
        B.dwconv_rms_norm_bwd(d, h, gy, gm, rstd, gr, gx, gg, ws)
        wx, wg, sx, sg = K.rms_bwd(h, gy, gm, rstd, gr)
        R.within(gx, wx, sx, dtype, f"gx {rows}x{C}")
        R.within(gg, wg, sg, dtype, f"ggamma {rows}x{C}")
        assert intact()
        only = filled(rows, C, dtype=dtype)
        B.dwconv_rms_norm_bwd(d, h, gy, gm, rstd, gr, only, None, None)
        assert torch.equal(only, gx)
        again = filled(C, dtype=dtype)
        B.dwconv_rms_norm_bwd(d, h, gy, gm, rstd, gr, None, again, ws)
        if i % 5 == 4:  # h off 16 bytes and gx on them: which kernel runs depends on gx
            R.within(again, wg, sg, dtype, f"ggamma alone {rows}x{C}")
        else:
            assert torch.equal(again, gg)
        if gres:
            B.dwconv_rms_norm_bwd(d, h, gy, gm, rstd, gr, gr, None, None)  # over gres
            assert torch.equal(gr, gx)


def test_rms_norm_gradient_against_differences():
    """The loss sum(gy * y) moves by gx . d and ggamma . d for small steps d, as the 64-bit forward says."""
    rows, C = 7, 50
    g = gen(3)
    x, gy, gm = normal(g, rows, C), normal(g, rows, C), normal(g, C, mean=1.0)
    d = B.make_rms_desc(rows, C, 1e-3, "f32")
    y, rstd, gx, gg = filled(rows, C), filled(rows), filled(rows, C), filled(C)
    ws, _ = room(B.dwconv_rms_norm_bwd_workspace_size(d))
    B.dwconv_rms_norm(d, x, None, gm, None, y, rstd)
    B.dwconv_rms_norm_bwd(d, x, gy, gm, rstd, None, gx, gg, ws)

    def loss(xd, gd):
        return float((gy.double() * xd / torch.sqrt(xd.square().mean(-1, keepdim=True) + 1e-3) * gd).sum())

    step = 1e-5
    dx, dg = torch.randn(rows, C, generator=g, device="cuda").double(), torch.randn(C, generator=g, device="cuda").double()
    # a central difference is off by step^2 times third derivatives (of order 10 each here), and 2^-53 / step
    fx = (loss(x.double() + step * dx, gm.double()) - loss(x.double() - step * dx, gm.double())) / (2 * step)
    fg = (loss(x.double(), gm.double() + step * dg) - loss(x.double(), gm.double() - step * dg)) / (2 * step)
    assert abs(fx - float((gx.double() * dx).sum())) <= 1e-5 * float((gx.double() * dx).abs().sum()) + 1e-6
    assert abs(fg - float((gg.double() * dg).sum())) <= 1e-5 * float((gg.double() * dg).abs().sum()) + 1e-6


def test_rms_norm_special_values():
    """Zeros, infinities and NaN stay in their rows; codes of their blocks decode to NaN."""
    x = normal(gen(1), 6, 256, dtype="bf16")
    x[1] = 0
    x[2, 100] = float("inf")
    x[3, 200] = float("nan")
    y, rstd, y8 = filled(6, 256, dtype="bf16"), filled(6), new_act8(6, 256, 128)
    B.dwconv_rms_norm(B.make_rms_desc(6, 256, EPS, "bf16"), x, None, None, None, y, rstd, y8)
    assert bool((y[1] == 0).all()) and float(rstd[1]) == pytest.approx(1e3)
    assert float(rstd[2]) == 0 and bool(y[2, 100].isnan()) and int(y[2].isnan().sum()) == 1 and bool(y[3].isnan().all())
    for r in (0, 4, 5):
        assert bool(y[r].isfinite().all())
    scales = y8.tensors[1]
    assert bool(scales[2, 0].isnan()) and float(scales[2, 1]) == 0 and bool(scales[3].isnan().all()) and bool(scales[1] .eq(0).all())


def test_rms_norm_empty():
    d = B.make_rms_desc(0, 40, EPS, "bf16")
    B.dwconv_rms_norm(d, None, None, None, None, None)
    gg = filled(40, dtype="bf16")
    B.dwconv_rms_norm_bwd(d, None, None, None, None, None, None, gg, None)
    assert bool((gg == 0).all())


def test_rms_norm_beyond_32_bit_offsets():
    rows, C = (1 << 20) + 3, 2100  # more than 2^31 values
    x = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    x[-5:] = normal(gen(1), 5, C, dtype="bf16")
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    d = B.make_rms_desc(rows, C, EPS, "bf16")
    B.dwconv_rms_norm(d, x, None, None, None, y, rstd)
    _, _, wy = K.rms_fwd(x[-5:], None, None, EPS, "bf16")
    R.within(y[-5:], wy, K.slack_y(wy), "bf16")
    assert int(y[:-5].count_nonzero()) == 0
    gx, gg = torch.empty_like(x), filled(C, dtype="bf16")
    ws, intact = room(B.dwconv_rms_norm_bwd_workspace_size(d))
    B.dwconv_rms_norm_bwd(d, x, y, None, rstd, None, gx, gg, ws)
    wx, wg, sx, sg = K.rms_bwd(x[-5:], y[-5:], None, rstd[-5:], None)
    R.within(gx[-5:], wx, sx, "bf16")
    R.within(gg, wg, sg, "bf16")
    assert intact()


# ---- weights and the 1x1 product ----------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_weight8_codes_are_the_definition_bit_for_bit(dtype):
    for i, (o, k) in enumerate(((1, 1), (5, 17), (128, 128), (129, 127), (200, 300), (64, 1000), (513, 256))):
        w = normal(gen(i), o, k, dtype=dtype, std=0.1)
        if o > 128:
            w[128:] = 0
        for transpose in (0, 1):
            src = w.t().contiguous() if transpose else w
            codes = torch.full((o, B.weight8_pitch(k)), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            w8 = B.make_weight8(o, k, codes, torch.full((-(-o // 128), -(-k // 128)), -1.0, device="cuda"))
            B.dwconv_weight8_encode(src, w8, transpose)
            wc, ws = K.encode_weights(w)
            assert torch.equal(w8.tensors[1], ws), (o, k)
            assert torch.equal(codes.view(torch.uint8), wc.view(torch.uint8)), (o, k)


PRODUCTS = [(1, 1, 1), (1, 16, 8), (3, 17, 5), (16, 128, 128), (17, 128, 16), (2, 200, 333), (33, 256, 100), (64, 144, 130),
            (65, 512, 256), (100, 1000, 72), (128, 384, 260), (1, 4096, 4096), (40, 4096, 1024), (129, 128, 128), (130, 16, 8),
            (257, 160, 300), (300, 333, 77), (1000, 640, 256), (2295, 200, 333), (777, 1024, 520), (3136, 512, 1024), (20000, 64, 128)]


def check_product(rows, cin, cout, dtype, act="none", bias=True, x8=None, w8=None, seed=0):
    g = gen(seed + rows + 31 * cin + 977 * cout)
    if x8 is None:
        x8 = act8_of(normal(g, rows, cin) * torch.exp2(torch.randint(-8, 8, (rows, 1), generator=g, device="cuda").float()))
    if w8 is None:
        w8 = weight8_of(normal(g, cout, cin, std=cin ** -0.5))
    b = normal(g, cout, dtype=dtype) if bias else None
    y = filled(rows, cout, dtype=dtype)
    ws, intact = room(B.dwconv2d_pointwise8_workspace_size(rows, cin, cout))
    B.dwconv2d_pointwise8(x8, w8, b, act, y, ws)
    want, slack = K.product(*x8.tensors, *w8.tensors, b, act)
    R.within(y, want, slack, dtype, f"{rows}x{cin}->{cout} {act}")
    assert intact()
    return y


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_pointwise8(dtype):
    for i, (rows, cin, cout) in enumerate(PRODUCTS):
        check_product(rows, cin, cout, dtype, bias=i % 3 != 0)


@pytest.mark.parametrize("act", ["relu", "relu6", "silu", "gelu"])
def test_pointwise8_activations(act):
    for rows, cin, cout, dtype in ((5, 256, 200, "f32"), (300, 200, 130, "bf16"), (300, 256, 512, "f32"), (129, 128, 260, "f16")):
        check_product(rows, cin, cout, dtype, act)


def test_pointwise8_around_the_choice_of_kernel():
    """Pixels and channels on both sides of every bound between the kernels, and between their shapes."""
    for rows, cin, cout in ((16, 640, 130), (17, 640, 130), (32, 144, 200), (33, 144, 200), (64, 1280, 130), (65, 1280, 130), (64, 1152, 130),
                            (77, 1554, 1983), (301, 1290, 520), (384, 2048, 2048), (385, 2048, 2048), (1, 128 * 270, 64), (40, 128 * 130, 24),
                            (256, 1024, 256), (257, 1024, 257), (3105, 256, 1100), (4999, 1000, 1000)):
        check_product(rows, cin, cout, "bf16", "silu" if rows % 2 else "none")


def test_pointwise8_behind_its_copy():
    """Calls one after another that use one workspace, and read codes that the call before them writes: the same results."""
    rows = 2000
    g = gen(6)
    x, gm = normal(g, rows, 300), normal(g, 300, mean=1.0)
    x8, d = new_act8(rows, 300, 128), B.make_rms_desc(rows, 300, EPS, "f32")
    sizes = ((300, 200), (300, 77), (300, 1024))
    w8 = [weight8_of(normal(g, o, i, std=0.06)) for i, o in sizes]
    ys = [filled(rows, o) for _, o in sizes]
    ws, intact = room(max(B.dwconv2d_pointwise8_workspace_size(rows, i, o) for i, o in sizes))
    for _ in range(3):
        for t in ys:
            t.fill_(-7)
        x.mul_(-1.5)
        B.dwconv_rms_norm(d, x, None, gm, None, None, None, x8)
        for w, y in zip(w8, ys):
            B.dwconv2d_pointwise8(x8, w, None, "none", y, ws)
        for w, y in zip(w8, ys):
            want, slack = K.product(*x8.tensors, *w.tensors, None, "none")
            R.within(y, want, slack, "f32")
        assert intact()


def test_pointwise8_codes_at_any_byte():
    """Codes off 16 bytes (with and without channels that are), weights off 16 bytes."""
    for rows, cin, cout in ((5, 128, 64), (200, 256, 130), (150, 77, 40)):
        g = gen(rows)
        x8, w8 = act8_of(normal(g, rows, cin)), weight8_of(normal(g, cout, cin, std=0.1))
        want = check_product(rows, cin, cout, "f32", x8=x8, w8=w8)
        codes = offset_view(x8.tensors[0], 3)
        check_product(rows, cin, cout, "f32", x8=B.make_act8("e4m3", 128, codes, x8.tensors[1]), w8=w8)
        wc = offset_view(w8.tensors[0], 5)
        got = check_product(rows, cin, cout, "f32", x8=x8, w8=B.make_weight8(cout, cin, wc, w8.tensors[1]))
        assert got.shape == want.shape


def test_pointwise8_slices():
    for rows, cin, cout, off, total, dtype in ((5, 128, 64, 8, 96, "bf16"), (300, 128, 200, 3, 210, "f16"), (200, 64, 300, 4, 304, "f32")):
        g = gen(cout)
        x8, w8 = act8_of(normal(g, rows, cin)), weight8_of(normal(g, cout, cin, std=0.1))
        y = filled(rows, total, dtype=dtype)
        B.dwconv2d_pointwise8(x8, w8, None, "none", y, None, 0, off, total)
        want, slack = K.product(*x8.tensors, *w8.tensors, None, "none")
        R.within(y[:, off:off + cout], want, slack, dtype)
        y[:, off:off + cout] = -7
        assert bool((y == -7).all())


def test_pointwise8_reads_nothing_behind_its_rows():
    """Codes of NaN and infinite scales behind the last row and the last channel change nothing."""
    for rows, cin, cout in ((3, 144, 40), (130, 144, 40), (7, 100, 16), (200, 100, 16)):
        g = gen(rows)
        x8, w8 = act8_of(normal(g, rows, cin)), weight8_of(normal(g, cout, cin, std=0.1))
        codes, scales = x8.tensors
        big = torch.full((rows * cin + 4096,), 0x7f, dtype=torch.uint8, device="cuda")
        big[:rows * cin] = codes.view(torch.uint8).flatten()
        s2 = torch.full((scales.numel() + 512,), float("inf"), device="cuda")
        s2[:scales.numel()] = scales.flatten()
        y, z = filled(rows, cout), filled(rows, cout)
        ws, _ = room(B.dwconv2d_pointwise8_workspace_size(rows, cin, cout))
        B.dwconv2d_pointwise8(x8, w8, None, 0, y, ws)
        B.dwconv2d_pointwise8(B.make_act8("e4m3", 128, big.data_ptr(), s2.data_ptr(), rows, cin), w8, None, 0, z, ws)
        assert torch.equal(y, z) and bool(y.isfinite().all())


@pytest.mark.parametrize("rows", [4, 300])
def test_pointwise8_nan_scales(rows):
    """A pixel whose block overflowed gives NaN in its row alone; a block of weights that did, in its outputs alone."""
    x = normal(gen(2), rows, 256)
    x[1, 130] = float("inf")
    w = normal(gen(3), 300, 256)
    w[140, 5] = float("nan")
    x8 = act8_of(x)
    x8.tensors[1][1, 1] = float("nan")
    w8 = weight8_of(w)
    w8.tensors[1][1, 0] = float("nan")
    y = filled(rows, 300)
    B.dwconv2d_pointwise8(x8, w8, None, "none", y)
    assert bool(y[1].isnan().all()) and bool(y[:, 128:256].isnan().all())
    y[1], y[:, 128:256] = 0, 0
    assert bool(y.isfinite().all())


def test_pointwise8_empty():
    w8 = weight8_of(normal(gen(1), 16, 32))
    B.dwconv2d_pointwise8(B.make_act8("e4m3", 128, None, None, 0, 32), w8, None, "none", None, dtype="bf16")


def test_pointwise8_input_gradient():
    """gx = gy W from gy's codes and the weights encoded transposed, against the product of the values."""
    for rows, cin, cout in ((3, 128, 200), (500, 200, 144)):
        g = gen(rows)
        w, gy = normal(g, cout, cin, std=0.1), normal(g, rows, cout, std=0.02)
        w8 = B.make_weight8(cin, cout, torch.empty(cin, B.weight8_pitch(cout), dtype=torch.float8_e4m3fn, device="cuda"),
                            torch.empty(-(-cin // 128), -(-cout // 128), device="cuda"))
        B.dwconv_weight8_encode(w, w8, transpose=1)
        y8 = new_act8(rows, cout, 128)
        B.dwconv_act8_encode(gy, y8)
        gx = filled(rows, cin)
        ws, _ = room(B.dwconv2d_pointwise8_workspace_size(rows, cout, cin))
        B.dwconv2d_pointwise8(y8, w8, None, "none", gx, ws)
        values = R.decode(*y8.tensors, 128)
        wv = K.weight_values(*K.encode_weights(w), cin)
        slack = 2 * K.U * (264 + 8) * (values.abs() @ wv.abs())
        R.within(gx, values @ wv, slack, "f32")


def test_pointwise8_beyond_32_bit_offsets():
    rows, cin, cout = (1 << 19) + 5, 16, 4104  # y: more than 2^31 values
    x8 = act8_of(normal(gen(1), rows, cin))
    w8 = weight8_of(normal(gen(2), cout, cin))
    y = torch.empty(rows, cout, dtype=torch.bfloat16, device="cuda")
    B.dwconv2d_pointwise8(x8, w8, None, "none", y)
    for lo in (0, rows - 70):
        part = [t[lo:lo + 70] for t in x8.tensors]
        want, slack = K.product(*part, *w8.tensors, None, "none")
        R.within(y[lo:lo + 70], want, slack, "bf16")


# ---- clipping --------------------------------------------------------------------


def run_clip(grads, most, outs=None):
    lst = B.make_grads(grads, outs)
    ws, intact = room(B.dwconv_grad_norm_clip_workspace_size(lst))
    n = filled()
    B.dwconv_grad_norm_clip(lst, most, n, ws)
    assert intact()
    return n


SIZES = [[1], [5, 4096, 4097], [9 * 256, 256, 256, 256], [8191, 1, 0, 12345], [3] * 41, [70000] * 3 + [1] * 100, [17] * 1100, [5_000_000, 3]]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clip(dtype):
    for i, sizes in enumerate(SIZES):
        g = gen(i)
        grads = [normal(g, n, dtype=dtype, std=0.1 * 3 ** (k % 5)) for k, n in enumerate(sizes)]
        n, _ = K.clip(grads, 1.0)
        for most in (0.3 * float(n), 2 * float(n)):
            outs = [torch.full_like(t, -7) for t in grads]
            got = run_clip(grads, most, outs)
            n, want = K.clip(grads, most)
            assert abs(float(got) - float(n)) <= float(K.slack_norm(n)), sizes[:4]
            for o, w in zip(outs, want):
                R.within(o, w, 2 * K.slack_norm(w.abs()), dtype)
            again = [t.clone() for t in grads]
            run_clip(again, most)  # in place
            assert all(torch.equal(a, o) for a, o in zip(again, outs))


def test_clip_mixed_types_views_and_counted_only():
    """Tensors of several types, off 16 bytes, one that only counts; without clipping nothing changes."""
    g = gen(1)
    grads = [normal(g, 5000), offset_view(normal(g, 9000, dtype="bf16")), normal(g, 77, dtype="f16"), offset_view(normal(g, 4096))]
    n, want = K.clip(grads, 3.0)
    outs = [torch.full_like(grads[0], -7), offset_view(torch.full_like(grads[1], -7), 3), None, torch.full_like(grads[3], -7)]
    kept = grads[2].clone()
    got = run_clip(grads, 3.0, outs)
    assert abs(float(got) - float(n)) <= float(K.slack_norm(n)) and torch.equal(grads[2], kept)
    for o, w, t in zip(outs, want, ("f32", "bf16", "f16", "f32")):
        if o is not None:
            R.within(o, w, 2 * K.slack_norm(w.abs()), t)
    before = [t.clone() for t in grads]
    run_clip(grads, float("inf"))
    run_clip(grads, 2 * float(n))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_clip_beyond_the_range_of_squares():
    """Values whose squares leave fp32 on either side, beside ordinary ones and alone."""
    for dtype, big in (("f32", 1e30), ("bf16", 1e30), ("f32", 1e-30), ("bf16", 1e-30), ("f32", 1e-42)):
        g = gen(4)
        for std in (0.0, 1.0):
            grads = [normal(g, 10000, dtype=dtype, std=std), (torch.randn(5001, generator=g, device="cuda") * big).to(R.DT[dtype])]
            n, want = K.clip(grads, 0.5 * float(K.clip(grads, 1.0)[0]))
            outs = [torch.empty_like(t) for t in grads]
            most = 0.5 * float(n)
            got = run_clip(grads, most, outs) if most > 2 ** -149 else run_clip(grads, 1.0, outs)
            assert abs(float(got) - float(n)) <= float(K.slack_norm(n)) + 2.0 ** -149


def test_clip_infinities_and_nan():
    for bad in (float("inf"), float("nan")):
        g = normal(gen(1), 5000)
        g[77] = bad
        out = torch.empty_like(g)
        n = run_clip([g], 1.0, [out])
        assert not bool(n.isfinite())
        if bad == float("inf"):
            assert bool(n == bad) and bool(out[77].isnan()) and int(out.count_nonzero()) == 1
        else:
            assert bool(n.isnan()) and bool(out.isnan().all())


def test_clip_nothing():
    n = filled()
    B.dwconv_grad_norm_clip(B.make_grads([]), 1.0, n, None)
    assert float(n) == 0
    e = torch.empty(0, device="cuda")
    n = run_clip([e, e], 1.0)
    assert float(n) == 0


def test_clip_many_elements():
    """More than 2^31 elements in one tensor."""
    g = torch.full(((1 << 31) + 70001,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    g[-1] = 3.0
    n = run_clip([g], 1.0)
    want = ((g.numel() - 1) * 2.0 ** -20 + 9.0) ** 0.5
    assert abs(float(n) - want) <= float(K.slack_norm(torch.tensor(want)))
    k = 1.0 / want
    assert abs(float(g[-1]) - 3 * k) <= 2 ** -8 * 3 * k and abs(float(g[0]) - k * 2.0 ** -10) <= 2 ** -8 * k * 2.0 ** -10


# ---- together -----------------------------------------------------------------------


def block_step(dev_graph=None):
    """A block's step: norm with the residual to codes, the 1x1 layer, a second norm's backward, gx through the transposed
    weights, the norm's backward, and clipping of what has gradients."""
    rows, C, O = 700, 256, 384
    g = gen(9)
    t = {k: normal(g, *s, dtype="bf16", std=d) for k, (s, d) in dict(
        x=((rows, C), 1.0), res=((rows, C), 2.0), w=((O, C), 0.06), bias=((O,), 0.1), gy=((rows, O), 0.02), gres=((rows, C), 0.02)).items()}
    t["gamma"] = normal(g, C, dtype="bf16", std=0.1, mean=1.0)
    d = B.make_rms_desc(rows, C, EPS, "bf16")
    t.update(h=filled(rows, C, dtype="bf16"), rstd=filled(rows), y=filled(rows, O, dtype="bf16"), gh=filled(rows, C, dtype="bf16"),
             gx=filled(rows, C, dtype="bf16"), gg=filled(C, dtype="bf16"), norm=filled())
    x8, y8 = new_act8(rows, C, 128), new_act8(rows, O, 128)
    w8, wt8 = (B.make_weight8(o, i, torch.empty(o, B.weight8_pitch(i), dtype=torch.float8_e4m3fn, device="cuda"),
                              torch.empty(-(-o // 128), -(-i // 128), device="cuda")) for o, i in ((O, C), (C, O)))
    lst = B.make_grads([t["gg"]])
    ws = room(B.dwconv_rms_norm_bwd_workspace_size(d))[0]
    cs = room(B.dwconv_grad_norm_clip_workspace_size(lst))[0]

    def step():
        B.dwconv_weight8_encode(t["w"], w8)
        B.dwconv_weight8_encode(t["w"], wt8, transpose=1)
        B.dwconv_rms_norm(d, t["x"], t["res"], t["gamma"], t["h"], None, t["rstd"], x8)
        B.dwconv2d_pointwise8(x8, w8, t["bias"], "none", t["y"])
        B.dwconv_act8_encode(t["gy"], y8)
        B.dwconv2d_pointwise8(y8, wt8, None, "none", t["gh"])
        B.dwconv_rms_norm_bwd(d, t["h"], t["gh"], t["gamma"], t["rstd"], t["gres"], t["gx"], t["gg"], ws)
        B.dwconv_grad_norm_clip(lst, 0.01, t["norm"], cs)

    return t, x8, y8, w8, wt8, step


def test_a_block_of_them():
    """Each step of a block against its 64-bit form from what the step before it left."""
    t, x8, y8, w8, wt8, step = block_step()
    step()
    h, r, y = K.rms_fwd(t["x"], t["res"], t["gamma"], EPS, "bf16")
    assert torch.equal(t["h"], h)
    check_codes(x8, y, "e4m3", 128, "block")
    want, slack = K.product(*x8.tensors, *w8.tensors, t["bias"], "none")
    R.within(t["y"], want, slack, "bf16")
    want, slack = K.product(*y8.tensors, *wt8.tensors, None, "none")
    R.within(t["gh"], want, slack, "bf16")
    gx, gg, sx, sg = K.rms_bwd(t["h"], t["gh"], t["gamma"], t["rstd"], t["gres"])
    R.within(t["gx"], gx, sx, "bf16")
    unclipped = filled(256, dtype="bf16")
    B.dwconv_rms_norm_bwd(B.make_rms_desc(700, 256, EPS, "bf16"), t["h"], t["gh"], t["gamma"], t["rstd"], None, None, unclipped,
                          room(B.dwconv_rms_norm_bwd_workspace_size(B.make_rms_desc(700, 256, EPS, "bf16")))[0])
    R.within(unclipped, gg, sg, "bf16")
    n, clipped = K.clip([unclipped], 0.01)
    assert float(n) > 0.01 and abs(float(t["norm"]) - float(n)) <= float(K.slack_norm(n))
    R.within(t["gg"], clipped[0], 2 * K.slack_norm(clipped[0].abs()), "bf16")


def test_a_captured_block():
    """The same step captured into a graph, on a stream of its own, replayed on other inputs: bitwise the eager results."""
    t, x8, y8, w8, wt8, step = block_step()
    step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for k in ("x", "gy", "w"):
        t[k].mul_(-0.5)
    names = ("h", "rstd", "y", "gh", "gx", "gg", "norm")
    step()
    torch.cuda.synchronize()
    want = {k: t[k].clone() for k in names}
    codes = x8.tensors[0].view(torch.uint8).clone()
    for k in names:
        t[k].fill_(-7)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t[k], want[k]) for k in names) and torch.equal(x8.tensors[0].view(torch.uint8), codes)


def test_two_streams_at_once():
    """Products and clips on two streams at the same time, each with its own workspace, give what they give alone."""
    cases = []
    for i, (rows, cin, cout) in enumerate(((5, 2048, 512), (900, 500, 300), (40, 512, 2048), (3000, 256, 512))):
        g = gen(i)
        x8, w8 = act8_of(normal(g, rows, cin)), weight8_of(normal(g, cout, cin, std=0.1))
        ws = room(B.dwconv2d_pointwise8_workspace_size(rows, cin, cout))[0]
        grads = [normal(g, 100_000 + i)]
        outs = [torch.empty_like(grads[0])]
        lst = B.make_grads(grads, outs)
        cs = room(B.dwconv_grad_norm_clip_workspace_size(lst))[0]
        cases.append((x8, w8, ws, filled(rows, cout), lst, cs, filled(), outs[0]))

    def one(c):
        B.dwconv2d_pointwise8(c[0], c[1], None, "none", c[3], c[2])
        B.dwconv_grad_norm_clip(c[4], 1.0, c[6], c[5])

    for c in cases:
        one(c)
    torch.cuda.synchronize()
    want = [(c[3].clone(), c[7].clone()) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c in cases:
            c[3].fill_(-7)
            c[7].fill_(-7)
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i % 2]):
                one(c)
        torch.cuda.synchronize()
        assert all(torch.equal(c[3], y) and torch.equal(c[7], o) for c, (y, o) in zip(cases, want))
