"""The operators around a block's layers where their kernels' limits lie: pairs of thread blocks over several tiles, blocks
that follow one another on an SM, ranges beside ordinary values, long chains of additions (plain 64-bit forms: block_ref.py)."""
import pytest

torch = pytest.importorskip("torch")

import block_ref as K
from block_pairs import PAIRS
import train_ref as R
from depthwise_convolution_dwconv2d_gb300 import binding as B
from test_gpu_block import EPS, _lib, _no_wait_gave_up, act8_of, check_product, filled, gen, normal, offset_view, room, run_clip, weight8_of  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- products by pairs of thread blocks -------------------------------------------


def test_pairs_leave_nothing_behind():
    """Blocks that follow a pair at once on its SMs, in its shared memory: pairs (one tile and several each), tiles, rows,
    norms and clips one after another on two streams, a hundred times, give bitwise what each gave by itself."""
    g = gen(1)
    calls = []
    for rows, cin, cout in ((2816, 896, 2816), (3136, 512, 1024), (900, 512, 300), (16, 2048, 512)):
        x8, w8 = act8_of(normal(g, rows, cin)), weight8_of(normal(g, cout, cin, std=0.05))
        y = filled(rows, cout, dtype="bf16")
        calls.append((lambda x8=x8, w8=w8, y=y: B.dwconv2d_pointwise8(x8, w8, None, "none", y), y))
    x, y = normal(g, 3000, 512, dtype="bf16"), filled(3000, 512, dtype="bf16")
    d = B.make_rms_desc(3000, 512, EPS, "bf16")
    calls.insert(1, (lambda: B.dwconv_rms_norm(d, x, None, None, None, y), y))
    grads = [normal(g, 20000)]
    out = [filled(20000)]
    lst = B.make_grads(grads, out)
    ws = room(B.dwconv_grad_norm_clip_workspace_size(lst))[0]
    calls.insert(3, (lambda: B.dwconv_grad_norm_clip(lst, 1.0, None, ws), out[0]))
    want = []
    for call, o in calls:
        call()
        torch.cuda.synchronize()
        want.append(o.clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    halves = calls[0::2], calls[1::2]
    for _ in range(100):
        for s, part in zip(streams, halves):
            with torch.cuda.stream(s):
                for call, _o in part:
                    call()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for (_, o), w in zip(calls, want))


@pytest.mark.parametrize("rows,cin,cout,dtype,act,rounds", PAIRS)
def test_pairs(rows, cin, cout, dtype, act, rounds):
    y = check_product(rows, cin, cout, dtype, act)
    assert torch.equal(check_product(rows, cin, cout, dtype, act), y)


def test_pairs_to_slices():
    """Several tiles per pair into channels of wider rows, in vectors and in pieces: what lies between is not written."""
    rows, cin, cout = 2700, 896, 2816
    g = gen(2)
    x8, w8 = act8_of(normal(g, rows, cin)), weight8_of(normal(g, cout, cin, std=0.05))
    want, slack = K.product(*x8.tensors, *w8.tensors, None, "none")
    for off, total, dtype in ((16, 2848, "bf16"), (3, 2823, "f16"), (8, 2832, "f32")):
        y = filled(rows, total, dtype=dtype)
        B.dwconv2d_pointwise8(x8, w8, None, "none", y, None, 0, off, total)
        R.within(y[:, off:off + cout], want, slack, dtype)
        y[:, off:off + cout] = -7
        assert bool((y == -7).all())


# ---- RMS norm, backward ------------------------------------------------------------


@pytest.mark.parametrize("size,gsize", [(2.0 ** 50, 2.0 ** 83), (2.0 ** -56, 2.0 ** -83)])
def test_rms_norm_bwd_keeps_its_range_in_every_kernel(size, gsize):
    """t * h leaves fp32 (or its normal numbers) where t * (h r) does not: rows in registers, rows that do not begin alike,
    rows too wide, with gamma and without."""
    for rows, C, dtype, apart, gamma in ((5, 200, "f32", False, True), (5, 200, "f32", True, True), (4, 77, "bf16", True, False),
                                         (300, 96, "bf16", True, True), (2, 40000, "bf16", False, True), (3, 9001, "f32", False, False)):
        g = gen(C)
        h, gy = normal(g, rows, C, std=size).to(R.DT[dtype]), normal(g, rows, C, std=gsize).to(R.DT[dtype])
        gm = normal(g, C, dtype=dtype, std=0.2, mean=1.0) if gamma else None
        rstd = (1 / torch.sqrt(h.double().square().mean(-1))).float()
        if apart:
            h = offset_view(h)
        d = B.make_rms_desc(rows, C, 0.0, dtype)
        gx, gg = filled(rows, C, dtype=dtype), filled(C, dtype=dtype)
        ws, intact = room(B.dwconv_rms_norm_bwd_workspace_size(d))
        B.dwconv_rms_norm_bwd(d, h, gy, gm, rstd, None, gx, gg, ws)
        wx, wg, sx, sg = K.rms_bwd(h, gy, gm, rstd, None)
        R.within(gx, wx, sx, dtype, f"gx {rows}x{C}")
        R.within(gg, wg, sg, dtype, f"ggamma {rows}x{C}")
        assert intact()


@pytest.mark.parametrize("rows,C,dtype,apart", [(7_600_000, 7, "f32", False), (1_000_003, 7, "f32", True), (160_000, 1032, "bf16", False),
                                                (300_001, 77, "f16", False), (70_000, 77, "f16", True), (120_000_001, 1, "bf16", False),
                                                (20_000, 9001, "bf16", False)])
def test_rms_norm_bwd_long_chains(rows, C, dtype, apart):
    """ggamma where a thread adds up hundreds to thousands of rows. Of small whole numbers every partial sum is exact in 32
    bits, so no row may be missing or counted twice. Of others: at most 4096 additions in a thread, 64 rows of a block and
    join's 16 + 7 behind them, a product and r's per term."""
    g = gen(C)
    d = B.make_rms_desc(rows, C, EPS, dtype)
    ws, intact = room(B.dwconv_rms_norm_bwd_workspace_size(d))

    def ggamma(h, gy, rstd):
        if apart:
            h = offset_view(h)
        gg = filled(C, dtype=dtype)
        B.dwconv_rms_norm_bwd(d, h, gy, None, rstd, None, None, gg, ws)
        assert intact()
        return gg

    h = (2 * torch.randint(0, 2, (rows, C), generator=g, device="cuda", dtype=torch.int8) - 1).to(R.DT[dtype])
    gy = torch.randint(-1, 2, (rows, C), generator=g, device="cuda", dtype=torch.int8).to(R.DT[dtype])
    exact = (h.to(torch.int8) * gy.to(torch.int8)).sum(0, dtype=torch.int64)
    assert int(exact.abs().max()) < 2 ** 24
    assert torch.equal(ggamma(h, gy, torch.ones(rows, device="cuda")), exact.float().to(R.DT[dtype]))
    h *= 1 + torch.rand(C, generator=g, device="cuda").to(h.dtype)
    rstd = 0.5 + torch.rand(rows, generator=g, device="cuda")
    got = ggamma(h, gy, rstd)
    want, size = (torch.stack([f(gy[:, c].double() * (h[:, c].double() * rstd.double())).sum() for c in range(C)]) for f in (lambda v: v, torch.abs))
    R.within(got, want, (4096 + 64 + 16 + 7 + 3) * K.U * size, dtype)


# ---- clipping -----------------------------------------------------------------------


@pytest.mark.parametrize("dtype,big", [("f32", 1e30), ("bf16", 1e30), ("f32", 1e-30), ("bf16", 1e-30), ("f32", 1e-42), ("f16", 6e-8)])
def test_clip_scales_what_lies_beyond_the_range_of_squares(dtype, big):
    """Every out, where squares leave fp32 on either side: beside ordinary values and alone, clipped hard, little and not at all."""
    g = gen(4)
    for std in (0.0, 1.0):
        grads = [normal(g, 10000, dtype=dtype, std=std), (torch.randn(5001, generator=g, device="cuda") * big).to(R.DT[dtype])]
        n = float(K.clip(grads, 1.0)[0])
        for part in (0.5, 0.999, 2.0, 1e-3):
            most = float(torch.tensor(part * max(n, 1e-6)).float())
            want = K.clip(grads, most)[1]
            outs = [torch.full_like(t, -7) for t in grads]
            got = run_clip(grads, most, outs)
            assert abs(float(got) - n) <= float(K.slack_norm(n)) + 2.0 ** -149
            for o, w in zip(outs, want):
                R.within(o, w, 2 * K.slack_norm(w.abs()), dtype, f"{big} {std} {part}")


@pytest.mark.parametrize("sizes", [[5000, 77], [700_000, 77]])  # in one cluster, in two launches
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_clip_by_infinity_changes_no_other_gradient(sizes, bad):
    """max_norm INFINITY: an infinity or a NaN shows in the norm and stays where it is; all else is written as it was."""
    for dtype in ("f32", "f16", "bf16"):
        g = gen(1)
        grads = [normal(g, n, dtype=dtype) for n in sizes]
        grads[0][77] = bad
        outs = [torch.full_like(t, -7) for t in grads]
        n = run_clip(grads, float("inf"), outs)
        assert bool(n.isnan()) if bad != bad else float(n) == float("inf")
        for o, t in zip(outs, grads):
            assert torch.equal(o.nan_to_num(nan=123.0), t.nan_to_num(nan=123.0))
        before = [t.clone() for t in grads]
        run_clip(grads, float("inf"))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, before))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clip_around_the_choice_of_launches(dtype):
    """One cluster takes 128 units of 512 elements and 120 tensors: sizes on both sides, against 64 bits, repeated bitwise."""
    for sizes in ([65536], [65537], [512] * 120, [512] * 121, [500] * 119 + [4608], [500] * 119 + [4609], [131072], [70001, 3], [262145]):
        g = gen(len(sizes))
        grads = [normal(g, n, dtype=dtype, std=0.1) for n in sizes]
        most = float(torch.tensor(0.3 * float(K.clip(grads, 1.0)[0])).float())
        n, want = K.clip(grads, most)
        outs = [torch.full_like(t, -7) for t in grads]
        got = run_clip(grads, most, outs)
        assert abs(float(got) - float(n)) <= float(K.slack_norm(n)), sizes[-1]
        for o, w in zip(outs, want):
            R.within(o, w, 2 * K.slack_norm(w.abs()), dtype)
        again = [torch.full_like(t, -7) for t in grads]
        assert torch.equal(run_clip(grads, most, again), got) and all(torch.equal(a, o) for a, o in zip(again, outs))
