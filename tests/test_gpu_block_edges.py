"""The operators around a block's layers where their kernels' limits lie: pairs of thread blocks over several tiles, blocks
that follow one another on an SM, ranges beside ordinary values, long chains of additions (plain 64-bit forms: block_ref.py)."""
import pytest

torch = pytest.importorskip("torch")

import block_ref as K
import train_ref as R
from depthwise_convolution_dwconv2d_gb300 import binding as B
from test_gpu_block import EPS, _lib, _no_wait_gave_up, act8_of, filled, gen, normal, room, run_clip, weight8_of  # noqa: F401

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
