"""The bounds that the group norm's gradients are held to notice a missing sum: planted in the formula, on the CPU."""
import pytest

torch = pytest.importorskip("torch")

import train_bounds as T
import train_ref as R

# N, H, W, C, G: slabs, streams, slices wider than a block, channels that no vector divides
SHAPES = [(3, 7, 7, 64, 32), (2, 19, 23, 40, 4), (4, 28, 28, 128, 1), (1, 64, 65, 24, 3), (1, 128, 128, 16, 2), (1, 9, 9, 2056, 1),
          (5, 11, 3, 33, 11), (1, 200, 150, 8, 1), (2, 56, 56, 128, 32), (1, 5, 4, 1031, 1), (2, 4, 5, 1044, 2)]


@pytest.mark.parametrize("act", ["none", "relu6", "silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_forgotten_sum_is_far_over_the_bounds(dtype, act):
    for i, shape in enumerate(SHAPES):
        x, gamma, beta, gy = T.inputs(*shape, dtype, i, "cpu")
        mean, rstd = R.moments(x.double(), shape[-1], 1e-5)
        args = [t.double() for t in (x, gy, gamma, beta, mean, rstd)] + [act]
        (gx, _, _), (egx, _, _) = T.backward(*args)
        slack = egx + R.ROUND[dtype] * gx.abs() + R.STEP[dtype]
        for lost in ("s1", "s2"):
            wrong = T.backward(*args, without=lost)[0][0]
            assert float(((wrong - gx).abs() / slack).max()) > 16, (shape, lost)
            assert float((wrong - gx).abs().gt(slack).double().mean()) > 0.5, (shape, lost)
