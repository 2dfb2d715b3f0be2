"""The training example: its loss falls, and 8-bit checkpoints train as the full activations do."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_block_trains_from_checkpoints(example):
    """The loss halves in forty steps; from 8-bit checkpoints it ends within a tenth of where full activations take it."""
    ends = {}
    for keep in ("none", "i8", "e4m3"):
        losses, block = example.train(40, keep, N=4, H=14, W=14, C=64, groups=8)
        assert losses[-1] < 0.5 * losses[0], (keep, losses)
        ends[keep] = losses[-1]
    assert abs(ends["i8"] / ends["none"] - 1) < 0.1 and abs(ends["e4m3"] / ends["none"] - 1) < 0.1, ends


def test_checkpoints_hold_half_the_bytes(example):
    full = example.NormBlock(2, 8, 8, 128, 8, "bf16", "none").kept_bytes()
    kept = example.NormBlock(2, 8, 8, 128, 8, "bf16", "i8", 64).kept_bytes()
    assert kept == full / 2 * (1 + 4 / 64)
