"""Trains a channels-last depthwise block that keeps its activations in 8 bits.

  z = dwconv3x3(x, w) + b        dwconv2d_fwd_nhwc
  y = silu(group_norm(z))        dwconv2d_group_norm_nhwc, which writes z's checkpoint on its way
  loss = mean (y - target)^2 / 2

Between forward and backward the block keeps 8-bit checkpoints of x and z
instead of the tensors; both backward calls read them:

  (y - target) / n -> dz, dgamma, dbeta    dwconv2d_group_norm_nhwc_bwd
  dz -> dx, dw, db                         dwconv2d_bwd_nhwc

The target is what another block with weights of its own makes of the same
inputs. Run: python examples/train_block.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from depthwise_convolution_dwconv2d_gb300 import binding as B  # noqa: E402
from depthwise_convolution_dwconv2d_gb300 import build  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class NormBlock:
    """A depthwise 3x3 layer, group norm and SiLU over [N, H, W, C]. keep: "none" (activations in full), "i8" or "e4m3"."""

    def __init__(self, N, H, W, C, groups, dtype="bf16", keep="i8", block=64, seed=0):
        self.keep, self.dtype = keep, DTYPES[dtype]
        self.conv = B.make_desc(N, C, H, W, 3, 1, 1, 1, 1, dtype)
        self.norm = B.make_norm_desc(N, H, W, C, groups, "silu", 1e-5, dtype)
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g, device="cuda") * std + mean  # noqa: E731
        # weights are stepped in fp32 and used in the block's type
        self.master = [make(C, 3, 3, std=1 / 3), make(C, std=0.1), make(C, std=0.2, mean=1.0), make(C, std=0.2)]
        self.weights = [m.to(self.dtype) for m in self.master]
        self.grads = [torch.empty_like(w) for w in self.weights]
        empty = lambda *s, t=self.dtype: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.z, self.y, self.dz, self.dx = (empty(N, H, W, C) for _ in range(4))
        self.mean, self.rstd = empty(N, groups, t=torch.float32), empty(N, groups, t=torch.float32)
        room = lambda n: empty(max(n, 16), t=torch.uint8)  # noqa: E731
        self.ws = [room(B.dwconv2d_group_norm_nhwc_workspace_size(self.norm, p)) for p in (0, 1)]
        self.ws.append(room(B.dwconv2d_bwd_nhwc_workspace_size(self.conv)))
        self.x8 = self.z8 = self.x = None
        if keep != "none":
            code = torch.int8 if keep == "i8" else torch.float8_e4m3fn
            self.x8, self.z8 = (B.make_act8(keep, block, empty(N, H, W, C, t=code),
                                            empty(N, H, W, -(-C // block), t=torch.float32)) for _ in range(2))

    def forward(self, x):
        w, b, gamma, beta = self.weights
        if self.x8 is not None:
            B.dwconv_act8_encode(x, self.x8)
        else:
            self.x = x
        B.dwconv2d_fwd_nhwc(self.conv, x, w, b, self.z)
        B.dwconv2d_group_norm_nhwc(self.norm, self.z, gamma, beta, self.y, self.mean, self.rstd, self.ws[0], x8=self.z8)
        return self.y

    def backward(self, gy):
        w, b, gamma, beta = self.weights
        gw, gb, ggamma, gbeta = self.grads
        full = self.z8 is None
        B.dwconv2d_group_norm_nhwc_bwd(self.norm, self.z if full else None, gy, gamma, beta, self.mean, self.rstd,
                                       self.dz, ggamma, gbeta, self.ws[1], x8=self.z8)
        B.dwconv2d_bwd_nhwc(self.conv, self.x if full else None, self.dz, w, self.dx, gw, gb, self.ws[2], x8=self.x8)
        return self.dx

    def step(self, rate):
        for m, w, g in zip(self.master, self.weights, self.grads):
            m.sub_(g.float(), alpha=rate)
            w.copy_(m)

    def kept_bytes(self):
        """What the block holds between forward and backward, beside its weights."""
        if self.z8 is None:
            return 2 * self.z.numel() * self.z.element_size()
        return sum(t.numel() * t.element_size() for a in (self.x8, self.z8) for t in a.tensors)


def train(steps=20, keep="i8", dtype="bf16", N=8, H=28, W=28, C=256, groups=16, rate=8.0):
    """Losses of `steps` steps."""
    build.build()
    teacher = NormBlock(N, H, W, C, groups, dtype, "none", seed=1)
    block = NormBlock(N, H, W, C, groups, dtype, keep, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for _ in range(steps):
        x = torch.randn(N, H, W, C, generator=g, device="cuda").to(DTYPES[dtype])
        off = block.forward(x).float() - teacher.forward(x).float()
        losses.append(float(off.square().mean() / 2))
        block.backward((off * (C / off.numel())).to(DTYPES[dtype]))  # per channel: a mean over its own values
        block.step(rate / 16)
    return losses, block


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 40
    for keep in ("none", "i8", "e4m3"):
        losses, block = train(steps, keep)
        print("kept %5s: %6.2f MB between forward and backward, loss %.5f -> %.5f" % (
            keep, block.kept_bytes() / 1e6, losses[0], losses[-1]))
