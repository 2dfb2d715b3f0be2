"""How far the group norm's kernels may be from the 64-bit formulas, from the
roundings that they chain (torch, any device).

Everything is counted in units of 2^-24, and the bounds are twice the
first-order sums. Mean and rstd are the kernels' own, so a bound holds what one
pass rounds and nothing of the moments':
  xh = (x - mean) * rstd      2 roundings, u = xh * gamma + beta 2 more
  sigmoid of v                ex2 and rcp of the special-function unit (2 and 1
                              units in the last place, results below 2^-126
                              flushed to 0), v and its sum with 1 rounded, v
                              from 3 roundings
  sums                        JOINED additions behind one value at most: the
                              rows of a lane, 256 row lanes, 256 blocks
"""
import math

import torch

import train_ref as R

JOINED = 512
GELU, CUBIC = 2 * math.sqrt(2 / math.pi), 0.044715


def sigmoid_of(u, name):
    """v and sigmoid(v) with act(u) = u sigmoid(v), and a = u dv/du. GELU's (1 + tanh(w)) / 2 is sigmoid(2 w), which keeps
    its digits in the negative tail, where 64 bits of the former leave an error of 2^-53."""
    v = u if name == "silu" else GELU * (u + CUBIC * u ** 3)
    return v, torch.sigmoid(v), u if name == "silu" else GELU * u * (1 + 3 * CUBIC * u * u)


def act(u, name):
    return u * sigmoid_of(u, name)[1] if name == "gelu" else R.act(u, name)


def act_slope(u, name):
    if name != "gelu":
        return R.act_slope(u, name)
    _, q, a = sigmoid_of(u, name)
    return q + q * (1 - q) * a


def act_errors(u, du, name):
    """Errors of act(u) and act'(u) where u is off by du."""
    if name not in ("silu", "gelu"):
        return du, torch.zeros_like(u)
    v, q, a = sigmoid_of(u, name)
    dq = q * (1 - q) * 3 * v.abs() + 8 * q + 2.0 ** -126 / R.EPS32
    return (act_slope(u, name).abs() * du + u.abs() * dq + act(u, name).abs(),
            1.2 * du + dq * (1 + a.abs()) + 6 * (q + a.abs() * q * (1 - q)))


def forward(x, gamma, beta, mean, rstd, name):
    """y and its bound, all in 64 bits."""
    C = x.shape[-1]
    xh = (x - R.per_channel(mean, C)) * R.per_channel(rstd, C)
    u = xh * gamma + beta
    dy, _ = act_errors(u, 3 * (xh * gamma).abs() + u.abs(), name)
    return act(u, name), 2 * R.EPS32 * dy


def backward(x, gy, gamma, beta, mean, rstd, name, without=""):
    """(gx, ggamma, gbeta) and their bounds, all in 64 bits. without "s1" or "s2": a formula that forgets that sum."""
    N, H, W, C = x.shape
    G, m = mean.shape[1], H * W * C // mean.shape[1]
    rs = R.per_channel(rstd, C)
    xh = (x - R.per_channel(mean, C)) * rs
    u = xh * gamma + beta
    slope = act_slope(u, name)
    du = gy * slope
    _, dslope = act_errors(u, 3 * (xh * gamma).abs() + u.abs(), name)
    ddu = gy.abs() * (dslope + slope.abs())
    dh = xh.abs() * ddu + 3 * (xh * du).abs()  # of du * xh
    over = lambda v: R.per_channel(v.reshape(N, H * W, G, C // G).sum((1, 3)) / m, C)  # noqa: E731
    s1, s2 = over(gamma * du), over(gamma * du * xh)
    e1 = JOINED * over((gamma * du).abs()) + over(gamma.abs() * ddu)
    e2 = JOINED * over((gamma * du * xh).abs()) + over(gamma.abs() * dh)
    egx = rs * (gamma.abs() * ddu + 4 * (gamma * du).abs() + 4 * s1.abs() + 6 * (xh * s2).abs() + e1 + xh.abs() * e2)
    s1, s2 = (s1 * 0 if without == "s1" else s1), (s2 * 0 if without == "s2" else s2)
    gx = rs * (gamma * du - s1 - xh * s2)
    pixels = (0, 1, 2)
    egg = JOINED * (du * xh).abs().sum(pixels) + dh.sum(pixels)
    egb = JOINED * du.abs().sum(pixels) + ddu.sum(pixels)
    two = 2 * R.EPS32
    return (gx, (du * xh).sum(pixels), du.sum(pixels)), (two * egx, two * egg, two * egb)


def inputs(N, H, W, C, G, dtype, seed, device):
    """x, gamma, beta, gy, with a gy whose level per (sample, group) and whose share of xh are of its own size: both sums
    of a group then weigh as much as the term beside them."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    x = (rand(N, H, W, C) * torch.exp(0.5 * rand(C)) + 0.5 * rand(C)).to(R.DT[dtype])
    gamma, beta = (1 + 0.2 * rand(C).clamp(-2, 2)).to(R.DT[dtype]), (0.3 * rand(C)).to(R.DT[dtype])
    mean, rstd = R.moments(x.double(), G, 1e-5)
    xh = (x.double() - R.per_channel(mean, C)) * R.per_channel(rstd, C)
    sign = torch.where(torch.rand(N, G, generator=g, device=device) < 0.5, -1.0, 1.0).double()
    level, share = (sign * (0.5 + torch.rand(N, G, generator=g, device=device)) for _ in range(2))
    gy = R.per_channel(level, C) + R.per_channel(share, C) * xh + 0.3 * rand(N, H, W, C)
    return x, gamma, beta, (0.05 * gy).to(R.DT[dtype])
