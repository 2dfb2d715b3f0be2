"""Plain 64-bit forms of the operators around a block's layers (RMS norm,
8-bit 1x1 product, clipping), and how far the kernels may be from them.

Operands are taken as stored and widened exactly. Everything is counted in
units u = 2^-24 of the values or of the sums of the terms' sizes:
  r           a sum of squares (positive terms) behind at most ROW additions, so
              ROW u of itself; the root halves that; eps' addition, the
              multiplication by 1 / C, 1 / C and the root itself are one each
  y           two products more
  gx          t, its sum with h (SUM additions at most), c1 (3 products), then
              4 operations
  ggamma      one product and r's per term, CHAIN additions
  product     a block's 128 products of e4m3 are added by four instructions of
              33 terms; each term may be cut off at 2^-23 of the largest, 2 u
              of the sum of sizes, so 264 u; then a product of scales and an
              addition per block, and the bias
"""
import torch

import train_bounds as TB
import train_ref as R

U = R.EPS32
ROW, SUM, CHAIN = 128, 128, 256


def slack_rstd(r):
    return (ROW / 2 + 6) * U * r


def rms_fwd(x, residual, gamma, eps, dtype):
    """h as stored, r and y in 64 bits; x, residual, gamma as stored."""
    h = x if residual is None else (x.float() + residual.float()).to(R.DT[dtype])
    hd = h.double()
    r = 1 / torch.sqrt(hd.square().mean(-1) + eps)
    y = hd * r[:, None]
    return h, r, y if gamma is None else y * gamma.double()


def slack_y(y):
    return (ROW / 2 + 9) * U * y.abs()


def rms_bwd(h, gy, gamma, rstd, gres):
    """gx and ggamma in 64 bits from operands as stored, and the slack of each."""
    h, gy, r = h.double(), gy.double(), rstd.double()[:, None]
    t = gy if gamma is None else gy * gamma.double()
    xh, C = h * r, h.shape[-1]
    c1 = (t * xh).sum(-1, keepdim=True) / C
    gx = r * (t - xh * c1)
    size = (t * xh).abs().sum(-1, keepdim=True) / C
    slack = U * r * (4 * t.abs() + xh.abs() * (6 * c1.abs() + (SUM + 4) * size)) + 2 * U * gx.abs()
    if gres is not None:
        gx = gx + gres.double()
        slack = slack + U * gx.abs()
    return gx, (gy * xh).sum(0), slack, (CHAIN + 3) * U * (gy * xh).abs().sum(0)


def encode_weights(w):
    """Codes [cout, cin rounded up to 128] and scales, bit for bit."""
    o, k = w.shape
    no, nk = -(-o // 128), -(-k // 128)
    wb = torch.nn.functional.pad(w.float(), (0, nk * 128 - k, 0, no * 128 - o)).reshape(no, 128, nk, 128)
    amax = wb.abs().amax((1, 3), keepdim=True)
    scale = amax * torch.tensor(1.0 / 448.0, dtype=torch.float32, device=w.device)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale == 0, torch.zeros_like(scale), torch.ones_like(scale) / scale)
    codes = (wb * inv).to(torch.float8_e4m3fn).reshape(no * 128, nk * 128)[:o].contiguous()
    return codes, scale.reshape(no, nk).contiguous()


def weight_values(codes, scales, cin):
    s = scales.double().repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)
    return (codes.double() * s)[:, :cin]


def product(codes, scales, wcodes, wscales, bias, act):
    """y in 64 bits of the codes as given, and its slack."""
    cin = codes.shape[-1]
    x = codes.double() * scales.double().repeat_interleave(128, -1)[:, :cin]
    w = weight_values(wcodes, wscales, cin)
    u = x @ w.t()
    du = (264 + 2 * scales.shape[-1]) * (x.abs() @ w.abs().t())
    if bias is not None:
        u = u + bias.double()
        du = du + u.abs()
    dy, _ = TB.act_errors(u, du, act)
    return TB.act(u, act), 2 * U * dy


def clip(grads, most):
    n = torch.sqrt(sum((g.double().square().sum() for g in grads), torch.zeros((), dtype=torch.float64, device="cuda")))
    k = torch.clamp(most / (n + 1e-6), max=1.0)
    return n, [g.double() * k for g in grads]


def slack_norm(n):
    """Chains of at most 256 positive terms in 32 bits, their sums in 64, and the rounding of n."""
    return (256 / 2 + 2) * U * n
