"""Plain 64-bit forms of the channels-last training operators (torch, any
device), and the tolerances that their tests use.

Every reference takes the operands as stored (rounded to the tensor's type)
and widens them exactly. Tolerances are derived from the kernels' arithmetic:
fp32 sums whose error is at most (terms in a chain) * 2^-24 * (sum of the
terms' sizes), and one rounding to the storage type, 2^-24, 2^-11 or 2^-8 of
the value (half a unit in the last place; fp16 also half its smallest step).
"""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
STEP = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
EPS32 = 2.0 ** -24
CHAIN = 256  # longest chain of additions behind one output at the tests' sizes


def within(got, ref, slack, dtype, what=""):
    """|got - ref| <= one rounding of ref + slack (fp32 arithmetic), elementwise."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - ref).abs() - (ROUND[dtype] * ref.abs() + STEP[dtype] + slack)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3g} over the tolerance"


# ---- 8-bit checkpoints: the definition, in the fp32 operations it names -----

CODE_MAX = {"i8": 127.0, "e4m3": 448.0}


def encode(x, kind, block):
    """(codes, scales) of x [..., C], bit for bit."""
    C = x.shape[-1]
    nb = -(-C // block)
    xb = torch.nn.functional.pad(x.float(), (0, nb * block - C)).reshape(*x.shape[:-1], nb, block)
    amax = xb.abs().amax(-1, keepdim=True)
    scale = amax * torch.tensor(1.0 / CODE_MAX[kind], dtype=torch.float32, device=x.device)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale == 0, torch.zeros_like(scale), torch.ones_like(scale) / scale)
    v = xb * inv
    if kind == "i8":
        codes = torch.nan_to_num(v.round(), nan=0.0).to(torch.int8)
    else:
        codes = v.to(torch.float8_e4m3fn)
    return codes.reshape(*x.shape[:-1], nb * block)[..., :C].contiguous(), scale.squeeze(-1)


def decode(codes, scales, block):
    """The values in 64 bits (each is one fp32 product)."""
    s = scales.repeat_interleave(block, -1)[..., :codes.shape[-1]]
    return (codes.float() * s).double()


# ---- group norm ------------------------------------------------------------


def act(u, name):
    if name == "relu":
        return torch.clamp(u, min=0)
    if name == "relu6":
        return torch.clamp(u, 0, 6)
    if name == "silu":
        return u * torch.sigmoid(u)
    if name == "gelu":
        return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    return u


def act_slope(u, name):
    if name == "relu":
        return (u > 0).double()
    if name == "relu6":
        return ((u > 0) & (u < 6)).double()
    if name == "silu":
        q = torch.sigmoid(u)
        return q * (1 + u * (1 - q))
    if name == "gelu":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (u + 0.044715 * u ** 3))
        return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * k * (1 + 3 * 0.044715 * u * u)
    return torch.ones_like(u)


def moments(x, G, eps):
    """mean, rstd [N, G] of x [N, H, W, C] in 64 bits."""
    N, C = x.shape[0], x.shape[-1]
    v = x.reshape(N, -1, G, C // G)
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return mean, 1 / torch.sqrt(var + eps)


def per_channel(v, C):
    """[N, G] -> [N, 1, 1, C]"""
    return v.repeat_interleave(C // v.shape[1], 1)[:, None, None, :]


def norm_fwd(x, gamma, beta, G, eps, name):
    mean, rstd = moments(x, G, eps)
    C = x.shape[-1]
    u = (x - per_channel(mean, C)) * per_channel(rstd, C) * gamma + beta
    return act(u, name), mean, rstd


def norm_bwd(x, gy, gamma, beta, mean, rstd, name):
    """gx, ggamma, gbeta, and the sizes their tolerances go by."""
    N, H, W, C = x.shape
    G = mean.shape[1]
    mu, rs = per_channel(mean, C), per_channel(rstd, C)
    xh = (x - mu) * rs
    du = gy * act_slope(xh * gamma + beta, name)
    dv = du * gamma
    m = H * W * (C // G)
    group = lambda v: v.reshape(N, H * W, G, C // G).sum((1, 3))  # noqa: E731
    s1, s2 = per_channel(group(dv) / m, C), per_channel(group(dv * xh) / m, C)
    gx = rs * (dv - s1 - xh * s2)
    t1, t2 = per_channel(group(dv.abs()) / m, C), per_channel(group((dv * xh).abs()) / m, C)
    size = rs * (dv.abs() + gy.abs() * gamma.abs() + CHAIN * (t1 + xh.abs() * t2))
    return gx, (du * xh).sum((0, 1, 2)), du.sum((0, 1, 2)), size, (gy * xh).abs().sum((0, 1, 2)), gy.abs().sum((0, 1, 2))


# ---- depthwise backward ----------------------------------------------------


def conv_bwd(x, gy, w, d):
    """gx, gw, gb of y = dwconv(x, w) + b, channels-last, from the definition; w [C*m, kh, kw]; d a binding.Desc.
    Then the sums of the terms' sizes behind gx and gw."""
    N, H, W, C = x.shape
    m, kh, kw = d.multiplier, d.kh, d.kw
    Ho, Wo = gy.shape[1:3]
    Hp = max(H + 2 * d.pad_h, (Ho - 1) * d.stride_h + (kh - 1) * d.dil_h + 1)
    Wp = max(W + 2 * d.pad_w, (Wo - 1) * d.stride_w + (kw - 1) * d.dil_w + 1)
    xp = x.new_zeros(N, Hp, Wp, C)
    xp[:, d.pad_h:d.pad_h + H, d.pad_w:d.pad_w + W] = x
    gxp, gxa = torch.zeros_like(xp), torch.zeros_like(xp)
    gw, gwa = torch.zeros_like(w), torch.zeros_like(w)
    for a in range(kh):
        for b in range(kw):
            r = slice(a * d.dil_h, a * d.dil_h + (Ho - 1) * d.stride_h + 1, d.stride_h)
            q = slice(b * d.dil_w, b * d.dil_w + (Wo - 1) * d.stride_w + 1, d.stride_w)
            xs = xp[:, r, q].repeat_interleave(m, -1)
            gw[:, a, b] = (gy * xs).sum((0, 1, 2))
            gwa[:, a, b] = (gy * xs).abs().sum((0, 1, 2))
            t = gy * w[:, a, b]
            gxp[:, r, q] += t.reshape(N, Ho, Wo, C, m).sum(-1)
            gxa[:, r, q] += t.abs().reshape(N, Ho, Wo, C, m).sum(-1)
    cut = (slice(None), slice(d.pad_h, d.pad_h + H), slice(d.pad_w, d.pad_w + W))
    return gxp[cut], gw, gy.sum((0, 1, 2)), gxa[cut], gwa, gy.abs().sum((0, 1, 2))
