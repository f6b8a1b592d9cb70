"""The feed-forward operators in 8 bits from their formulas, in 64 bits, and what their codes
and sums may be off by."""
import math

import torch

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10),
       "e5m2": (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}
BF = torch.bfloat16
HALF = {torch.float32: 2.0 ** -24, BF: 2.0 ** -8}      # half a step, relative


def values(codes, scales):
    """What codes and 1x128 scales stand for, in 64 bits."""
    return (codes.double().view(*scales.shape, 128) * scales.double()[..., None]).view(codes.shape)


def weight_values(codes, scales):
    """The same for 128x128 scales."""
    return codes.double() * scales.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


def quantise(x, fmt="e4m3"):
    """Codes and 1x128 scales of x, as the package's quantisation makes them."""
    dtype, most, _, _ = FP8[fmt]
    b = x.float().reshape(*x.shape[:-1], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax == 0, 1.0, amax / most)
    return (b / s).clamp(-most, most).to(dtype).reshape(x.shape), s[..., 0].contiguous()


def quantise_weight(w, fmt="e4m3"):
    dtype, most, _, _ = FP8[fmt]
    *lead, n, k = w.shape
    b = w.float().reshape(*lead, n // 128, 128, k // 128, 128)
    s = b.abs().amax((-3, -1), keepdim=True) / most
    s = torch.where(s == 0, 1.0, s)
    return (b / s).clamp(-most, most).to(dtype).reshape(w.shape), s[..., 0, :, 0].contiguous()


def check_codes(codes, scales, v, err, fmt, what=""):
    """codes and scales against the values v (64 bits) that the kernel may have been err (of v's
    shape, or a number) off before it quantised them: a scale is amax / FMAX of values that are
    at most that far off (and rounded once), a code stands for the nearest value: off by half
    a step of the code's binade, or of the smallest binade."""
    dtype, most, half, least = FP8[fmt]
    assert codes.dtype is dtype and scales.dtype is torch.float32
    err = torch.as_tensor(err, device=v.device, dtype=torch.float64).expand(v.shape)
    blocks = (*v.shape[:-1], v.shape[-1] // 128, 128)
    amax, e = v.abs().view(blocks).amax(-1), err.reshape(blocks).amax(-1)
    s = scales.double()
    zero = amax == 0
    off = (s * most - amax).abs() - (e + amax * 2.0 ** -22)
    bad = (off > 0) & ~(zero & (s == 1))
    assert not bad.any(), f"{what}: scales {int(bad.sum())} off, worst {float(off.max()):.3g}"
    got = values(codes, scales)
    s = s.repeat_interleave(128, -1)
    binade = torch.exp2(torch.floor(torch.log2(((v.abs() + err) / s * (1 + 2.0 ** -20)).clamp_min(1e-300))))
    off = (got - v).abs() - (s * (half * binade).clamp_min(least) * (1 + 2.0 ** -20) + err)
    assert off.max() <= 0, f"{what}: codes off by {float(off.max()):.3g} at {int(off.argmax())}"


def check_codes_sharp(codes, scales, v, rel, fmt, what=""):
    """Codes of values v that the kernel has to a relative error of rel: the code of v over
    the kernel's own scale, or the next one where the quotient is that near a border."""
    dtype, most, _, _ = FP8[fmt]
    q = v / scales.double().repeat_interleave(128, -1)
    lo = (q * (1 - rel)).clamp(-most, most).float().to(dtype).float()
    hi = (q * (1 + rel)).clamp(-most, most).float().to(dtype).float()
    got = codes.float()
    bad = (got != lo) & (got != hi)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes of {bad.numel()} differ"


# ------------------------------------------------------------------------------- norm
def norm(x, w=None, r=None, eps=1e-6):
    """h (in x's type), rstd and y, in 64 bits from there."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    v = h.double()
    rstd = (v.square().mean(1) + eps).rsqrt()
    y = v * rstd[:, None]
    return h, rstd, y if w is None else y * w.double()


def norm_backward(dy, h, rstd, w=None, dh=None):
    """grad_x, grad_weight, and the sums of magnitudes that their errors go by."""
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    g = dy if w is None else dy * w.double()
    K = h.shape[1]
    dx = r * (g - h * (r * r * (g * h).sum(1, keepdim=True) / K))
    mag = r * (g.abs() + h.abs() * (r * r * (g * h).abs().sum(1, keepdim=True) / K))
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, (dy * h * r).sum(0), mag, (dy * h * r).abs().sum(0)


# ------------------------------------------------------------------------------ gated
def sigmoid_of(g, act):
    """sigmoid(z(g)) and dz/dg."""
    if act == "silu":
        return torch.sigmoid(g), torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return torch.sigmoid(c * (g + 0.044715 * g ** 3)), c * (1 + 3 * 0.044715 * g ** 2)


def gated(g, u, act):
    return g * sigmoid_of(g, act)[0] * u


def gated_backward(dh, g, u, act):
    s, dz = sigmoid_of(g, act)
    return torch.cat([dh * u * (s + g * s * (1 - s) * dz), dh * g * s], -1)


def written(idx, groups):
    """Rows that the contiguous calls write."""
    n = idx.numel()
    lead = idx[torch.arange(n, device=idx.device) // 128 * 128]
    return (idx >= 0) & (idx < groups) & (idx == lead)
