"""Plain fp64 forms of the dense block operators (test support).

Written from the definitions; nothing here is shared with the library.  All
functions take and return float64 tensors (on any device).
"""
import math

import torch

D = torch.float64


def step(dtype) -> float:
    """Half a step of rounding to ``dtype``, relative to the value."""
    return torch.finfo(dtype).eps / 2


def phi(act, g):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "relu":
        return torch.clamp_min(g, 0)
    return 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))


def phi_slope(act, g):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s + g * s * (1 - s)
    if act == "relu":
        return (g > 0).to(D)
    return 0.5 * (1 + torch.erf(g / math.sqrt(2))) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def ffn_forward(act, u, wg, wu, wd):
    g, p = u @ wg.T, u @ wu.T
    a = phi(act, g) * p
    return a @ wd, g, p, a


def ffn_backward(act, u, g, p, dy, wg, wu, wd):
    """du, dWg, dWu, dW2T, and the dg, dp, a they are made of."""
    da = dy @ wd.T
    dg, dp, a = da * p * phi_slope(act, g), da * phi(act, g), phi(act, g) * p
    return dg @ wg + dp @ wu, dg.T @ u, dp.T @ u, a.T @ dy, dg, dp, a


def norm_forward(x, y, *, eps, alpha=1.0, beta=1.0, post_norm=False, w_post=None, w_pre=None, gate=None, per=0):
    """r, u, rstd_post, rstd_pre (None where undefined)."""
    r, kp = alpha * x, None
    if y is not None:
        b = y
        if post_norm:
            kp = 1 / torch.sqrt((y * y).mean(1) + eps)
            b = b * kp[:, None]
            if w_post is not None:
                b = b * w_post
        if gate is not None:
            b = b * gate[torch.arange(len(x), device=x.device) // per]
        r = r + beta * b
    kr = 1 / torch.sqrt((r * r).mean(1) + eps)
    u = r * kr[:, None]
    if w_pre is not None:
        u = u * w_pre
    return r, u, kp, kr


def quantize(x32):
    """Codes and fp32 scales of float32 rows, in float32 as the definition has it."""
    amax = x32.abs().amax(1) if x32.numel() else x32.new_zeros(x32.shape[0])
    scale = amax / torch.full_like(amax, 127)  # by a tensor: torch turns a number into a product with its inverse
    bad = ~torch.isfinite(x32).all(1)
    q = torch.zeros_like(x32)
    use = (scale > 0) & ~bad
    q[use] = torch.round(x32[use] / scale[use][:, None]).clamp(-127, 127)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    return q.to(torch.int8), scale
