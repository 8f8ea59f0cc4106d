"""phi and phi' of the gated block element by element, against fp64.

One-hot weights make every product one exact term: g and p of a token are the
two elements of its u, y is a = phi(g) p, and du holds dg and dp.  g runs over
every 16-bit value up to 12 in size.

Tolerance: one rounding to the type (h relative, or half its smallest step),
and R = 2^-16 for the fp32 evaluation.  The largest part of R is the exponent
of e^(-g^2/2): two roundings, 2^-24 each, of an argument up to 72, 8.6e-6; the
tail's formula is within 1e-6, and the hardware's exponential, reciprocal and
about ten operations are within 2^-22 each: 1.2e-5 < 2^-16 = 1.5e-5.  SiLU's
exponent is at most 12.  phi' is a sum of two terms of opposite sign; its error
is relative to their sizes.  Exponentials below 2^-126 are flushed.
"""
import math

import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb

pytestmark = pytest.mark.gpu

D = torch.float64
R = 2.0 ** -16


def _values(dtype, most=12.0):
    """Every value of the type up to `most` in size, both signs."""
    top = int(torch.tensor(most, dtype=dtype).view(torch.int16))
    bits = torch.arange(top + 1, dtype=torch.int32).to(torch.int16)
    v = bits.view(dtype)
    return torch.cat([v, -v]).cuda()


def _tail(g):
    """P(N < g) with full relative accuracy."""
    return torch.special.erfc(-g / math.sqrt(2)) / 2


def _phi(act, g):
    return g * _tail(g) if act == "gelu" else ref.phi(act, g)


def _slope_terms(act, g):
    """The two terms of phi'."""
    if act == "gelu":
        return _tail(g), g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s, g * s / (1 + torch.exp(g))
    return (g > 0).to(D), torch.zeros_like(g)


def _layer(dtype, act):
    wg, wu, wd = (torch.zeros(8, 8, dtype=dtype, device="cuda") for _ in range(3))
    wg[0, 0] = wu[0, 1] = wd[0, 0] = 1
    return pb.GatedFfnLayer(wg, wu, wd, act=act)


def _within(got, want, size, dtype, flushed):
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2  # half a subnormal step
    tol = ref.step(dtype) * want.abs() + R * size + tiny + flushed
    off = (got.to(D) - want).abs()
    at = int((off - tol).argmax())
    assert torch.all(off <= tol), (at, float(got[at]), float(want[at]), float(tol[at]))


@pytest.mark.parametrize("tokens", [100, 0], ids=["few", "all"])
@pytest.mark.parametrize("up", [1.0, 4096.0])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_activation_and_its_slope(cuda_device, dtype, act, up, tokens):
    g = _values(dtype)
    if tokens:  # the kernel of few tokens, on values from -4 to -8, where GELU's tail is smallest against 1
        g = g[(g <= -4) & (g >= -8)]
        g = g[torch.linspace(0, len(g) - 1, tokens, device="cuda").long()]
    T = len(g)
    layer = _layer(dtype, act)
    ws = pb.make_gated_ffn_workspace(layer, T, True)
    u = torch.zeros(T, 8, dtype=dtype, device="cuda")
    u[:, 0], u[:, 1] = g, up
    y, gate, upo = torch.empty_like(u), torch.empty_like(u), torch.empty_like(u)
    pb.pi_gated_ffn_forward(layer, u, y, ws, gate=gate, up=upo)
    G = g.to(D)
    assert torch.equal(gate[:, 0], g) and torch.all(upo[:, 0] == up)
    want = _phi(act, G) * up
    flushed = G.abs() * up * 2.0 ** -125
    _within(y[:, 0], want, want.abs(), dtype, flushed)
    dy = torch.zeros_like(u)
    dy[:, 0] = 1
    du = torch.empty_like(u)
    pb.pi_gated_ffn_backward(layer, u, gate, upo, dy, ws, du)
    assert pb.pi_get_device_status(ws) == 0
    c, k = _slope_terms(act, G)
    _within(du[:, 0], (c + k) * up, (c.abs() + k.abs()) * up, dtype, flushed + up * 2.0 ** -125)
    _within(du[:, 1], want / up, want.abs() / up, dtype, flushed + 2.0 ** -125)


@pytest.mark.parametrize("tokens", [3, 300])
@pytest.mark.parametrize("act,at", [("relu", -1.0), ("relu", 0.0), ("silu", -1.28125), ("gelu", -0.75)])
def test_large_gradients_times_a_small_slope(cuda_device, act, at, tokens):
    """dg = da p phi'(g) where da p lies past fp32's largest value and phi' is zero or small: dg is finite."""
    dtype, big = torch.bfloat16, 2.0 ** 66
    layer = _layer(dtype, act)
    ws = pb.make_gated_ffn_workspace(layer, tokens, True)
    u, gate, upo, dy = (torch.zeros(tokens, 8, dtype=dtype, device="cuda") for _ in range(4))
    gate[:, 0], upo[:, 0], dy[:, 0] = at, big, big
    du = torch.empty_like(u)
    pb.pi_gated_ffn_backward(layer, u, gate, upo, dy, ws, du)
    c, k = _slope_terms(act, gate[:, 0].to(D))
    want = (c + k) * big * big
    assert want.abs().max() < 1e38
    tol = ref.step(dtype) * want.abs() + R * (c.abs() + k.abs()) * big * big
    assert torch.all((du[:, 0].to(D) - want).abs() <= tol)
