"""Plain 64-bit definitions of the BF16 products, the dense layer and the
combine's gradient, with the error bounds that the tests hold the kernels to.
Nothing here uses the package.

Bounds, with u = 2^-24 (half an ulp of fp32):
  * A sum of n exact products in fp32 in any order, each step rounded or
    truncated, is off by at most gamma(n) S, S the sum of the magnitudes.
  * Rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24.
  * exp and the fast quotient are each good to 2 ulp (4 u), so that s = 1 / (1 +
    exp(-g)) is good to 10 u of itself and 1 - s to 11 u absolutely.  Below
    2^-126 fp32 has no normal s: the quotient by a divisor of 2^126 and more is
    0, off by less than 2^-126 (TINY allows that twice, for the quotient's own
    limit and for a product that rounds below it), which what s is multiplied
    by carries into the result: |u| (1 + |g|) |dh|, or |g| |dh|.
  * The normal distribution function is good to 10 u of itself (a polynomial of
    6e-9, ten steps of it, an exponential and a quotient of 4 u each),
    exp(-v^2 / 2) to (v^2 / 2 + 4) u * 2 of itself.
"""
import math

import torch

from moe_reference import U, gamma

TINY = 2.0 ** -125
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def product(a, w):
    """a [m, k], w [n, k]: (a w^T, bound of the fp32 sum's error)."""
    a, w = a.double(), w.double()
    return a @ w.T, gamma(w.shape[1]) * (a.abs() @ w.abs().T)


def sigmoid(v):
    return torch.special.expit(v)


def silu_back(v):
    s = sigmoid(v)
    return s * (1 + v * (1 - s))


def cdf(v):
    """Normal distribution function, without the cancellation of 1 + erf far below zero."""
    return 0.5 * torch.special.erfc(-v * math.sqrt(0.5))


def phi(v):
    return torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)


def activation(v, dv, act):
    """(act(v), bound of its error) for fp32 values v that are off by dv.  |act'| <= 1.2."""
    if act == "none":
        return v, dv
    if act == "relu":
        return v.clamp_min(0), dv
    out = v * sigmoid(v) if act == "silu" else v * cdf(v)
    return out, 1.2 * dv + 16 * U * out.abs() + TINY * (1 + v.abs())


def gated(y, dy):
    """SwiGLU of [m, 2n] (gate, up): |silu'| <= 1.1, the two factors' errors together."""
    (g, u), (dg, du) = y.chunk(2, 1), dy.chunk(2, 1)
    s = g * sigmoid(g)
    return s * u, 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * U * (s * u).abs() + TINY * (1 + g.abs() * (u.abs() + du))


def activation_back(z, dy, act):
    """(dz, bound of its fp32 error) for exact z and dy."""
    if act == "none":
        return dy, torch.zeros_like(dy)
    if act == "relu":
        return torch.where(z > 0, dy, torch.zeros_like(dy)), torch.zeros_like(dy)
    if act == "silu":
        return dy * silu_back(z), dy.abs() * (24 * U * sigmoid(z) + TINY) * (1 + z.abs()) + TINY
    d = cdf(z) + z * phi(z)
    off = 12 * U * cdf(z) + z.abs() * phi(z) * (z * z + 16) * U
    return dy * d, dy.abs() * (off + 4 * U * d.abs() + TINY * (1 + z.abs())) + TINY


def gated_back(z, dh, ddh):
    """(dz [m, 2n], bound) of SwiGLU for dh off by ddh and exact z."""
    g, u = z.chunk(2, 1)
    s = sigmoid(g)
    dg, du = dh * u * silu_back(g), dh * g * s
    off = (24 * U * s + TINY) * (1 + g.abs())
    eg = ddh * (u * silu_back(g)).abs() + (dh.abs() + ddh) * u.abs() * off + TINY
    eu = ddh * (g * s).abs() + (dh.abs() + ddh) * g.abs() * (s * 24 * U + TINY) + TINY
    return torch.cat([dg, du], 1), torch.cat([eg, eu], 1)


def linear(x, w, bias=None, act="none", residual=None):
    """(out, bound, z, bound) before the last rounding."""
    y, dy = product(x, w)
    if bias is not None:
        y = y + bias.double()
        dy = dy + U * (y.abs() + dy)
    out, d = gated(y, dy) if act == "swiglu" else activation(y, dy, act)
    if residual is not None:
        out = out + residual.double()
        d = d + U * (out.abs() + d)
    return out, d, y, dy


def close(got, want, off):
    """Whether `got` is `want`, off by `off` before its rounding to got's type."""
    h = HALF[got.dtype]
    return ((got.double() - want).abs() <= h * (want.abs() + off) + off).all()


def combine_back(dout, y, w, dst):
    """(dy by pair [T, k, H], dw [T, k], bound of dw)."""
    at = dst.long().clamp_min(0)
    d, v = dout.double()[:, None, :], y.double()[at]
    live = (dst >= 0).double()
    dw = (d * v).sum(2) * live
    return w.double()[..., None] * d, dw, gamma(dout.shape[1]) * (d * v).abs().sum(2) * live
