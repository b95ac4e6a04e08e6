"""Plain 64-bit forms of the residual epilogue and of its gradient, in torch
(any device), straight from their definitions, with the errors that the
library's FP32 arithmetic may have."""
import math

import torch

ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU, ACT_SWIGLU = 0, 1, 2, 3, 8
HALF_BF16, SUM = 2.0 ** -8, 2.0 ** -23
TINY = 2.0 ** -126


def act(z, a):
    s = torch.special.expit
    if a == ACT_RELU:
        return z.clamp(min=0)
    if a == ACT_GELU:
        return z * s(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if a == ACT_SILU:
        return z * s(z)
    if a == ACT_SWIGLU:
        return z[:, 0::2] * s(z[:, 0::2]) * z[:, 1::2]
    return z


def epilogue(z, dz, a, residual=None):
    """(D, its tolerance, z's tolerance) for a product plus bias z that is off
    by dz in FP32.

    No activation has a slope above 1.13; the logistic form is off by a few
    units of FP32's last place and by its argument's rounding (at most 64
    units where the result is not yet zero); the residual's sum is one more
    rounding, and then there is one to BF16."""
    d = act(z, a)
    if a == ACT_SWIGLU:
        g, u = z[:, 0::2], z[:, 1::2]
        slip = 1.13 * dz[:, 0::2] * u.abs() + (g * torch.special.expit(g)).abs() * dz[:, 1::2] + dz[:, 0::2] * dz[:, 1::2]
    else:
        slip = 1.13 * dz
    if a not in (ACT_NONE, ACT_RELU):
        slip = slip + 64 * SUM * d.abs()
    if residual is not None:
        d = d + residual.double()
        slip = slip + SUM * (d.abs() + slip)
    return d, (d.abs() + slip) * HALF_BF16 + slip + TINY, (z.abs() + dz) * HALF_BF16 + dz + TINY


def slope(z, a):
    s = torch.special.expit
    if a == ACT_RELU:
        return (z > 0).double()
    if a == ACT_GELU:
        r = 2 * math.sqrt(2 / math.pi)
        u = r * (z + 0.044715 * z ** 3)
        return s(u) + z * s(u) * s(-u) * r * (1 + 0.134145 * z ** 2)
    if a == ACT_SILU:
        return s(z) + z * s(z) * s(-z)
    return torch.ones_like(z)


def gradient(dD, z, a):
    """(dz, its tolerance before the rounding to BF16, dbias, its tolerance).

    A slope is a sum of two terms of at most 1.13 and |z s t u'| (below 1.2),
    each off by its logistic values (a few units) and by their arguments'
    roundings: e^u off by |u| half units where s t is not yet zero, |u| below
    90 and |u| s(u) s(-u) below 0.3: 8 units of 2.4 in all.  dz: one product
    more (SwiGLU two, and g s(g) off by 64 units of itself).

    The logistic values s and 1 - s are FP32 numbers, and one below the normal
    range (an argument below -87.3) may be flushed to zero: s is then off by up
    to 2^-126, so z s by |z| 2^-126, and dz by |d| times the sum of both (SwiGLU:
    times |u|, and g s(g) by |g| 2^-126)."""
    d = dD.double()
    if a == ACT_SWIGLU:
        z = z.double()
        g, u = z[:, 0::2], z[:, 1::2]
        dz, slip = torch.empty_like(z), torch.empty_like(z)
        dz[:, 0::2], dz[:, 1::2] = d * u * slope(g, ACT_SILU), d * g * torch.special.expit(g)
        slip[:, 0::2] = (d * u).abs() * (20 * SUM + (1 + g.abs()) * TINY)
        slip[:, 1::2] = dz[:, 1::2].abs() * 66 * SUM + (d * g).abs() * TINY
    elif a == ACT_NONE:
        dz, slip = d, torch.zeros_like(d)
    else:
        dz = d * slope(z.double(), a)
        slip = d.abs() * ((1 if a == ACT_RELU else 20) * SUM + (1 + z.double().abs()) * TINY)
    slip = slip + TINY
    # an FP32 sum of M terms, in any order
    return dz, slip, dz.sum(0), slip.sum(0) + dz.shape[0] * SUM * dz.abs().sum(0)
