"""Plain forms in 64 bits of the linear layer, and the bounds its tests hold it to.

Beside the roundings of operator_refs (half a step of a 16-bit output, 2^-23 of the terms' magnitude for each step of an
fp32 sum) two bounds belong to the activations. Their relative error: exp2 and the reciprocal are off by one step (2^-23)
each, the exponent u by three roundings and two constants, so by less than 3 * 2^-23 * |u|, and a few roundings of 2^-24
stand around them; the normal distribution's polynomial is off by 3.8e-6. The slope's absolute error: p (1 - p), which
multiplies each of those errors, falls faster than the powers of x beside it rise, and their products stay below two, so
ten steps of each bound the whole: 2e-6 for the logistic forms, 4e-6 with the polynomial.
"""
import math

import torch

import operator_refs as ref

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
MOST_SLOPE = 1.13  # of any activation here
SLOPE_ERROR = 4e-6
FLUSHED = 2.0 ** -120  # an exp2 below fp32's normal numbers may give zero: times |x|


def act(name, v):
    """(value, slope, relative error of the fp32 value) in 64 bits."""
    step = 2.0 ** -23
    if name == "none":
        return v, torch.ones_like(v), torch.zeros_like(v)
    if name == "relu":
        return v.clamp(min=0), (v > 0).double(), torch.zeros_like(v)
    if name == "gelu":
        cdf = torch.special.ndtr(v)
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi), 4e-6 + (v * v + 12) * step
    u = v if name == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
    du = 1.0 if name == "silu" else math.sqrt(8 / math.pi) * (1 + 0.134145 * v * v)
    p = torch.sigmoid(u)
    return v * p, p + v * p * (1 - p) * du, (3 * u.abs() + 4) * step


def mats(x, w, layout):
    """x and w [K, C] in 64 bits."""
    return x.double(), (w.double().t() if layout == "nk" else w.double()).contiguous()


def check_forward(y, z, x, w, bias, residual, name, gated, layout):
    xd, wd = mats(x, w, layout)
    K, N = xd.shape[1], y.shape[1]
    want, terms = xd @ wd, xd.abs() @ wd.abs()
    if bias is not None:
        want, terms = want + bias.double(), terms + bias.double().abs()
    if z is not None:
        ref.assert_within(z, want, terms, K + 1, "z")
    off = (K + 1) * 2.0 ** -23 * terms
    value, _, eps = act(name, want[:, :N])
    err = MOST_SLOPE * off[:, :N] + eps * (value.abs() + MOST_SLOPE * off[:, :N]) + FLUSHED * want[:, :N].abs()
    if gated:
        up, up_off = want[:, N:], off[:, N:]
        err = err * (up.abs() + up_off) + value.abs() * up_off + 2.0 ** -24 * (value * up).abs()
        value = value * up
    if residual is not None:
        value = value + residual.double()
        err = err + 2.0 ** -24 * value.abs()
    bound = err + ref.HALF[y.dtype] * (value.abs() + err) + ref.TINY[y.dtype]
    outside(y, value, bound, "y")


def outside(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)  # a NaN is bad too
    if bool(bad.any()):
        at = tuple(int(i) for i in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: {got[at].item()} for "
                             f"{want[at].item()}, bound {bound[at].item():.3g}")


def grad_of_z(dy, z, name, gated):
    """(dz, bound of its error in fp32) in 64 bits; z: the pre-activations the kernel reads."""
    d, N = dy.double(), dy.shape[1]
    if z is None:
        return d, torch.zeros_like(d)
    z = z.double()
    value, slope, eps = act(name, z[:, :N])
    slope_err = (0.0 if name in ("none", "relu") else SLOPE_ERROR) * torch.ones_like(value)
    if not gated:
        return d * slope, d.abs() * (slope_err + 2.0 ** -23 * slope.abs())
    up = z[:, N:]
    dz = torch.cat([d * up * slope, d * value], 1)
    err = torch.cat([(d * up).abs() * (slope_err + 2.0 ** -22 * slope.abs()),
                     d.abs() * (eps * value.abs() + FLUSHED * z[:, :N].abs()) + 2.0 ** -23 * (d * value).abs()], 1)
    return dz, err


def check_backward(dx, dw, db, dy, x, w, z, name, gated, layout):
    xd, wd = mats(x, w, layout)
    dz, err = grad_of_z(dy, z, name, gated)
    C, M = dz.shape[1], dz.shape[0]
    if db is not None:
        e = err.sum(0) + M * 2.0 ** -23 * (dz.abs() + err).sum(0)
        outside(db, dz.sum(0), e + ref.HALF[db.dtype] * (dz.sum(0).abs() + e) + ref.TINY[db.dtype], "db")
    # an operand of the products is rounded to 16 bits; dy itself, where it is dz, is not rounded again
    if z is not None:
        err = err + ref.HALF[x.dtype] * (dz.abs() + err) + ref.TINY[x.dtype]
    far = dz.abs() + err
    for got, want, e, terms, n in (
            (dx, dz @ wd.t(), lambda: err @ wd.abs().t(), lambda: far @ wd.abs().t(), C),
            (dw if layout == "kn" or dw is None else dw.t(), xd.t() @ dz, lambda: xd.abs().t() @ err,
             lambda: xd.abs().t() @ far, M)):
        if got is not None:
            e = e() + n * 2.0 ** -23 * terms()
            outside(got, want, e + ref.HALF[got.dtype] * (want.abs() + e) + ref.TINY[got.dtype], f"gradient {tuple(got.shape)}")
