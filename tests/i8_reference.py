"""Plain float64 forms of the 8-bit products and the bounds on a kernel's error.

Codes and sums are exact, so a product's error is that of the scales: the sum's
conversion, top / 127, and two multiplications, 2^-24 each.
"""
import torch

from ffn_reference import ACT_REL, LIPSCHITZ, act, f64, stored

U = 2.0 ** -24


def codes(X):
    """(codes, top / 127) of the rows, exact."""
    x = f64(X)
    top = x.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(127 * x / torch.where(top > 0, top, torch.ones_like(top))), torch.zeros_like(x))
    return q, top[:, 0] / 127


def product(X, Q, scale, bias):
    q, s = codes(X)
    z = (q @ f64(Q).T) * s[:, None] * f64(scale)[None, :]
    e = 5 * U * z.abs() + 2.0 ** -140
    if bias is not None:
        b = f64(bias)
        z = z + b
        e = e + U * (z.abs() + b.abs())
    return z, e


def linear(X, Q, scale, bias, residual, name, dtype):
    z, ez = product(X, Q, scale, bias)
    y = act(name, z)
    ey = LIPSCHITZ * ez + ACT_REL * y.abs()
    if residual is not None:
        r = f64(residual)
        y = y + r
        ey = ey + U * (y.abs() + r.abs())
    return y, stored(y, ey, dtype)


def gated(X, Qg, sg, Qu, su, bg, bu, name, dtype):
    g, eg = product(X, Qg, sg, bg)
    u, eu = product(X, Qu, su, bu)
    a = act(name, g)
    ea = LIPSCHITZ * eg + ACT_REL * a.abs()
    h = a * u
    return h, stored(h, a.abs() * eu + u.abs() * ea + ea * eu + U * h.abs(), dtype)
