"""Plain float64 forms of the feed-forward calls and the bounds on a kernel's error.

The bounds follow from the arithmetic that include/vq.h states: products of
16-bit values are exact in float32, a sum of K terms in float32 is off by at
most (K + 32) * 2^-23 of the sum of magnitudes (each addition rounds or
truncates once), an activation formed with the hardware's exponential is off by
2^-16 of its value, and each stored value is rounded once (half a unit in the
last place, u, or half the smallest subnormal).
"""
import math

import torch

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
LIPSCHITZ = 1.2                        # no activation here is steeper
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
ACT_REL = 2.0 ** -16


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64)


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "sigmoid":
        return torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if name == "sigmoid":
        return torch.sigmoid(z) * torch.sigmoid(-z)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)


def sum_error(K):
    return (K + 32) * 2.0 ** -23


def stored(value, error, dtype):
    """Bound on a stored value's error, from the bound on the float32 value's."""
    return error + UNIT[dtype] * (value.abs() + error) + TINY[dtype]


def product(X, W, bias):
    """(X W^T + bias, bound on its float32 error)."""
    z = X @ W.T
    mag = X.abs() @ W.abs().T
    if bias is not None:
        z = z + bias
        mag = mag + bias.abs()
    return z, sum_error(X.shape[1]) * mag


def linear(X, W, bias, residual, name, dtype):
    """[(value, bound)] of Y and Z."""
    X, W, bias, residual = f64(X), f64(W), f64(bias), f64(residual)
    z, ez = product(X, W, bias)
    y = act(name, z)
    ey = LIPSCHITZ * ez + ACT_REL * y.abs()
    if residual is not None:
        y = y + residual
        ey = ey + 2.0 ** -23 * (y.abs() + residual.abs())
    return [(y, stored(y, ey, dtype)), (z, stored(z, ez, dtype))]


def gated(X, Wg, Wu, bg, bu, name, dtype):
    """[(value, bound)] of H, G and U."""
    X = f64(X)
    g, eg = product(X, f64(Wg), f64(bg))
    u, eu = product(X, f64(Wu), f64(bu))
    a = act(name, g)
    ea = LIPSCHITZ * eg + ACT_REL * a.abs()
    h = a * u
    eh = a.abs() * eu + u.abs() * ea + ea * eu + 2.0 ** -23 * h.abs()
    return [(h, stored(h, eh, dtype)), (g, stored(g, eg, dtype)), (u, stored(u, eu, dtype))]


def gradients(dzs, X, Ws, dtype, name):
    """[(value, bound)] of dX, every dW, every db, from [(dz, scale of its terms)]."""
    T = X.shape[0]
    M = dzs[0][0].shape[1]
    ez = [ACT_REL * s for _, s in dzs]                        # float32 error of dz
    er = [stored(d, e, dtype) for (d, _), e in zip(dzs, ez)]  # and after its rounding
    dX = sum(d @ W for (d, _), W in zip(dzs, Ws))
    eX = sum(e @ W.abs() + sum_error(len(Ws) * M) * ((d.abs() + e) @ W.abs()) for (d, _), e, W in zip(dzs, er, Ws))
    out = [(dX, stored(dX, eX, dtype))]
    for (d, _), e in zip(dzs, er):
        v = d.T @ X
        out.append((v, stored(v, e.T @ X.abs() + sum_error(T) * ((d.abs() + e).T @ X.abs()), dtype)))
    for (d, _), e in zip(dzs, ez):
        v = d.sum(0)
        out.append((v, stored(v, e.sum(0) + sum_error(T) * (d.abs() + e).sum(0), dtype)))
    return out


def linear_backward(dY, X, W, Z, name, dtype):
    dY, X, W = f64(dY), f64(X), f64(W)
    if name == "none":
        dz = dY
    else:
        dz = dY * act_grad(name, f64(Z))
    # the derivative's terms are at most about 1.2 in size: their rounding is relative to |dY|
    return gradients([(dz, 2 * dY.abs())], X, [W], dtype, name)


def gated_backward(dH, X, Wg, Wu, G, U, name, dtype):
    dH, X, Wg, Wu, G, U = (f64(t) for t in (dH, X, Wg, Wu, G, U))
    a, da = act(name, G), act_grad(name, G)
    return gradients([(dH * U * da, 2 * (dH * U).abs()), (dH * a, 2 * (dH * a).abs())], X, [Wg, Wu], dtype, name)
