"""Plain float64 forms of the cross entropy calls and the bounds on a kernel's error.

From the arithmetic that include/vq.h states: logits are float32 sums of exact
products (see ffn_reference.sum_error); the logarithm of a sum of exponentials moves by
at most the largest error of a logit, and by the relative errors of the
exponentials and of the sum; exp(x) formed as 2^(x log2 e) is off by three roundings of
x, relative to its value, and 2^-22 for the hardware's power; dz is rounded to the
tensors' type before it is multiplied, in fp16 times 2^13 over the largest |dloss|.
"""
import torch

from ffn_reference import TINY, UNIT, f64, stored, sum_error

U = 2.0 ** -24


def logits(X, W):
    """(z, bound on its float32 error)."""
    X, W = f64(X), f64(W)
    return X @ W.T, sum_error(X.shape[1]) * (X.abs() @ W.abs().T)


def forward(X, W, labels, ignore):
    """[(loss, bound), (lse, bound)]; labels inside the vocabulary or ignored."""
    z, ez = logits(X, W)
    labels = labels.cpu()
    V = z.shape[1]
    on = labels != ignore
    at = torch.where(on, labels, torch.zeros_like(labels))
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    below = z.amax(1, keepdim=True) - z
    # each term: its exponential; the sum: 34 terms in a lane and its exchanges, then joins of parts of 64 words or more,
    # each with two exponentials of the parts' distances (together no more than the range) and three roundings
    joins = V / 64 / 64 + 8
    rel = (p * (3 * U * below + 2.0 ** -22)).sum(1) + 40 * U + joins * (2 * 2.0 ** -22 + 3 * U)
    rel = rel + (p * 6 * U * below).sum(1)
    e = ez.amax(1) + rel + 4 * U * (lse.abs() + 1)
    loss = lse - z.gather(1, at[:, None])[:, 0]
    el = e + ez.gather(1, at[:, None])[:, 0] + U * loss.abs()
    zero = torch.zeros_like(loss)
    tiny = torch.full_like(loss, 2.0 ** -140)
    return [(torch.where(on, loss, zero), torch.where(on, el, tiny)), (torch.where(on, lse, zero), torch.where(on, e, tiny))]


def backward(dloss, X, W, labels, lse, ignore):
    """[(dX, bound), (dW, bound)] for the float32 lse given."""
    dtype = X.dtype
    z, ez = logits(X, W)
    X, W, g, lse, labels = f64(X), f64(W), f64(dloss), f64(lse), labels.cpu()
    on = labels != ignore
    rows = on.nonzero()[:, 0]
    X0 = X
    z, ez, X, g, lse, labels = z[rows], ez[rows], X[rows], g[rows], lse[rows], labels[rows]
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(p)
    hot[torch.arange(len(rows)), labels] = 1
    dz = (p - hot) * g[:, None]
    # a probability's relative error: the logit's, its distance's and product's roundings, the power's
    rel = torch.expm1(ez + 3 * U * (z - lse[:, None]).abs() + 2.0 ** -22)
    rel = torch.where(p > 0, p * rel, torch.zeros_like(p))   # below float64's range nothing is left to be off
    # dloss is divided by its largest and dz multiplied by the quotient; the results are multiplied back
    e = g.abs()[:, None] * (rel + U * hot) + 5 * U * dz.abs()
    top = float(g.abs().max()) if len(rows) else 0.0
    tiny = TINY[dtype]
    if dtype == torch.float16 and top > 0:
        tiny = tiny * top * 2.0 ** -12                        # the largest |dloss| becomes 2^13
    e = e + UNIT[dtype] * (dz.abs() + e) + tiny
    V, T = dz.shape[1], len(rows)
    dX, eX = torch.zeros_like(X0), torch.zeros_like(X0)
    dX[rows] = dz @ W
    eX[rows] = e @ W.abs() + sum_error(V) * ((dz.abs() + e) @ W.abs())
    dW = dz.T @ X
    eW = e.T @ X.abs() + sum_error(T) * ((dz.abs() + e).T @ X.abs())
    return [(dX, stored(dX, eX, dtype)), (dW, stored(dW, eW, dtype))]
