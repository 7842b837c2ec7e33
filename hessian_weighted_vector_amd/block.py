"""A gated feed-forward block: trained dense, compressed, then served compressed.

    H = act(X Wg^T) * (X Wu^T),   Y = X + H Wd^T

``GatedBlock`` holds the dense matrices and runs the forward and backward
passes; ``CompressedBlock`` holds the three as compressed matrices and runs the
block for a few tokens without decoding them to memory.
``python -m hessian_weighted_vector_amd.block`` takes a synthetic block through
all of it: training steps, calibration, one fit a matrix, prefill dense and one
token at a time compressed, with times and errors.
"""
import argparse

import numpy as np
import torch

from . import vq


class GatedBlock:
    """Dense weights, bfloat16 or float16: Wg and Wu [M, N], Wd [N, M]."""

    def __init__(self, Wg, Wu, Wd, act="silu"):
        if Wu.shape != Wg.shape or tuple(Wd.shape) != (Wg.shape[1], Wg.shape[0]):
            raise ValueError("Wg and Wu must be [M, N] and Wd [N, M]")
        self.Wg, self.Wu, self.Wd, self.act = Wg, Wu, Wd, act

    def forward(self, X, keep=False):
        """Y, or with keep (Y, kept), which backward takes."""
        r = vq.gated(X, self.Wg, self.Wu, act=self.act, want_pre=keep)
        H = r[0] if keep else r
        Y = vq.linear(H, self.Wd, residual=X)
        return (Y, (X, r)) if keep else Y

    def backward(self, dY, kept):
        """(dX, dWg, dWu, dWd).

        dX is rounded to the type twice, as the block's two terms (the gated product's gradient
        and the residual's, dY) are two tensors of it.
        """
        X, (H, G, U) = kept
        dH, dWd, _ = vq.linear_backward(dY, H, self.Wd)
        dX, dWg, dWu, _, _ = vq.gated_backward(dH, X, self.Wg, self.Wu, G, U, act=self.act)
        return dX.add_(dY), dWg, dWu, dWd

    def calibrate(self, X):
        """The Hessian diagonals of the block's inputs and of H: mean squares by column (float32)."""
        H = vq.gated(X, self.Wg, self.Wu, act=self.act)
        return X.float().square().mean(0), H.float().square().mean(0)

    def compress(self, h_in, h_mid, seed=0, **fit):
        """One fit a matrix; `fit` are vq.fit's arguments (d, K1, iters1, ...)."""
        g = np.random.default_rng(seed)
        mats = []
        for W, h in ((self.Wg, h_in), (self.Wu, h_in), (self.Wd, h_mid)):
            M, N = W.shape
            n_sub = M * N // fit["d"]
            out = vq.fit(W.float(), h, perm1=g.permutation(n_sub).astype(np.int32),
                         perm2=g.permutation(n_sub).astype(np.int32), **fit)
            mats.append(vq.QMatrix.from_fit(out, M, N, fit["d"]))
        return CompressedBlock(*mats, act=self.act)


class CompressedBlock:
    """The block from its compressed matrices, for a few tokens of any of the types.

    Every 32 tokens read the matrices anew: a prompt is faster through GatedBlock.
    """

    def __init__(self, gate, up, down, act="silu"):
        if (up.M, up.N) != (gate.M, gate.N) or (down.M, down.N) != (gate.N, gate.M):
            raise ValueError("gate and up must be [M x N] and down [N x M]")
        self.gate, self.up, self.down, self.act = gate, up, down, act

    def forward(self, X):
        return vq.qlinear(self.down, vq.qgated(self.gate, self.up, X, act=self.act), residual=X)


def _time(f, n=20):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n * 1e3


def main(argv=None):
    p = argparse.ArgumentParser(prog="python -m hessian_weighted_vector_amd.block",
                                description="Train, compress and serve a synthetic gated feed-forward block.")
    p.add_argument("--model", type=int, default=2048, help="columns of the block's input")
    p.add_argument("--hidden", type=int, default=8192, help="rows of gate and up")
    p.add_argument("--tokens", type=int, default=2048, help="tokens of a training batch and of the prompt")
    p.add_argument("--steps", type=int, default=5, help="training steps")
    p.add_argument("--lr", type=float, default=0.1, help="step on the squared error's mean over the tokens")
    p.add_argument("--codebook", type=int, default=4096, help="first-stage centroids")
    a = p.parse_args(argv)
    if not torch.cuda.is_available():
        raise SystemExit("a GPU is needed")

    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(scale, *shape):
        return scale * torch.randn(shape, generator=g, device="cuda")

    N, M, T = a.model, a.hidden, a.tokens
    names = ("Wg", "Wu", "Wd")
    teacher = GatedBlock(*(normal(s[1] ** -0.5, *s).bfloat16() for s in ((M, N), (M, N), (N, M))))
    # the student starts off the teacher; float32 masters, bfloat16 copies for the kernels
    master = {k: getattr(teacher, k).float() + normal(0.3 * getattr(teacher, k).shape[1] ** -0.5, *getattr(teacher, k).shape)
              for k in names}
    block = GatedBlock(*(master[k].bfloat16() for k in names))
    X = normal(1.0, T, N).bfloat16()
    want = teacher.forward(X)
    for step in range(a.steps):
        Y, kept = block.forward(X, keep=True)
        diff = Y.float() - want.float()
        _, *grads = block.backward(diff.bfloat16(), kept)
        print("step %d  mean square error %.5f" % (step, float(diff.square().mean())), flush=True)
        for k, d in zip(names, grads):
            master[k].add_(d.float(), alpha=-a.lr / T)
            getattr(block, k).copy_(master[k])

    h_in, h_mid = block.calibrate(X)
    small = block.compress(h_in, h_mid, d=8, K1=a.codebook, iters1=4, K2=256, iters2=3, outlier_frac=0.01)
    prompt = block.forward(X)
    for t in (1, 8):
        Yd, Yq = prompt[:t].float(), small.forward(X[:t]).float()
        rel = float((Yq - Yd).norm() / (Yd - X[:t].float()).norm())
        print("%d token(s): compressed against dense, relative to the block's output %.3f; %.1f us compressed, %.1f us dense"
              % (t, rel, _time(lambda: small.forward(X[:t])), _time(lambda: block.forward(X[:t]))), flush=True)
    print("prompt of %d tokens: %.1f us" % (T, _time(lambda: block.forward(X))))


if __name__ == "__main__":
    main()
