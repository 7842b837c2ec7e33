"""A gated feed-forward block: trained dense, compressed, then served compressed.

    H = act(X Wg^T) * (X Wu^T),   Y = X + H Wd^T

``GatedBlock`` holds the dense matrices and runs the forward and backward
passes; ``Head`` projects its output onto a vocabulary and holds the loss.
``CompressedBlock`` holds the three as compressed matrices and runs the block for
a few tokens without decoding them to memory; ``Int8Block`` holds them in 8-bit
integers, for prompts.
``python -m hessian_weighted_vector_amd.block`` takes a synthetic block through
all of it: training steps against a teacher's outputs, with --vocab fine-tuning steps
under a head's cross entropy with AdamW, calibration, one fit a matrix, a prompt dense and
in 8 bits and one token at a time compressed, with times and errors.
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

    def to_int8(self):
        """The block in 8-bit integers, a scale a row."""
        return Int8Block(*(vq.Int8Matrix.from_dense(W) for W in (self.Wg, self.Wu, self.Wd)), act=self.act)

    def compress(self, h_in, h_mid, seed=0, int8_prompts=False, **fit):
        """One fit a matrix; `fit` are vq.fit's arguments (d, K1, iters1, ...).

        With int8_prompts the fits' reconstructions are kept in 8 bits beside the compressed
        matrices, and more tokens than the compressed products are for go through them.
        """
        g = np.random.default_rng(seed)
        mats, eight = [], []
        for W, h in ((self.Wg, h_in), (self.Wu, h_in), (self.Wd, h_mid)):
            M, N = W.shape
            n_sub = M * N // fit["d"]
            out = vq.fit(W.float(), h, perm1=g.permutation(n_sub).astype(np.int32),
                         perm2=g.permutation(n_sub).astype(np.int32), **fit)
            mats.append(vq.QMatrix.from_fit(out, M, N, fit["d"]))
            if int8_prompts:
                eight.append(vq.Int8Matrix.from_dense(out["W_hat"]))
        return CompressedBlock(*mats, act=self.act, prompt=Int8Block(*eight, act=self.act) if int8_prompts else None)


class Head:
    """A projection onto a vocabulary, W [V, N], with the mean cross entropy of the learnt tokens."""

    def __init__(self, W):
        self.W = W

    def loss(self, X, labels, ignore_index=-100):
        """(mean loss over the tokens that are not ignored, kept), kept for backward."""
        loss, lse = vq.cross_entropy(X, self.W, labels, ignore_index)
        n = (labels != ignore_index).sum().clamp(min=1)
        return loss.sum() / n, (X, labels, lse, n, ignore_index)

    def backward(self, kept, scale=1.0):
        """(dX, dW) of scale times the mean loss; fp16 callers take a scale that keeps the gradients in range."""
        X, labels, lse, n, ignore_index = kept
        dloss = torch.full((X.shape[0],), float(scale), dtype=torch.float32, device=X.device) / n
        return vq.cross_entropy_backward(dloss, X, self.W, labels, lse, ignore_index)


class Int8Block:
    """The block from 8-bit matrices, for any number of bfloat16 or float16 tokens."""

    def __init__(self, gate, up, down, act="silu"):
        if (up.M, up.N) != (gate.M, gate.N) or (down.M, down.N) != (gate.N, gate.M):
            raise ValueError("gate and up must be [M x N] and down [N x M]")
        if gate._struct.ldq != up._struct.ldq:                # the pair's rows are read together
            gate, up = gate.compact(), up.compact()
        self.gate, self.up, self.down, self.act = gate, up, down, act

    def forward(self, X):
        return vq.linear_i8(self.down, vq.gated_i8(self.gate, self.up, X, act=self.act), residual=X)


class CompressedBlock:
    """The block from its compressed matrices, for a few tokens of any of the types.

    Every 32 tokens read the matrices anew: a prompt is faster through GatedBlock, or through
    `prompt`, an Int8Block that takes calls of more than 32 bfloat16 or float16 tokens.
    """

    FEW = 32

    def __init__(self, gate, up, down, act="silu", prompt=None):
        if (up.M, up.N) != (gate.M, gate.N) or (down.M, down.N) != (gate.N, gate.M):
            raise ValueError("gate and up must be [M x N] and down [N x M]")
        self.gate, self.up, self.down, self.act, self.prompt = gate, up, down, act, prompt

    def forward(self, X):
        if self.prompt is not None and X.shape[0] > self.FEW and X.dtype != torch.float32:
            return self.prompt.forward(X)
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


def fine_tune(block, master, X, want, a, g):
    """Steps of block and head under the cross entropy of the word that a teacher's head likes best.

    The first quarter of the tokens is a prompt that is not learnt.  `master` holds the float32
    matrices; block's are their copies, and AdamW writes both.
    """
    N = X.shape[1]
    teacher = torch.randn((a.vocab, N), generator=g, dtype=torch.float32, device="cuda") * N ** -0.5
    labels = (want.float() @ teacher.T).argmax(1)
    labels[:X.shape[0] // 4] = -100
    master["head"] = 0.5 * teacher
    head = Head(master["head"].bfloat16())
    params = [block.Wg, block.Wu, block.Wd, head.W]
    opt = vq.AdamW(params, masters=[master[k] for k in ("Wg", "Wu", "Wd", "head")], lr=a.tune_lr, state_bits=a.state_bits)
    for step in range(a.tune):
        Y, kept = block.forward(X, keep=True)
        loss, at = head.loss(Y, labels)
        dY, dW = head.backward(at)
        _, *grads = block.backward(dY, kept)
        opt.step(grads + [dW])
        print("fine-tuning step %d  loss %.5f" % (step, float(loss)), flush=True)


def main(argv=None):
    p = argparse.ArgumentParser(prog="python -m hessian_weighted_vector_amd.block",
                                description="Train, compress and serve a synthetic gated feed-forward block.")
    p.add_argument("--model", type=int, default=2048, help="columns of the block's input")
    p.add_argument("--hidden", type=int, default=8192, help="rows of gate and up")
    p.add_argument("--tokens", type=int, default=2048, help="tokens of a training batch and of the prompt")
    p.add_argument("--steps", type=int, default=5, help="training steps")
    p.add_argument("--lr", type=float, default=0.1, help="step on the squared error's mean over the tokens")
    p.add_argument("--vocab", type=int, default=0, help="words of a head; above 0, block and head are fine-tuned under its cross entropy")
    p.add_argument("--tune", type=int, default=3, help="fine-tuning steps of block and head")
    p.add_argument("--tune-lr", type=float, default=1e-4, help="learning rate of AdamW in them")
    p.add_argument("--state-bits", type=int, default=8, choices=(8, 32), help="of AdamW's moments")
    p.add_argument("--codebook", type=int, default=4096, help="first-stage centroids")
    a = p.parse_args(argv)
    if not torch.cuda.is_available():
        raise SystemExit("a GPU is needed")

    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(scale, *shape):
        return scale * torch.randn(shape, generator=g, dtype=torch.float32, device="cuda")

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

    if a.vocab:
        fine_tune(block, master, X, want, a, g)

    h_in, h_mid = block.calibrate(X)
    small = block.compress(h_in, h_mid, int8_prompts=True, d=8, K1=a.codebook, iters1=4, K2=256, iters2=3, outlier_frac=0.01)
    prompt = block.forward(X)
    for t in (1, 8):
        Yd, Yq = prompt[:t].float(), small.forward(X[:t]).float()
        rel = float((Yq - Yd).norm() / (Yd - X[:t].float()).norm())
        print("%d token(s): compressed against dense, relative to the block's output %.3f; %.1f us compressed, %.1f us dense"
              % (t, rel, _time(lambda: small.forward(X[:t])), _time(lambda: block.forward(X[:t]))), flush=True)
    print("prompt of %d tokens: %.1f us" % (T, _time(lambda: block.forward(X))))
    eight = block.to_int8()
    rel = float((eight.forward(X).float() - prompt.float()).norm() / (prompt.float() - X.float()).norm())
    print("the same in 8 bits: relative to the block's output %.4f; %.1f us" % (rel, _time(lambda: eight.forward(X))))


if __name__ == "__main__":
    main()
