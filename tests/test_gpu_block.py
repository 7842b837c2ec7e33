"""The gated feed-forward block: dense passes, compressed form, workspaces and replayed graphs (GPU).

Forward and gradients of the whole block are held to bounds on their Frobenius
norms.  A stored intermediate is off by u of its norm (rounding to the type)
and by what its kernel's bound allows; a product with W carries an error on by
at most ||W||, the spectral norm.  With u the unit roundoff and s = 2^-12 for
every kernel's float32 sums and activations:
    H:  e_H  = (u + s) ||H|| + s ||X|| (||Wg|| max|U| + ||Wu|| max|A|)
    Y:  e_Y  = u ||Y|| + s ||H|| ||Wd|| + e_H ||Wd||
    dH: e_dH = (u + s) ||dY|| ||Wd||
    dG, dU (rounded for the products, from G and U rounded once themselves): with
        p = max|dG/dH| and the like, e_dG = p e_dH + 4 u ||dG|| + u ||dG by G and U||
    dX: u ||dX|| + e_dG ||Wg|| + e_dU ||Wu|| + s (...)
each taken twice over here, so that terms of second order have room.
"""
import sys

import numpy as np
import pytest
import torch

import ffn_reference as ref
from hessian_weighted_vector_amd import block, vq

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
S = 2.0 ** -12


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def make(seed, T, M, N, dtype):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64)

    b = block.GatedBlock(*((s[1] ** -0.5 * normal(*s)).to(dtype).cuda() for s in ((M, N), (M, N), (N, M))))
    return b, normal(T, N).to(dtype).cuda(), normal(T, N).to(dtype).cuda()


def spectral(W):
    return float(torch.linalg.matrix_norm(W, 2))


@pytest.mark.parametrize("size", [(1, 64, 40), (33, 129, 72), (200, 700, 264)])
@pytest.mark.parametrize("dt", DT)
def test_block_forward_backward(size, dt):
    say("block", size, dt)
    dtype = DT[dt]
    u = ref.UNIT[dtype]
    b, X, dY = make(5, *size, dtype)
    Y, kept = b.forward(X, keep=True)
    got = (Y,) + b.backward(dY, kept)
    assert torch.equal(b.forward(X).view(torch.int16), Y.view(torch.int16))

    Xd, Wg, Wu, Wd, D = (ref.f64(t) for t in (X, b.Wg, b.Wu, b.Wd, dY))
    G, U = Xd @ Wg.T, Xd @ Wu.T
    A, A1 = ref.act("silu", G), ref.act_grad("silu", G)
    H = A * U
    dH = D @ Wd
    dG, dU = dH * U * A1, dH * A
    want = (Xd + H @ Wd.T, dG @ Wg + dU @ Wu + D, dG.T @ Xd, dU.T @ Xd, D.T @ H)

    ng, nu, nd = spectral(Wg), spectral(Wu), spectral(Wd)
    nX, nD = float(Xd.norm()), float(D.norm())
    eH = (u + S) * float(H.norm()) + S * nX * (ng * float(U.abs().max()) + nu * float(A.abs().max()))
    edH = (u + S) * nD * nd
    # silu'' is below 0.5: G off by u |G| moves dG by at most 0.5 u |dH U G|
    eG = (float((U * A1).abs().max()) * edH + 4 * u * float(dG.norm()) + 0.5 * u * float((dH * U * G).norm())
          + S * float(dG.norm() + dH.norm()))
    eU = (float(A.abs().max()) * edH + 4 * u * float(dU.norm()) + ref.LIPSCHITZ * u * float((dH * G).norm())
          + S * float(dU.norm() + dH.norm()))
    carried = float(dG.norm()) * ng + float(dU.norm()) * nu
    bound = (eH * nd + S * float(H.norm()) * nd, eG * ng + eU * nu + S * carried + 2 * u * nD, eG * spectral(Xd) + S * float(dG.norm()) * nX,
             eU * spectral(Xd) + S * float(dU.norm()) * nX, eH * spectral(D) + S * float(H.norm()) * nD)
    for name, g, w, e in zip(("Y", "dX", "dWg", "dWu", "dWd"), got, want, bound):
        off = float((ref.f64(g) - w).norm())
        limit = 2 * (e + u * float(w.norm()))
        say("   %s error / bound = %.3g" % (name, off / limit))
        assert off <= limit, name


def test_compressed_block_and_command(capsys):
    """Served from fits of the block's matrices, and the command that runs all of it."""
    say("compressed block")
    b, X, _ = make(6, 64, 256, 128, torch.bfloat16)
    small = b.compress(*b.calibrate(X), d=8, K1=256, iters1=2, K2=64, iters2=2, outlier_frac=0.02)
    What = [m._keep for m in (small.gate, small.up, small.down)]
    assert all(k[0].shape == (256, 8) for k in What)
    Y = small.forward(X[:5])
    by_one = torch.cat([small.forward(X[i:i + 1]) for i in range(5)])
    assert torch.equal(Y.view(torch.int16), by_one.view(torch.int16))
    with pytest.raises(ValueError, match="down"):
        block.CompressedBlock(small.gate, small.up, small.up)
    with pytest.raises(ValueError, match="Wd"):
        block.GatedBlock(b.Wg, b.Wu, b.Wg)
    block.main(["--model", "128", "--hidden", "256", "--tokens", "64", "--steps", "3", "--codebook", "64"])
    lines = capsys.readouterr().out.splitlines()
    errors = [float(s.split()[-1]) for s in lines if s.startswith("step")]
    assert len(errors) == 3 and errors[2] < errors[0]
    assert sum("compressed against dense" in s for s in lines) == 2


CALLS = {
    "linear": lambda X, W, dY, Z, ws: (vq.linear(X, W, ws=ws),),
    "linear_backward": lambda X, W, dY, Z, ws: vq.linear_backward(dY, X, W, Z, "silu", want_db=True, ws=ws),
    "gated": lambda X, W, dY, Z, ws: (vq.gated(X, W, W, ws=ws),),
    "gated_backward": lambda X, W, dY, Z, ws: vq.gated_backward(dY, X, W, W, Z, Z, want_db=True, ws=ws),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("size", [(1, 70, 41), (40, 96, 8200), (300, 264, 520)])
def test_own_workspace(call, size):
    """A workspace of the caller's gives the same bits; one that is too small is refused before any launch."""
    say("workspace", call, size)
    T, M, N = size
    g = torch.Generator().manual_seed(9)
    X, W, dY, Z = ((torch.randn(s, generator=g)).bfloat16().cuda() for s in ((T, N), (M, N), (T, M), (T, M)))
    want = CALLS[call](X, W, dY, Z, None)
    big = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for w, o in zip(want, CALLS[call](X, W, dY, Z, big)):
        assert torch.equal(w.view(torch.int16), o.view(torch.int16))
    if "backward" in call:
        with pytest.raises(vq.VQError, match="workspace"):
            CALLS[call](X, W, dY, Z, big[:256])


def test_graph_replays():
    """One captured pass of the block, replayed on new inputs, gives the eager bits each time."""
    say("graph")
    b, X, dY = make(7, 24, 520, 264, torch.bfloat16)
    small = b.compress(*b.calibrate(X), d=8, K1=256, iters1=1, K2=64, iters2=1, outlier_frac=0.01)

    def whole():
        Y, kept = b.forward(X, keep=True)
        return (Y,) + b.backward(dY, kept) + (small.forward(X[:1]), small.forward(X))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        whole()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = whole()
    g = np.random.default_rng(3)
    for _ in range(4):
        X.copy_(torch.from_numpy(g.standard_normal(tuple(X.shape))))
        dY.copy_(torch.from_numpy(g.standard_normal(tuple(dY.shape))))
        want = whole()
        graph.replay()
        torch.cuda.synchronize()
        for k, (o, w) in enumerate(zip(out, want)):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16)), k


def test_timing_records():
    """Each feed-forward call has one record, keyed by its name and K = 0 whatever the codebooks' sizes."""
    say("timing")
    b, X, dY = make(8, 6, 64, 48, torch.bfloat16)
    small = b.compress(*b.calibrate(X), d=8, K1=16, iters1=1, K2=8, iters2=1)
    other = b.compress(*b.calibrate(X), d=8, K1=32, iters1=1, K2=8, iters2=1)
    vq.timing_enable()
    try:
        _, kept = b.forward(X, keep=True)
        b.backward(dY, kept)
        small.forward(X)
        other.forward(X)
        records = {(name, K): n for name, K, n, *_ in vq.timing_records()}
    finally:
        vq.timing_enable(False)
    assert records == {("gated", 0): 1, ("linear", 0): 1, ("linear_backward", 0): 1, ("gated_backward", 0): 1,
                       ("qgated", 0): 2, ("qlinear", 0): 2}


def test_stream_and_device_handles(monkeypatch):
    """The raw handles are those of torch's public calls, and the calls run as well on the public ones alone."""
    say("handles")
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            assert vq._stream() == s.cuda_stream == vq._public_stream(vq._device())
    assert vq._device() == torch.cuda.current_device()
    b, X, _ = make(9, 3, 40, 24, torch.bfloat16)
    want = b.forward(X)
    monkeypatch.setattr(vq, "_device", torch.cuda.current_device)
    monkeypatch.setattr(vq, "_raw_stream", vq._public_stream)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.forward(X)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
