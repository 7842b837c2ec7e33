"""The block with a head, its loss and the optimizer's step together, and its 8-bit prompts (GPU)."""
import pytest
import torch

import ffn_reference as ref
import loss_reference
from hessian_weighted_vector_amd import block, vq

pytestmark = pytest.mark.gpu


def make(seed, T, M, N, V, dtype):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64)

    b = block.GatedBlock(*((s[1] ** -0.5 * normal(*s)).to(dtype).cuda() for s in ((M, N), (M, N), (N, M))))
    h = block.Head((2 * N ** -0.5 * normal(V, N)).to(dtype).cuda())
    labels = torch.randint(0, V, (T,), generator=g)
    labels[:T // 4] = -100
    return b, h, normal(T, N).to(dtype).cuda(), labels.cuda()


def mean_loss(X, Wg, Wu, Wd, W, labels):
    """The whole chain in float64."""
    G, U = X @ Wg.T, X @ Wu.T
    Y = X + (ref.act("silu", G) * U) @ Wd.T
    z = Y @ W.T
    on = labels != -100
    per = torch.logsumexp(z, 1) - z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    return per[on].sum() / on.sum()


@pytest.mark.parametrize("dtype,scale", [(torch.bfloat16, 1.0), (torch.float16, 1024.0)])
@pytest.mark.parametrize("size", [(8, 64, 40, 50), (70, 129, 72, 333), (300, 700, 264, 1000)])
def test_gradients_of_the_whole_chain(size, dtype, scale):
    """Block, head and loss against float64's automatic gradients.

    Every stored intermediate is rounded to u of itself (H, Y, dz, dY, dH, dG, dU, the gradients: eight), each
    carried on by products whose sums average independent roundings; in the 2-norm each
    gradient is held to sixteen of them.
    """
    b, h, X, labels = make(1, *size, dtype)
    Y, kept = b.forward(X, keep=True)
    loss, at = h.loss(Y, labels)
    dY, dW = h.backward(at, scale)
    got = b.backward(dY, kept) + (dW,)
    leaves = [ref.f64(t).requires_grad_() for t in (X, b.Wg, b.Wu, b.Wd, h.W)]
    want = mean_loss(*leaves, labels.cpu())
    want.backward()
    u = ref.UNIT[dtype]
    want = float(want.detach())
    assert abs(float(loss) - want) <= 16 * u * abs(want)
    for name, g, leaf in zip(("dX", "dWg", "dWu", "dWd", "dW"), got, leaves):
        off = float((ref.f64(g) / scale - leaf.grad).norm() / leaf.grad.norm())
        assert off <= 16 * u, (name, off)


def test_head_without_learnt_tokens():
    b, h, X, labels = make(2, 40, 64, 40, 50, torch.bfloat16)
    labels.fill_(-100)
    loss, at = h.loss(X, labels)
    dX, dW = h.backward(at)
    assert float(loss) == 0.0 and not bool(dX.any()) and not bool(dW.any())


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_training_step(bits):
    """A whole training step in one graph: forward, loss, gradients, AdamW; replays equal eager steps bit for bit."""
    def program():
        b, h, X, labels = make(3, 200, 264, 136, 500, torch.bfloat16)
        params = [b.Wg, b.Wu, b.Wd, h.W]
        opt = vq.AdamW(params, masters=[p.float() for p in params], lr=1e-3, state_bits=bits, capturable=True)

        def step():
            Y, kept = b.forward(X, keep=True)
            loss, lse = vq.cross_entropy(Y, h.W, labels)
            dY, dW = vq.cross_entropy_backward(dloss, Y, h.W, labels, lse)
            opt.step(list(b.backward(dY, kept)[1:]) + [dW])
            return loss

        dloss = torch.full((200,), 1 / 150, device="cuda")
        return step, opt, X, labels

    eager, opt, X, labels = program()
    replayed, opt2, X2, labels2 = program()
    eager()
    replayed()                                               # the tables of both are made before the capture
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        out = replayed()
    g = torch.Generator().manual_seed(4)
    for k in range(4):
        x = torch.randn(X.shape, generator=g)
        lab = torch.randint(0, 500, labels.shape, generator=g)
        lab[:50 * (k % 3)] = -100
        for t, l in ((X, labels), (X2, labels2)):
            t.copy_(x)
            l.copy_(lab)
        loss = eager()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, out)
        for p, q in zip(opt.masters + opt.params, opt2.masters + opt2.params):
            assert torch.equal(p, q)
    assert int(opt.steps) == int(opt2.steps) == 5


@pytest.mark.parametrize("T", [1, 20, 33, 200])
def test_int8_block(T):
    """The block in 8 bits: its products' bounds on the codes it holds, one product after the other."""
    import i8_reference as i8
    b, _, X, _ = make(5, T, 200, 136, 8, torch.bfloat16)
    e = b.to_int8()
    H = vq.gated_i8(e.gate, e.up, X)
    value, bound = i8.gated(X, e.gate.q, e.gate.scale, e.up.q, e.up.scale, None, None, "silu", torch.bfloat16)
    assert bool(((ref.f64(H) - value).abs() <= bound).all())
    value, bound = i8.linear(H, e.down.q, e.down.scale, None, X, "none", torch.bfloat16)
    assert bool(((ref.f64(e.forward(X)) - value).abs() <= bound).all())
    # a code is off by half a step of its row's largest, 1 / 254 of it, and the scale by 2^-24 of itself, which is
    # at most 2^-24 of the largest: together 1 / 254 (1 + 254 2^-24) < 1 / 254 (1 + 2^-16)
    for W, q in ((b.Wg, e.gate), (b.Wu, e.up), (b.Wd, e.down)):
        back = q.q.double() * q.scale.double()[:, None]
        worst = float(((back - W.double()).abs() / W.double().abs().amax(1, keepdim=True)).max())
        assert worst <= (1 + 2.0 ** -16) / 254


def test_compressed_block_with_int8_prompts():
    b, _, X, _ = make(6, 100, 256, 128, 8, torch.bfloat16)
    fit = dict(d=8, K1=64, iters1=1, K2=16, iters2=1, outlier_frac=0.01)
    h_in, h_mid = b.calibrate(X)
    plain, small = b.compress(h_in, h_mid, **fit), b.compress(h_in, h_mid, int8_prompts=True, **fit)
    assert plain.prompt is None
    assert torch.equal(small.forward(X[:32]), plain.forward(X[:32]))
    assert torch.equal(small.forward(X), small.prompt.forward(X))
    assert torch.equal(small.forward(X.float()), plain.forward(X.float()))     # float32 tokens stay with the compressed form
    with pytest.raises(ValueError, match="down"):
        block.Int8Block(small.prompt.gate, small.prompt.up, small.prompt.up)


def test_command(capsys):
    for extra, steps in (([], 0), (["--vocab", "300", "--tune", "2", "--state-bits", "32"], 2), (["--vocab", "500"], 3)):
        block.main(["--model", "128", "--hidden", "256", "--tokens", "64", "--steps", "1", "--codebook", "64"] + extra)
        lines = capsys.readouterr().out.splitlines()
        tuned = [float(s.split()[-1]) for s in lines if s.startswith("fine-tuning step")]
        assert len(tuned) == steps and all(x == x for x in tuned)
        assert sum("in 8 bits" in s for s in lines) == 1


def test_timing_records():
    b, h, X, labels = make(7, 50, 64, 48, 30, torch.bfloat16)
    e = b.to_int8()
    opt = vq.AdamW([h.W])
    vq.timing_enable()
    try:
        loss, at = h.loss(X, labels)
        opt.step([h.backward(at)[1]])
        e.forward(X)
        vq.quantize_rows(X)
        records = {(name, K): n for name, K, n, *_ in vq.timing_records()}
    finally:
        vq.timing_enable(False)
    assert records == {("cross_entropy", 0): 1, ("cross_entropy_backward", 0): 1, ("adamw", 0): 1, ("gated_i8", 0): 1,
                       ("linear_i8", 0): 1, ("quantize_rows", 0): 1}
