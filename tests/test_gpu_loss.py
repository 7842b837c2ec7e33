"""Cross entropy over a vocabulary and its gradient against float64, every value within a derived bound."""
import pytest
import torch

import loss_reference as ref
from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu

IGN = -100
HALF = [torch.bfloat16, torch.float16]


def inputs(T, V, N, dtype, seed, masked=0.3, ldx=0, ldw=0, offset=0, scale=2.0):
    """Tokens whose label's logit is raised, rows ldx and ldw longer than N, offset elements into their buffers."""
    g = torch.Generator().manual_seed(seed)

    def view(x, more):
        rows, cols = x.shape
        buf = torch.full((rows * (cols + more) + offset + 8,), 3.0, dtype=dtype, device="cuda")
        v = buf[offset:offset + rows * (cols + more)].view(rows, cols + more)[:, :cols]
        v.copy_(x)
        return v

    W = torch.randn((V, N), generator=g) * scale / N ** 0.5
    labels = torch.randint(0, V, (T,), generator=g)
    X = torch.randn((T, N), generator=g) + 3 * torch.rand((T, 1), generator=g) * W[labels]
    off = torch.rand(T, generator=g) < masked
    labels = torch.where(off, torch.full_like(labels, IGN), labels).cuda()
    return view(X, ldx), view(W, ldw), labels, torch.randn(T, generator=g).cuda()


def within(got, want, what):
    value, bound = want
    got = ref.f64(got)
    assert got.shape == value.shape
    bad = ~((got - value).abs() <= bound)
    assert not bool(bad.any()), "%s: %d of %d, first %s: %r against %r, bound %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(value[bad][0]), float(bound[bad][0]))


def check(X, W, labels, dloss):
    loss, lse = vq.cross_entropy(X, W, labels, ignore_index=IGN)
    want = ref.forward(X, W, labels, IGN)
    within(loss, want[0], "loss")
    within(lse, want[1], "lse")
    dX, dW = vq.cross_entropy_backward(dloss, X, W, labels, lse, ignore_index=IGN)
    want = ref.backward(dloss, X, W, labels, lse, IGN)
    within(dX, want[0], "dX")
    within(dW, want[1], "dW")
    return loss, lse, dX, dW


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,V,N", [
    (1, 1, 1), (1, 2, 8), (1, 1000, 64), (2, 63, 15), (3, 64, 136), (15, 65, 32), (16, 257, 513), (17, 255, 7), (31, 4001, 100),
    (32, 256, 256), (33, 256, 64), (33, 1, 3), (64, 129, 1), (100, 1000, 129), (128, 128, 128), (257, 513, 72), (300, 5003, 40),
    (511, 300, 321), (200, 1088, 2994), (126, 500, 5001), (700, 257, 1500), (1, 100, 5000),
    (5, 333, 4097), (8, 40, 4100), (16, 500, 2049), (30, 700, 1030), (7, 33000, 520),
    (25, 9001, 131), (32, 33001, 72), (18, 100, 64)])
def test_sizes(T, V, N, dtype):
    check(*inputs(T, V, N, dtype, T * 1000 + V))


@pytest.mark.parametrize("T,V,N,dtype", [
    (40, 40000, 1040, torch.bfloat16), (128, 33000, 2056, torch.float16), (70, 17000, 3000, torch.bfloat16),
    (16, 40000, 2600, torch.float16), (9, 45000, 4096, torch.bfloat16), (20, 40001, 2601, torch.bfloat16)])
def test_few_tokens_of_large_vocabularies(T, V, N, dtype):
    """Where a round of workgroups reads the whole vocabulary, and where few tokens go through tiles."""
    X, W, labels, dloss = inputs(T, V, N, dtype, V + T)
    first = check(X, W, labels, dloss)
    again = (*vq.cross_entropy(X, W, labels, ignore_index=IGN),)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("ldx,ldw,offset", [(0, 1, 0), (1, 0, 0), (3, 5, 1), (8, 8, 8), (16, 0, 3)])
@pytest.mark.parametrize("T", [5, 20, 70])
def test_strides_and_alignment(T, ldx, ldw, offset):
    check(*inputs(T, 333, 96, torch.bfloat16, 5, ldx=ldx, ldw=ldw, offset=offset))


@pytest.mark.parametrize("T", [4, 90, 600])
@pytest.mark.parametrize("masked", [0.0, 0.97, 1.1])
def test_masks(T, masked):
    """No token ignored, nearly all, and all: zeros then, dW among them."""
    X, W, labels, dloss = inputs(T, 700, 64, torch.float16, 11, masked=masked)
    loss, lse, dX, dW = check(X, W, labels, dloss)
    off = labels == IGN
    assert not bool(loss[off].any()) and not bool(lse[off].any()) and not bool(dX[off].any())
    if masked > 1:
        assert not bool(dW.any())


@pytest.mark.parametrize("T", [8, 200])
def test_ignored_rows_may_hold_anything(T):
    """NaN and infinities in X, dloss and lse of ignored tokens reach nothing."""
    X, W, labels, dloss = inputs(T, 500, 72, torch.bfloat16, 12, masked=0.5)
    loss, lse, dX, dW = check(X, W, labels, dloss)
    off = (labels == IGN).nonzero()[:, 0]
    X2, dl2, ls2 = X.clone(), dloss.clone(), lse.clone()
    X2[off[::2]], X2[off[1::2]] = float("nan"), float("inf")
    dl2[off] = float("nan")
    ls2[off] = float("-inf")
    a, b = vq.cross_entropy(X2, W, labels, ignore_index=IGN)
    c, d = vq.cross_entropy_backward(dl2, X2, W, labels, ls2, ignore_index=IGN)
    for x, y in ((loss, a), (lse, b), (dX, c), (dW, d)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T", [8, 200])
def test_non_finite_values_stay_in_their_rows(T):
    X, W, labels, dloss = inputs(T, 500, 72, torch.bfloat16, 13, masked=0.0)
    loss, lse, dX, _ = check(X, W, labels, dloss)
    X[3, 5] = float("nan")
    X[6, 0] = float("inf")
    a, b = vq.cross_entropy(X, W, labels, ignore_index=IGN)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[3] = bad[6] = True
    assert bool(torch.isnan(a[bad]).all()) and torch.equal(a[~bad], loss[~bad]) and torch.equal(b[~bad], lse[~bad])
    c, d = vq.cross_entropy_backward(dloss, X, W, labels, b, ignore_index=IGN)
    assert torch.equal(c[~bad], dX[~bad]) and not bool(torch.isfinite(c[3]).any())
    assert not bool(torch.isfinite(d).all())


@pytest.mark.parametrize("T", [6, 80])
def test_labels_outside_the_vocabulary(T):
    """NaN for the token, nothing read out of range, the others unchanged."""
    X, W, labels, dloss = inputs(T, 130, 64, torch.bfloat16, 14, masked=0.0)
    loss, lse, dX, _ = check(X, W, labels, dloss)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    for t, l in ((0, 130), (2, -1), (3, 1 << 40), (5, -(1 << 62))):
        labels[t] = l
        bad[t] = True
    a, b = vq.cross_entropy(X, W, labels, ignore_index=IGN)
    assert bool(torch.isnan(a[bad]).all()) and torch.equal(a[~bad], loss[~bad]) and torch.equal(b, lse)
    c, d = vq.cross_entropy_backward(dloss, X, W, labels, lse, ignore_index=IGN)
    assert bool(torch.isnan(c[bad]).all()) and torch.equal(c[~bad], dX[~bad]) and bool(torch.isnan(d).all())
    # the same number as ignore_index is simply ignored
    a, _ = vq.cross_entropy(X, W, labels, ignore_index=130)
    assert float(a[0]) == 0.0


def test_extreme_logits():
    """Logits far apart: a certain token (loss 0), a hopeless one, and float32's largest spread."""
    for T in (4, 40):
        X = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
        W = torch.zeros((300, 8), dtype=torch.bfloat16, device="cuda")
        X[:, 0] = 1.0
        W[7, 0] = 200.0
        W[8, 0] = -3e38
        labels = torch.full((T,), 7, device="cuda")
        labels[1], labels[2] = 8, 9
        dloss = torch.ones(T, device="cuda")
        loss, lse, dX, dW = check(X, W, labels, dloss)
        assert float(loss[0]) == 0.0 and float(loss[2]) == 200.0 and float(loss[1]) > 2.9e38
        assert torch.equal(lse, torch.full_like(lse, 200.0))


def test_all_logits_minus_infinity():
    X = torch.full((40, 8), float("inf"), dtype=torch.bfloat16, device="cuda")
    W = torch.full((70, 8), -1.0, dtype=torch.bfloat16, device="cuda")
    for T in (3, 40):
        loss, lse = vq.cross_entropy(X[:T], W, torch.zeros(T, dtype=torch.int64, device="cuda"))
        assert bool((lse == float("-inf")).all()) and bool(torch.isnan(loss).all())


def test_fp16_small_weights_of_the_loss():
    """dloss of 1e-6, and of very different tokens: the power of two keeps dz's precision."""
    X, W, labels, dloss = inputs(120, 3000, 64, torch.float16, 15)
    W.mul_(0.05)
    dloss.fill_(2.0 ** -3)
    dloss[1::2] *= 2.0 ** -9
    check(X, W, labels, dloss)
    check(X, W, labels, torch.zeros_like(dloss))


def test_wanted_outputs_and_empty_batches():
    X, W, labels, dloss = inputs(50, 200, 64, torch.bfloat16, 16)
    loss, lse, dX, dW = check(X, W, labels, dloss)
    a, none = vq.cross_entropy_backward(dloss, X, W, labels, lse, want_dw=False)
    assert none is None and torch.equal(a, dX)
    none, b = vq.cross_entropy_backward(dloss, X, W, labels, lse, want_dx=False)
    assert none is None and torch.equal(b, dW)
    a, b = vq.cross_entropy(X[:0], W, labels[:0])
    assert a.shape == b.shape == (0,)
    dX, dW = vq.cross_entropy_backward(dloss[:0], X[:0], W, labels[:0], b)
    assert dX.shape == (0, 64) and dW.shape == (200, 64) and not bool(dW.any())


def test_against_differences():
    """The gradient against differences of the kernel's own loss, along random directions."""
    X, W, labels, _ = inputs(40, 150, 24, torch.float16, 17, scale=1.0)
    n = int((labels != IGN).sum())
    dloss = torch.full((40,), 1.0 / n, device="cuda")
    loss, lse = vq.cross_entropy(X, W, labels)
    dX, dW = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    g = torch.Generator().manual_seed(1)
    for t, grad in ((X, dX), (W, dW)):
        # steps of an exact power of two that the values' type holds; the difference's own error: third
        # derivatives (h^2), the losses' float32 roundings (2^-20 / h)
        d = torch.sign(torch.randn(t.shape, generator=g)).cuda()
        h = 2.0 ** -7
        keep = t.clone()
        t.copy_((keep.float() + h * d).half())
        up, dup = vq.cross_entropy(X, W, labels)[0].double().sum() / n, t.double()
        t.copy_((keep.float() - h * d).half())
        down, ddown = vq.cross_entropy(X, W, labels)[0].double().sum() / n, t.double()
        t.copy_(keep)
        want = float((grad.double() * (dup - ddown)).sum())   # along the difference as it was stored
        size = float((grad.double().abs() * (dup - ddown).abs()).sum())
        assert abs(float(up - down) - want) <= 0.02 * size + 2.0 ** -18


def exact_on_gpu(X, W, labels, dloss, lse):
    """dX and dW in float64 on the GPU, for sizes past the CPU's."""
    x, w = X.double(), W.double()
    p = torch.exp(x @ w.T - lse.double()[:, None])
    on = labels != IGN
    p[on.nonzero()[:, 0], labels[on]] -= 1
    p *= (dloss.double() * on)[:, None]
    return p @ w, p.T @ x


@pytest.mark.parametrize("dtype,V,ldw", [(torch.bfloat16, 50000, 0), (torch.float16, 40001, 1)])
def test_pieces_of_the_vocabulary(dtype, V, ldw):
    """Several pieces, the last a ragged one: rows of dW at their places, dX summed over all, 256 x 256 tiles."""
    T, N = 4100, 64
    X, W, labels, dloss = inputs(T, V, N, dtype, 18, masked=0.2, ldw=ldw)
    assert vq.load().vq_cross_entropy_backward_workspace_bytes(T, V, N, 0, N + ldw, 1, 1) < T * V * 2
    loss, lse = vq.cross_entropy(X, W, labels)
    z = X.double() @ W.double().T
    on = labels != IGN
    want = torch.logsumexp(z, 1)
    # a logit's bound, and of the sum of exponentials 64 roundings of 2^-22
    tol = ref.sum_error(N) * float((X.double().abs() @ W.double().abs().T).max()) + 64 * 2.0 ** -22
    assert float(((lse.double() - want).abs() * on).max()) <= tol
    picked = z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    assert float(((loss.double() - (want - picked)).abs() * on).max()) <= 2 * tol
    del z
    dX, dW = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    wx, ww = exact_on_gpu(X, W, labels, dloss, lse)
    # two independent roundings of relative size UNIT (dz, the result): twice that in the 2-norm
    for got, ref64 in ((dX, wx), (dW, ww)):
        assert float((got.double() - ref64).norm() / ref64.norm()) <= 2 * ref.UNIT[dtype]
    # every row by itself: none is missing, doubled or misplaced
    for got, ref64 in ((dX[on], wx[on]), (dW, ww)):
        rel = (got.double() - ref64).norm(dim=1) / ref64.norm(dim=1).clamp(min=1e-9)
        assert float(rel.max()) <= 0.05


def test_pieces_of_copied_rows_with_split_sums():
    """Few tokens over a vocabulary whose rows are copied in two pieces, N over several workgroups."""
    T, V, N = 40, 17513, 4570
    X, W, labels, _ = inputs(T, V, N, torch.bfloat16, 24, masked=0.2)
    labels[:4] = torch.tensor([0, V - 1, 8959, 8960], device="cuda")     # first, last, and where the pieces meet
    loss, lse = vq.cross_entropy(X, W, labels)
    z = X.double() @ W.double().T
    on = labels != IGN
    want = torch.logsumexp(z, 1)
    tol = ref.sum_error(N) * float((X.double().abs() @ W.double().abs().T).max()) + 64 * 2.0 ** -22
    picked = z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    assert float(((lse.double() - want).abs() * on).max()) <= tol
    assert float(((loss.double() - (want - picked)).abs() * on).max()) <= 2 * tol


def test_same_bits_every_time_and_on_another_stream():
    X, W, labels, dloss = inputs(700, 3000, 128, torch.bfloat16, 19)
    first = check(X, W, labels, dloss)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        loss, lse = vq.cross_entropy(X, W, labels)
        dX, dW = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    st.synchronize()
    for a, b in zip(first, (loss, lse, dX, dW)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [9, 150])
def test_captured_graphs(T):
    """Two graphs that share a workspace, replayed in turn on new data with eager calls between."""
    X, W, labels, dloss = inputs(T, 900, 64, torch.bfloat16, 20)
    lib = vq.load()
    n = max(lib.vq_cross_entropy_workspace_bytes(T, 900, 64, 0, 64),
            lib.vq_cross_entropy_backward_workspace_bytes(T, 900, 64, 0, 64, 1, 1))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    f, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(f, stream=st):
        loss, lse = vq.cross_entropy(X, W, labels, ws=ws)
    with torch.cuda.graph(b, stream=st):
        dX, dW = vq.cross_entropy_backward(dloss, X, W, labels, lse, ws=ws)
    for k in range(4):
        X2, _, labels2, dloss2 = inputs(T, 900, 64, torch.bfloat16, 30 + k, masked=0.2 * k)
        X.copy_(X2)
        labels.copy_(labels2)
        dloss.copy_(dloss2)
        f.replay()
        b.replay()
        torch.cuda.synchronize()
        want = check(X, W, labels, dloss)
        for got, w in zip((loss, lse, dX, dW), want):
            assert torch.equal(got, w)


def test_python_refusals():
    X, W, labels, dloss = inputs(10, 20, 16, torch.bfloat16, 21)
    with pytest.raises(TypeError, match="labels"):
        vq.cross_entropy(X, W, labels.int())
    with pytest.raises(ValueError, match="labels"):
        vq.cross_entropy(X, W, labels[:9])
    with pytest.raises(TypeError, match="W must"):
        vq.cross_entropy(X, W.half(), labels)
    with pytest.raises(ValueError, match="contiguous rows"):
        vq.cross_entropy(X.t().contiguous().t(), W, labels)
    with pytest.raises(ValueError, match="lse"):
        vq.cross_entropy_backward(dloss, X, W, labels, dloss[:3])
    with pytest.raises(vq.VQError, match="workspace"):
        vq.cross_entropy(X, W, labels, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_value_check(monkeypatch):
    X, W, labels, dloss = inputs(40, 50, 16, torch.bfloat16, 22)
    monkeypatch.setenv("VQ_CHECK", "1")
    _, lse = vq.cross_entropy(X, W, labels)
    dloss[3] = float("inf")
    with pytest.raises(vq.VQError, match="dloss"):
        vq.cross_entropy_backward(dloss, X, W, labels, lse)
    W[3, 3] = float("nan")
    with pytest.raises(vq.VQError, match="W holds"):
        vq.cross_entropy(X, W, labels)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("n", [6927, 683, 1365])
def test_one_weight_for_every_token(dtype, n):
    """A dloss of 1 / n that the type does not hold: its rounding must not move the whole gradient one way.

    The coefficient of the result along the exact gradient: independent roundings of u over thousands of terms leave
    it within u / 4 of 1 (their sum along one direction is that of hundreds of terms at least: u / sqrt(100) and less).
    """
    X, W, labels, _ = inputs(800, 2000, 48, dtype, 23, masked=0.0)
    dloss = torch.full((800,), 1.0 / n, device="cuda")
    _, lse = vq.cross_entropy(X, W, labels)
    for got, want in zip(vq.cross_entropy_backward(dloss, X, W, labels, lse), exact_on_gpu(X, W, labels, dloss, lse)):
        along = float((got.double() * want).sum() / want.square().sum())
        assert abs(along - 1) <= ref.UNIT[dtype] / 4
