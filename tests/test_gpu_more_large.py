"""Offsets past 32 bits: the last rows and elements of the largest tensors of the loss, 8-bit and AdamW calls."""
import math

import pytest
import torch

from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu

V, N = 1 << 20, 4104              # 8.6 GB in 16 bits, 4.3 GB in 8


@pytest.mark.parametrize("T", [3, 40])
def test_cross_entropy_of_the_largest_vocabulary(T):
    """All words alike but the last few: closed forms of the loss and of the gradient's last rows."""
    W = torch.zeros((V, N), dtype=torch.bfloat16, device="cuda")
    W[V - 1, N - 1] = 8.0
    W[V - 2, 0] = 2.0
    X = torch.ones((T, N), dtype=torch.bfloat16, device="cuda")
    labels = torch.full((T,), V - 1, device="cuda")
    labels[1] = 5
    loss, lse = vq.cross_entropy(X, W, labels)
    total = math.exp(8.0) + math.exp(2.0) + V - 2
    want = torch.full((T,), math.log(total) - 8.0)
    want[1] = math.log(total)
    # sums of 2^20 float32 terms in a tree and one logarithm
    assert float((loss.cpu() - want).abs().max()) <= 1e-5
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dX, dW = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    p = [math.exp(8.0) / total, math.exp(2.0) / total, 1.0 / total]
    rows = {V - 1: p[0] - (T - 1) / T, V - 2: p[1], V - 3: p[2], 5: p[2] - 1 / T, V // 2 + 1: p[2]}
    for v, x in rows.items():
        got = dW[v].float()
        # dz is rounded once before the sum over T equal terms, the result once more: 2^-8 each, twice over for the difference
        assert bool((got == got[0]).all()) and abs(float(got[0]) - x) <= 2.0 ** -6 * abs(x), v
    # dX: only two words have weights
    want0, wantn = p[1] * 2.0 / T, (p[0] - 1) * 8.0 / T
    assert abs(float(dX[0, 0]) - want0) <= 2.0 ** -6 * want0 and abs(float(dX[0, N - 1]) - wantn) <= 2.0 ** -6 * abs(wantn)
    assert abs(float(dX[1, N - 1]) - p[0] * 8.0 / T) <= 2.0 ** -6 * p[0] * 8.0 / T and not bool(dX[:, 1:N - 1].any())


@pytest.mark.parametrize("T", [1, 5, 40])
def test_int8_rows_past_4_gb(T):
    ld = -(-N // 64) * 64
    q = torch.zeros((V, ld), dtype=torch.int8, device="cuda")
    q[V - 1, N - 1], q[V - 2, 3] = 100, -7
    Q = vq.Int8Matrix(q[:, :N], torch.full((V,), 0.5, device="cuda"))
    assert Q.q.data_ptr() == q.data_ptr()
    X = torch.ones((T, N), dtype=torch.float16, device="cuda")
    Y = vq.linear_i8(Q, X)
    assert bool((Y[:, V - 1] == 50.0).all()) and bool((Y[:, V - 2] == -3.5).all()) and not bool(Y[:, :V - 2].any())
    H = vq.gated_i8(Q, Q, X, act="none")
    assert bool((H[:, V - 1] == 2500.0).all()) and not bool(H[:, :V - 2].any())


def test_cross_entropy_of_the_most_tokens():
    """2^20 tokens by more than 2^19 words: more tiles than one launch takes."""
    T, words, n = 1 << 20, (1 << 19) + 1000, 8
    g = torch.Generator().manual_seed(70)
    X = torch.randn((T, n), generator=g).bfloat16().cuda()
    W = torch.randn((words, n), generator=g).bfloat16().cuda()
    labels = torch.randint(0, words, (T,), generator=g).cuda()
    labels[::5] = -100
    loss, lse = vq.cross_entropy(X, W, labels)
    at = torch.tensor([0, 1, 2, 127, 128, T // 2 + 1, T - 2, T - 1])
    z = X[at.cuda()].cpu().double() @ W.cpu().double().T
    want = torch.logsumexp(z, 1)
    for i, t in enumerate(at.tolist()):
        if t % 5 == 0:
            assert float(loss[t]) == 0.0 and float(lse[t]) == 0.0
            continue
        # products exact in float32 but for 8 additions of at most 128, exponents rounded to 2^-24 of at most 256
        assert abs(float(lse[t]) - float(want[i])) <= 1e-4
        assert abs(float(loss[t]) - float(want[i] - z[i, int(labels[t])])) <= 1e-4
    assert bool(torch.isfinite(loss).all()) and bool((loss[labels != -100] > 0).all())


def test_more_tokens_than_one_launch_has_threads():
    """2^32 threads: of the codes from 2^26 rows on, of small tiles from 2^23."""
    T = (1 << 26) + 5
    X = torch.ones((T, 2), dtype=torch.float16, device="cuda")
    X[T - 1, 1], X[1 << 23, 0] = 0.5, -1.0
    Q = vq.Int8Matrix(torch.tensor([[3, 4]], dtype=torch.int8, device="cuda"), torch.full((1,), 0.5, device="cuda"))
    Y = vq.linear_i8(Q, X)[:, 0]
    # the code of 0.5 beside 1 is 64 (63.5 to even): 127 * 3 + 64 * 4 over 127, halved
    assert float(Y[T - 1]) == pytest.approx((127 * 3 + 64 * 4) / 254, rel=2.0 ** -10) and float(Y[1 << 23]) == 0.5
    Y[T - 1], Y[1 << 23] = 3.5, 3.5
    assert bool((Y == 3.5).all())


def test_more_small_tiles_than_one_launch_takes():
    T, M = 1 << 28, 193                                       # 104 GB of results
    X = torch.ones((T, 1), dtype=torch.float16, device="cuda")
    X[T - 1, 0], X[T // 2, 0] = 2.0, -2.0
    q = torch.ones((M, 1), dtype=torch.int8, device="cuda")
    Q = vq.Int8Matrix(q, torch.ones(M, device="cuda"))
    H = vq.gated_i8(Q, Q, X, act="none")
    assert bool((H[T - 1] == 4.0).all()) and bool((H[T // 2] == 4.0).all())
    assert bool((H[:1 << 20] == 1.0).all()) and bool((H[T - 1 - (1 << 20):T - 1] == 1.0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_2_31_elements(bits):
    n = (1 << 31) + 4099
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 31) - 1, 1 << 31, n - 1]
    for i in at:
        g[i] = 1.0
    opt = vq.AdamW([p], [g], lr=0.5, weight_decay=0.0, state_bits=bits)
    opt.step()
    for i in at:
        assert abs(float(p[i]) + 0.5) <= 2.0 ** -8
    assert int(torch.count_nonzero(p)) == len(at)
    assert abs(float(opt.state["m"][0][n - 1].float()) * (float(opt.state["m_scale"][0][-1]) if bits == 8 else 1) - 0.1) <= 1e-6
