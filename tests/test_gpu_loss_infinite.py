"""A dloss that is not finite changes its own row of dX and dW, and no other row of dX."""
import pytest
import torch

from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("weight", [0.3, 64.0, 1e-5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 7, 2100])                  # the tokens counted by one workgroup each, and by one
def test_rows_of_finite_tokens(T, dtype, weight, bad):
    g = torch.Generator().manual_seed(T)
    V, N = 300, 72
    X, W = (torch.randn(s, generator=g).to(dtype).cuda() for s in ((T, N), (V, N)))
    labels = torch.randint(0, V, (T,), generator=g).cuda()
    loss, lse = vq.cross_entropy(X, W, labels)
    dloss = torch.full((T,), weight, device="cuda")
    want, _ = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    assert bool(torch.isfinite(want).all())
    at = T // 2
    dloss[at] = bad
    got, _ = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    others = torch.arange(T, device="cuda") != at
    assert torch.equal(got[others], want[others]) and not bool(torch.isfinite(got[at]).any())
    # of an ignored token it has no part at all
    labels[at] = -100
    dloss[at] = weight
    want = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    dloss[at] = bad
    got = vq.cross_entropy_backward(dloss, X, W, labels, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
