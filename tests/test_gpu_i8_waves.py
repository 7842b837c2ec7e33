"""8-bit products of few tokens by 128 to 255 groups of 16 long rows: workgroups of sixteen waves."""
import pytest
import torch

import i8_reference as ref
from hessian_weighted_vector_amd import vq
from test_gpu_i8 import HALF, matrix, values, within

pytestmark = pytest.mark.gpu


# groups of 16 rows: 128, the least; 157; 255, the most; rows of 8129 columns are the shortest
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N", [(2048, 8192), (2500, 9001), (4065, 8129), (2049, 16500)])
def test_sixteen_waves(M, N, dtype):
    g = torch.Generator().manual_seed(M)
    X = values((32, N), dtype, g)
    R = values((32, M), dtype, g)
    b = values((1, M), dtype, g)[0].contiguous()
    Q, q, s = matrix(M, N, g)
    Q2, q2, s2 = matrix(M, N, g)
    linear = ref.linear(X, q, s, b, R, "silu", dtype)
    gated = ref.gated(X, q, s, q2, s2, None, b, "silu", dtype)
    all_linear = vq.linear_i8(Q, X, bias=b, residual=R, act="silu")
    all_gated = vq.gated_i8(Q, Q2, X, bias_up=b)
    for T in (1, 2, 3, 15, 16, 17, 20, 32):
        got = vq.linear_i8(Q, X[:T], bias=b, residual=R[:T], act="silu")
        within(got, tuple(t[:T] for t in linear), "linear, %d tokens" % T)
        assert torch.equal(got, all_linear[:T])
        got = vq.gated_i8(Q, Q2, X[:T], bias_up=b)
        within(got, tuple(t[:T] for t in gated), "gated, %d tokens" % T)
        assert torch.equal(got, all_gated[:T])


@pytest.mark.parametrize("T", [1, 2, 5, 20])
def test_rows_that_are_not_finite_and_zeros(T):
    g = torch.Generator().manual_seed(5)
    Q, q, s = matrix(2300, 8200, g)
    X = values((T, 8200), torch.bfloat16, g)
    X[T - 1, 8199] = float("inf")
    got = vq.linear_i8(Q, X)
    assert bool(torch.isnan(got[T - 1]).all()) and bool(torch.isfinite(got[:T - 1]).all())
    assert not bool(vq.linear_i8(Q, torch.zeros_like(X)).any())


def test_odd_rows_of_tokens():
    """Tokens that begin at odd elements of their buffer."""
    g = torch.Generator().manual_seed(6)
    Q, q, s = matrix(2100, 8333, g)
    for T in (1, 2, 9):
        X = values((T, 8333), torch.float16, g, 1, 3)
        within(vq.linear_i8(Q, X), ref.linear(X, q, s, None, None, "none", torch.float16), "%d tokens" % T)
