"""A dense product of more small tiles than one launch takes."""
import pytest
import torch

from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu


def test_gated_of_the_most_tokens():
    """2^28 tokens by a pair of 193 rows: 2^23 tiles of 128 tokens by 64 rows, and 104 GB of results."""
    T, M = 1 << 28, 193
    X = torch.ones((T, 1), dtype=torch.float16, device="cuda")
    X[T - 1, 0], X[T // 2, 0] = 2.0, -2.0
    W = torch.ones((M, 1), dtype=torch.float16, device="cuda")
    H = vq.gated(X, W, W, act="none")
    assert bool((H[T - 1] == 4.0).all()) and bool((H[T // 2] == 4.0).all())
    assert bool((H[:1 << 20] == 1.0).all()) and bool((H[T - 1 - (1 << 20):T - 1] == 1.0).all())
