"""The codes of float32 rows over the whole range of the type."""
import pytest
import torch

from ffn_reference import f64
from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu

LARGEST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("N", [1, 9, 300, 5000])
@pytest.mark.parametrize("top", [LARGEST, 3e38, 2.0 ** 121, 2.0 ** 120, 2.7e36, 1.0, 2.0 ** -100, 2.0 ** -126, 2.0 ** -149])
def test_float32_rows_of_every_size(top, N):
    g = torch.Generator().manual_seed(N)
    X = ((2 * torch.rand((16, N), generator=g, dtype=torch.float64) - 1) * top).float()
    X[:, N - 1] = top
    X[3, N - 1] = -top
    X[5] = top
    q, s = vq.quantize_rows(X.cuda())
    x = f64(X)
    most = x.abs().amax(1, keepdim=True)
    # 127 x and the quotient are rounded once each, at most 127 2^-24 apiece (a subnormal 127 x is exact)
    assert bool(((127 * x / most - q.cpu().double()).abs() <= 0.5 + 127 * 2.0 ** -23).all())
    assert q[:, N - 1].tolist() == [-127 if r == 3 else 127 for r in range(16)]
    assert bool(((most[:, 0] / 127 - f64(s)).abs() <= 2.0 ** -24 * most[:, 0] / 127 + 2.0 ** -150).all())


def test_a_power_of_two_changes_no_code():
    g = torch.Generator().manual_seed(8)
    X = torch.randn((64, 777), generator=g)
    X[:, 5] = X.abs().amax(1)                                # the largest magnitude of each row, below 8
    want, _ = vq.quantize_rows(X.cuda())
    for power in range(110, 126):
        got, _ = vq.quantize_rows((X * 2.0 ** power).cuda())
        assert torch.equal(got, want), power
