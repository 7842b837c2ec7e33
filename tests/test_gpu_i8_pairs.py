"""Pairs of 8-bit matrices whose codes' rows are not equally far apart."""
import pytest
import torch

from hessian_weighted_vector_amd import block, vq

pytestmark = pytest.mark.gpu


def matrices(M, N, more, seed):
    """One matrix twice: kept in place in rows `more` bytes wider, and made with the nearest rows."""
    g = torch.Generator().manual_seed(seed)
    ld = -(-N // 64) * 64
    wide = torch.randint(-128, 128, (M, ld + more), generator=g).to(torch.int8).cuda()
    scale = (1e-3 + 1e-3 * torch.rand(M, generator=g)).cuda()
    q = wide[:, :N]
    near = torch.zeros((M, ld), dtype=torch.int8, device="cuda")
    near[:, :N] = q
    return vq.Int8Matrix(q, scale), vq.Int8Matrix(near[:, :N], scale)


@pytest.mark.parametrize("T", [1, 20, 70])
def test_pair_of_different_rows(T):
    g = torch.Generator().manual_seed(T)
    wide, gate = matrices(96, 200, 64, 1)
    _, up = matrices(96, 200, 64, 2)
    _, down = matrices(200, 96, 0, 3)
    X = torch.randn((T, 200), generator=g).bfloat16().cuda()
    assert wide.q.stride(0) == 320 and gate.q.stride(0) == up.q.stride(0) == 256
    want = vq.gated_i8(gate, up, X)
    for a, b in ((wide, up), (gate, wide)):
        with pytest.raises(ValueError, match="compact"):
            vq.gated_i8(a, b, X)
    near = wide.compact()
    assert near is not wide and near.q.stride(0) == 256 and near.scale is wide.scale and gate.compact() is gate
    assert torch.equal(vq.gated_i8(near, up.compact(), X), want)
    assert torch.equal(vq.linear_i8(near, X), vq.linear_i8(wide, X))
    a, b = block.Int8Block(wide, up, down), block.Int8Block(gate, up, down)
    assert torch.equal(a.forward(X), b.forward(X))
    a, b = block.Int8Block(up, wide, down), block.Int8Block(up, gate, down)
    assert torch.equal(a.forward(X), b.forward(X))
    both = block.Int8Block(wide, wide, down)                  # the same rows: as they are
    assert both.gate is wide and torch.equal(both.forward(X), block.Int8Block(gate, gate, down).forward(X))
