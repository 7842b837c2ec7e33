"""8-bit moments are, byte for byte, the codes of float32's quotients.

The arithmetic before the codes is the same with 32-bit moments, so an optimizer with those, begun
from the same values, holds what is coded; here it is divided as float32 divides.
"""
import pytest
import torch

from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu

B = 256


def spread(s, n):
    return torch.repeat_interleave(s, B)[:n]


def root_of(x):
    """float32's root: torch's own of many elements is not always the nearest, that of 64 bits rounded is."""
    return x.double().sqrt().float()


def codes(x, scale, root):
    """The nearest e4m3 codes (ties to even) of x / scale, or of the roots of x, at least the smallest where x > 0."""
    v = root_of(x) if root else x
    s = spread(scale, len(x))
    y = torch.where(s > 0, v / torch.where(s > 0, s, torch.ones_like(s)), v).clamp(-448, 448)
    if root:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn)


def check(grads, betas):
    n = len(grads[0])
    opts = [vq.AdamW([torch.zeros(n, dtype=torch.float32, device="cuda")], lr=1e-3, betas=betas, state_bits=bits) for bits in (8, 32)]
    small, wide = opts
    for g in grads:
        g = g.cuda()
        # the wide one begins where the codes are: one product, and for v its square
        for k in ("m", "v"):
            x = small.state[k][0].float() * spread(small.state[k + "_scale"][0], n)
            wide.state[k][0].copy_(x if k == "m" else x * x)
        for opt in opts:
            opt.step([g])
        for k in ("m", "v"):
            x, scale = wide.state[k][0].cpu(), small.state[k + "_scale"][0].cpu()
            pad = torch.zeros(len(scale) * B)
            pad[:n] = torch.where(torch.isnan(x), 0.0, x.abs())              # a NaN has no part in its block's scale
            top = pad.view(-1, B).amax(1)
            want = (root_of(top) if k == "v" else top) * torch.tensor(1 / 448, dtype=torch.float32)
            none = torch.isnan(torch.nn.functional.pad(x, (0, len(pad) - n), value=float("nan"))).view(-1, B).all(1)
            wrong = ((scale != want) & ~none).nonzero()[:, 0]                # blocks of NaN alone have any scale
            assert len(wrong) == 0, "%s_scale: %d, first at %d: %r, %r" % (k, len(wrong), wrong[0], scale[wrong[0]], want[wrong[0]])
            got, want = small.state[k][0].cpu(), codes(x, scale, k == "v")
            bad = ((want.view(torch.uint8) != got.view(torch.uint8)) & ~(torch.isnan(want.float()) & torch.isnan(got.float()))).nonzero()[:, 0]
            assert len(bad) == 0, "%s: %d codes, first at %d: %r" % (k, len(bad), bad[0], float(x[bad[0]]))


def test_values_of_every_size():
    """Blocks from subnormal moments to infinite ones: divided ones and multiplied ones."""
    g = torch.Generator().manual_seed(1)
    n = 4000 * B + 77
    size = spread(10.0 ** torch.linspace(-42, 17, 4001, dtype=torch.float64), n)
    grads = [(torch.randn(n, generator=g, dtype=torch.float64) * torch.exp(2 * torch.randn(n, generator=g, dtype=torch.float64)) * size).float()
             for _ in range(3)]
    check(grads, (0.9, 0.97))


@pytest.mark.parametrize("of", ["quotients", "roots"])
def test_values_next_to_ties(of):
    """Moments of nothing but the gradient: quotients at the middle of two codes and a few last places beside it."""
    g = torch.Generator().manual_seed(2)
    c = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    middle = torch.cat([(c[1:] + c[:-1]) / 2, (c[:1] / 2)])                  # 126 of them, below 448
    blocks = 4000
    s = torch.exp(4 * torch.randn(blocks, 1, generator=g))
    x = torch.full((blocks, B), 448.0) * s
    scale = (x[:, :1] if of == "quotients" else root_of(x[:, :1] * x[:, :1])) * torch.tensor(1 / 448, dtype=torch.float32)
    at = torch.randint(0, 126, (blocks, B - 1), generator=g)
    near = middle[at] * scale
    places = torch.randint(-3, 4, near.shape, generator=g)
    near = (near.view(torch.int32) + places.int()).view(torch.float32)
    x[:, 1:] = near * torch.where(torch.rand(near.shape, generator=g) < 0.5, -1.0, 1.0)
    check([x.reshape(-1)], (0.0, 0.0))
