"""torch's default type has no part in what the calls allocate: float32 is float32 under every one of them."""
import pytest
import torch

from hessian_weighted_vector_amd import block, vq

TYPES = [torch.bfloat16, torch.float16, torch.float64]


@pytest.fixture(params=TYPES, ids=lambda t: str(t)[6:])
def default_type(request):
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield request.param
    torch.set_default_dtype(before)


class Library:
    """Every entry point succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def no_gpu(monkeypatch):
    """The binding on CPU tensors, with nothing behind it: what it allocates can be looked at."""
    monkeypatch.setattr(vq, "load", Library)
    monkeypatch.setattr(vq, "_home", lambda X, name="X": -1)
    monkeypatch.setattr(vq, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(vq, "_stream", lambda: 0)
    for name in ("_cross_entropy_need", "_cross_entropy_backward_need"):
        monkeypatch.setattr(vq, name, lambda *args: 0)


def test_allocations(default_type, no_gpu, monkeypatch):
    X = torch.zeros((4, 32), dtype=torch.bfloat16)
    q, scale = vq.quantize_rows(X)
    assert q.dtype == torch.int8 and scale.dtype == torch.float32
    assert vq.Int8Matrix.from_dense(X).scale.dtype == torch.float32
    labels = torch.zeros(4, dtype=torch.int64)
    assert [t.dtype for t in vq.cross_entropy(X, X, labels)] == [torch.float32] * 2
    params = [torch.zeros(300, dtype=torch.bfloat16)]
    for bits in (8, 32):
        opt = vq.AdamW(params, state_bits=bits, capturable=True)
        assert opt.lr.dtype == torch.float32 and opt.steps.dtype == torch.int64
        for k, ts in opt.state.items():
            want = torch.float32 if bits == 32 or "scale" in k else torch.float8_e4m3fn
            assert ts is None or all(t.dtype == want for t in ts), k
    seen = []
    monkeypatch.setattr(vq, "cross_entropy_backward", lambda dloss, *rest: seen.append(dloss.dtype))
    head = block.Head(X)
    head.backward((X, labels, None, labels.new_ones(()), -100), scale=2.0)
    assert seen == [torch.float32]


@pytest.mark.gpu
def test_values(default_type):
    """The same bits as under float32."""
    f32 = torch.float32

    def values():
        g = torch.Generator().manual_seed(1)
        X, W = (torch.randn(s, generator=g, dtype=f32).bfloat16().cuda() for s in ((50, 96), (700, 96)))
        labels = torch.randint(0, 700, (50,), generator=g).cuda()
        labels[3] = -100
        head = block.Head(W)
        loss, kept = head.loss(X, labels)
        Q = vq.Int8Matrix.from_dense(W)
        out = [loss, kept[2], *head.backward(kept), *vq.cross_entropy(X, W, labels), *vq.quantize_rows(X.float()), Q.q, Q.scale,
               vq.linear_i8(Q, X)]
        for bits in (8, 32):
            p = [torch.randn(1000, generator=g, dtype=f32).cuda()]
            opt = vq.AdamW(p, [torch.randn(1000, generator=g, dtype=f32).cuda()], lr=1e-2, state_bits=bits, capturable=True)
            opt.step()
            opt.step()
            out += [p[0], opt.state["m"][0].view(torch.uint8)]
        torch.cuda.synchronize()
        return out

    got = values()
    torch.set_default_dtype(f32)
    for a, b in zip(got, values()):
        assert a.dtype == b.dtype and torch.equal(a, b)
