"""Refusals of the cross entropy calls without a GPU, and the reference's own gradients."""
import pytest
import torch

import loss_reference as ref
from hessian_weighted_vector_amd import vq

FAKE = 0x10000            # never dereferenced
BF16, F16, F32 = 0, 1, 2


def forward(T=4, V=8, N=16, dt=BF16, X=FAKE, ldx=16, W=FAKE + 4096, ldw=16, labels=FAKE + 8192, loss=FAKE + 12288,
            lse=FAKE + 16384, ws=None, n=0):
    lib = vq.load()
    st = lib.vq_cross_entropy(T, V, N, dt, X, ldx, W, ldw, labels, -100, loss, lse, ws, n, None)
    return st, lib.vq_last_error().decode()


@pytest.mark.parametrize("change,msg", [
    (dict(T=-1), "T must"), (dict(T=(1 << 20) + 1), "T must"), (dict(V=0), "V and N"), (dict(N=0), "V and N"),
    (dict(V=(1 << 20) + 1), "V and N"), (dict(dt=F32), "dtype"), (dict(X=None), "null"), (dict(W=None), "null"),
    (dict(labels=None), "null"), (dict(loss=None), "null"), (dict(lse=None), "null"),
    (dict(ldx=15), "leading dimension of X"), (dict(ldw=15), "leading dimension of W"), (dict(X=FAKE + 1), "aligned"),
    (dict(labels=FAKE + 4), "labels is not aligned"), (dict(loss=FAKE + 2), "loss is not aligned"),
    (dict(lse=FAKE + 12288), "alias each other"), (dict(loss=FAKE + 8192), "alias inputs"),
])
def test_forward_refuses(change, msg):
    st, text = forward(**change)
    assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_cross_entropy:")


def test_workspaces():
    lib = vq.load()
    need = lib.vq_cross_entropy_workspace_bytes(4, 8, 16, FAKE, 16)
    assert need > 0
    st, text = forward(ws=FAKE + 65536, n=need - 1)
    assert st == vq.VQ_ERR_WORKSPACE
    st, text = forward(ws=FAKE + 65536 + 8, n=need)
    assert st == vq.VQ_ERR_INVALID and "16-byte" in text
    assert forward(T=0, X=None)[0] == vq.VQ_OK
    assert lib.vq_cross_entropy_workspace_bytes(4, 0, 16, FAKE, 16) == 0
    # odd rows of W are copied, a piece at a time
    a = lib.vq_cross_entropy_workspace_bytes(512, 512, 512, FAKE, 512)
    b = lib.vq_cross_entropy_workspace_bytes(512, 512, 512, FAKE, 513)
    assert b - a == 512 * 512 * 2
    big = lib.vq_cross_entropy_workspace_bytes(512, 1 << 20, 512, FAKE, 513) - \
        lib.vq_cross_entropy_workspace_bytes(512, 1 << 20, 512, FAKE, 512)
    assert big <= (129 << 20)
    # dz of a piece, not of the vocabulary
    n = lib.vq_cross_entropy_backward_workspace_bytes(8192, 1 << 20, 64, FAKE, 64, 0, 1)
    assert n <= (140 << 20)
    assert lib.vq_cross_entropy_backward_workspace_bytes(64, 64, 64, FAKE, 64, 0, 0) == 0


def test_backward_refuses():
    lib = vq.load()
    A, B, C, D = FAKE, FAKE + 4096, FAKE + 8192, FAKE + 16384

    def back(T=4, dloss=A, X=B, ldx=16, W=C, ldw=16, labels=D, lse=D + 4096, dX=D + 8192, lddx=16, dW=D + 12288, lddw=16, dt=F16):
        st = lib.vq_cross_entropy_backward(T, 8, 16, dt, dloss, X, ldx, W, ldw, labels, -100, lse, dX, lddx, dW, lddw, None, 0, None)
        return st, lib.vq_last_error().decode()

    for kw, msg in ((dict(dloss=None), "null"), (dict(X=None), "null"), (dict(W=None), "null"), (dict(labels=None), "null"),
                    (dict(lse=None), "null"), (dict(lddx=15), "leading dimension of dX"), (dict(lddw=8), "leading dimension of dW"),
                    (dict(dX=B), "alias inputs"), (dict(dW=C), "alias inputs"), (dict(dW=D + 8192), "alias each other"),
                    (dict(dX=A), "alias inputs"), (dict(dt=F32), "dtype"), (dict(T=-1), "T must"), (dict(dloss=A + 2), "dloss is not"),
                    (dict(lse=D + 4098), "lse is not"), (dict(dX=D + 8193), "aligned")):
        st, text = back(**kw)
        assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_cross_entropy_backward:"), kw
    assert back()[0] == vq.VQ_ERR_WORKSPACE
    assert back(dX=None, dW=None)[0] == vq.VQ_OK              # nothing wanted
    assert back(T=0, dW=None)[0] == vq.VQ_OK


def test_python_checks():
    X = torch.zeros((4, 16), dtype=torch.bfloat16)
    W = torch.zeros((8, 16), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bfloat16 or torch.float16"):
        vq.cross_entropy(X.float(), W.float(), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        vq.cross_entropy(X, W, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="matrices"):
        vq.cross_entropy_backward(torch.zeros(4), X[0], W, torch.zeros(4, dtype=torch.int64), torch.zeros(4))


def test_reference_against_differences():
    """The reference's gradients are those of sum(dloss * loss): central differences in float64."""
    g = torch.Generator().manual_seed(0)
    T, V, N = 5, 7, 3
    X = torch.randn((T, N), generator=g).half()
    W = torch.randn((V, N), generator=g).half()
    labels = torch.tensor([0, 6, -100, 3, 3])
    dloss = torch.randn(T, generator=g)
    lse = torch.logsumexp(ref.f64(X) @ ref.f64(W).T, 1)

    def total(x, w):
        z = x @ w.T
        on = labels != -100
        per = torch.logsumexp(z, 1) - z[torch.arange(T), labels.clamp(min=0)]
        return float((per * dloss.double() * on).sum())

    (dX, _), (dW, _) = ref.backward(dloss, X, W, labels, lse, -100)
    h = 1e-6
    for grad, which in ((dX, 0), (dW, 1)):
        for i in range(grad.shape[0]):
            for j in range(grad.shape[1]):
                a = [ref.f64(X).clone(), ref.f64(W).clone()]
                b = [ref.f64(X).clone(), ref.f64(W).clone()]
                a[which][i, j] += h
                b[which][i, j] -= h
                assert abs((total(*a) - total(*b)) / (2 * h) - float(grad[i, j])) < 1e-7
