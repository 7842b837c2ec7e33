"""Refusals of the feed-forward calls without a GPU: every case fails validation on the host."""
import math

import pytest
import torch

import ffn_reference as ref
from hessian_weighted_vector_amd import vq

FAKE = 0x10000            # never dereferenced
BF16, F16, F32 = 0, 1, 2


def linear(T=4, M=8, N=16, dt=BF16, act=0, X=FAKE, ldx=16, W=FAKE + 4096, ldw=16, b=None, R=None, ldr=8,
           Y=FAKE + 8192, ldy=8, Z=None, ldz=8, ws=None, n=0):
    lib = vq.load()
    return lib.vq_linear(T, M, N, dt, act, X, ldx, W, ldw, b, R, ldr, Y, ldy, Z, ldz, ws, n, None), \
        lib.vq_last_error().decode()


@pytest.mark.parametrize("change,msg", [
    (dict(T=-1), "T must"), (dict(M=0), "M and N"), (dict(N=0), "M and N"), (dict(N=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), "M and N"),
    (dict(dt=F32), "dtype"), (dict(dt=-1), "dtype"), (dict(act=6), "activation"), (dict(act=-1), "activation"),
    (dict(X=None), "null"), (dict(W=None), "null"), (dict(Y=None), "null"),
    (dict(ldx=15), "leading dimension of X"), (dict(ldw=15), "leading dimension of W"),
    (dict(ldy=7), "leading dimension of Y"), (dict(R=FAKE + 64, ldr=7), "leading dimension of R"),
    (dict(Z=FAKE + 64, ldz=7), "leading dimension of Z"), (dict(X=FAKE + 1), "aligned"),
    (dict(Y=FAKE), "alias"), (dict(Z=FAKE + 8192), "alias"), (dict(Z=FAKE), "alias"),
    (dict(R=FAKE + 8192, ldr=16), "in place"),
])
def test_linear_refuses(change, msg):
    st, text = linear(**change)
    assert st == vq.VQ_ERR_INVALID
    assert msg in text and text.startswith("vq_linear")


def test_gated_and_backward_refuse():
    lib = vq.load()
    A, B, C, D = FAKE, FAKE + 4096, FAKE + 8192, FAKE + 16384

    def gated(T=4, M=8, N=16, dt=BF16, act=2, X=A, Wg=B, Wu=C, ldw=16, H=D, ldh=8, G=None, U=None):
        return lib.vq_gated(T, M, N, dt, act, X, 16, Wg, Wu, ldw, None, None, H, ldh, G, U, 8, None, 0, None)

    for kw in (dict(Wu=None), dict(G=D + 4096), dict(ldw=8), dict(H=B), dict(G=D, U=D + 4096), dict(G=D + 64, U=D + 64),
               dict(dt=F32), dict(act=9), dict(T=-2)):
        assert gated(**kw) == vq.VQ_ERR_INVALID, kw
        assert lib.vq_last_error().decode().startswith("vq_gated:"), kw

    def lback(T=4, act=2, dY=A, X=B, W=C, Z=D, dX=D + 4096, dW=D + 8192, db=None, lddx=16):
        return lib.vq_linear_backward(T, 8, 16, F16, act, dY, 8, X, 16, W, 16, Z, 8, dX, lddx, dW, 16, db, None, 0, None)

    for kw in (dict(dY=None), dict(Z=None), dict(X=None), dict(W=None), dict(dX=A), dict(dW=B), dict(lddx=15), dict(act=-1)):
        assert lback(**kw) == vq.VQ_ERR_INVALID, kw
        assert lib.vq_last_error().decode().startswith("vq_linear_backward:"), kw

    def gback(dH=A, X=B, Wg=C, Wu=C + 2048, G=D, U=D + 2048, dX=D + 4096, dWg=D + 8192, dWu=D + 12288, dbg=None, dbu=None):
        return lib.vq_gated_backward(4, 8, 16, BF16, 2, dH, 8, X, 16, Wg, Wu, 16, G, U, 8, dX, 16, dWg, dWu, 16, dbg, dbu,
                                     None, 0, None)

    for kw in (dict(dH=None), dict(G=None), dict(U=None), dict(Wg=None), dict(X=None), dict(dWu=None), dict(dWu=D + 8192),
               dict(dbg=D + 32768), dict(dX=A), dict(dWg=B)):
        assert gback(**kw) == vq.VQ_ERR_INVALID, kw
        assert lib.vq_last_error().decode().startswith("vq_gated_backward:"), kw


def test_workspace_queries():
    lib = vq.load()
    # sizes that the calls reject
    assert lib.vq_linear_workspace_bytes(4, 0, 16, FAKE, 16, FAKE, 16) == 0
    assert lib.vq_gated_workspace_bytes(-1, 8, 16, FAKE, 16, FAKE, FAKE, 16) == 0
    # rows that are not 16-byte aligned are copied: the query depends on stride and address
    a = lib.vq_linear_workspace_bytes(512, 512, 512, FAKE, 512, FAKE, 512)
    b = lib.vq_linear_workspace_bytes(512, 512, 512, FAKE, 513, FAKE, 512)
    c = lib.vq_linear_workspace_bytes(512, 512, 512, FAKE + 2, 512, FAKE, 512)
    assert b - a == c - a == 512 * 512 * 2
    # the gradients of the pre-activations live in the workspace
    n = lib.vq_gated_backward_workspace_bytes(64, 96, 32, 2, FAKE, 96, FAKE, 32, FAKE, FAKE, 32, 1, 1, 0)
    assert n >= 2 * 64 * 96 * 2


def test_python_checks():
    X = torch.zeros((4, 16), dtype=torch.bfloat16)
    W = torch.zeros((8, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        vq.linear(X, W)
    with pytest.raises(TypeError, match="bfloat16 or torch.float16"):
        vq.linear(X.float(), W.float())
    with pytest.raises(ValueError, match="act must be one of"):
        vq.linear(X, W, act="tanh")
    with pytest.raises(ValueError, match="matrices"):
        vq.linear(X[0], W)
    with pytest.raises(ValueError, match="pre is needed"):
        vq.linear_backward(X, X, W, act="silu")


def test_reference_derivatives_against_differences():
    """The reference's act_grad is the derivative of its act (float64 central differences)."""
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.0123
    h = 1e-6
    for name in ref.ACTS:
        fd = (ref.act(name, z + h) - ref.act(name, z - h)) / (2 * h)
        assert torch.allclose(ref.act_grad(name, z), fd, rtol=0, atol=1e-8), name
        assert float(ref.act_grad(name, z).abs().max()) <= ref.LIPSCHITZ
    assert math.isclose(float(ref.act("gelu", torch.tensor(1.0, dtype=torch.float64))), 0.8413447460685429, rel_tol=1e-12)


def qmatrix(**change):
    f = dict(M=32, N=64, d=8, K1=16, K2=0, C1=FAKE, idx1=FAKE + 4096, C2=None, idx2=None, rscale=None, cscale=None,
             row_ptr=None, col=None, delta=None)
    f.update(change)
    return vq.QMatrixStruct(*[f[k] for k, _ in vq.QMatrixStruct._fields_])


@pytest.mark.parametrize("change,msg", [
    (dict(M=0), "positive"), (dict(N=60), "multiple"), (dict(d=9), "d must"), (dict(K1=0), "K must"),
    (dict(K1=257), "exceeds"), (dict(C1=None), "null"), (dict(idx1=None), "null"),
    (dict(C2=FAKE, K2=4), "idx2"), (dict(C2=FAKE, idx2=FAKE, K2=0), "K must"),
    (dict(row_ptr=FAKE), "col and delta"), (dict(row_ptr=FAKE, col=FAKE), "col and delta"),
])
def test_compressed_calls_refuse_bad_matrices(change, msg):
    import ctypes
    lib = vq.load()
    good, bad = qmatrix(), qmatrix(**change)
    X, Y = FAKE + 8192, FAKE + 16384
    assert lib.vq_qlinear(ctypes.byref(bad), 1, F32, 0, X, 64, None, None, 0, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
    assert msg in lib.vq_last_error().decode()
    for a, b in ((bad, good), (good, bad)):
        assert lib.vq_qgated(ctypes.byref(a), ctypes.byref(b), 1, F32, 0, X, 64, None, None, Y, 32, None, 0,
                             None) == vq.VQ_ERR_INVALID


def test_compressed_calls_refuse_bad_arguments():
    import ctypes
    lib = vq.load()
    X, Y = FAKE + 8192, FAKE + 16384

    def qlin(T=1, dt=F32, act=0, X=X, ldx=64, R=None, ldr=32, Y=Y, ldy=32):
        st = lib.vq_qlinear(ctypes.byref(qmatrix()), T, dt, act, X, ldx, None, R, ldr, Y, ldy, None, 0, None)
        return st, lib.vq_last_error().decode()

    for kw, msg in ((dict(T=-1), "T must"), (dict(dt=3), "dtype"), (dict(act=7), "activation"), (dict(X=None), "null"),
                    (dict(Y=None), "null"), (dict(ldx=63), "leading dimension of X"), (dict(ldy=31), "output"),
                    (dict(R=FAKE, ldr=31), "R"), (dict(Y=X), "alias"), (dict(X=X + 2), "aligned"),
                    (dict(R=Y, ldr=64), "in place")):
        st, text = qlin(**kw)
        assert st == vq.VQ_ERR_INVALID and msg in text, (kw, text)
    assert lib.vq_qlinear(None, 1, F32, 0, X, 64, None, None, 0, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
    assert lib.vq_qgated(ctypes.byref(qmatrix()), ctypes.byref(qmatrix(M=48)), 1, F32, 0, X, 64, None, None, Y, 48, None, 0,
                         None) == vq.VQ_ERR_INVALID
    assert "differ" in lib.vq_last_error().decode()
    assert lib.vq_sparse_delta(ctypes.byref(qmatrix()), FAKE, FAKE, None) == vq.VQ_ERR_INVALID
    # rows split over workgroups need their parts' workspace
    need = lib.vq_qlinear_workspace_bytes(32, 65536, 8, 4)
    assert need >= 2 * 4 * 32 * 4
    big = qmatrix(N=65536)
    assert lib.vq_qlinear(ctypes.byref(big), 4, F32, 0, X, 65536, None, None, 0, Y, 32, FAKE, need - 1,
                          None) == vq.VQ_ERR_WORKSPACE
    assert lib.vq_qlinear_workspace_bytes(32, 60, 8, 4) == 0


def test_qmatrix_checks():
    C1 = torch.zeros((16, 8))
    idx = torch.zeros(32 * 8, dtype=torch.uint16)
    with pytest.raises(ValueError, match="idx1 must have 256"):
        vq.QMatrix(32, 64, 8, C1, idx[:-1])
    with pytest.raises(TypeError, match="idx1 must be"):
        vq.QMatrix(32, 64, 8, C1, idx.to(torch.int32))
    with pytest.raises(ValueError, match="C1 must be"):
        vq.QMatrix(32, 64, 8, C1[:, :4], idx)
    with pytest.raises(ValueError, match="come together"):
        vq.QMatrix(32, 64, 8, C1, idx, C2=C1)
    with pytest.raises(ValueError, match="GPU"):
        vq.QMatrix(32, 64, 8, C1, idx)


def test_workspaces_off_16_bytes_are_refused():
    """Parts and copies in the workspace are accessed 16 bytes at a time: an odd base is an error, before any launch."""
    import ctypes
    lib = vq.load()
    T = M = N = 512
    A, B, C, D, E = (FAKE + (k << 24) for k in range(5))
    F, G, H = (FAKE + (k << 24) for k in range(5, 8))
    ld = 513                                  # odd rows: every operand is copied
    n = 1 << 30
    q = qmatrix(M=32, N=65536)                # rows split over workgroups

    calls = {
        "vq_linear": lambda ws: lib.vq_linear(T, M, N, BF16, 2, A, ld, B, ld, None, None, 0, C, M, None, 0, ws, n, None),
        "vq_gated": lambda ws: lib.vq_gated(T, M, N, BF16, 2, A, ld, B, C, ld, None, None, D, M, None, None, 0, ws, n, None),
        "vq_linear_backward": lambda ws: lib.vq_linear_backward(T, M, N, F16, 2, A, ld, B, ld, C, ld, D, ld, E, N, F, N, None,
                                                                ws, n, None),
        "vq_gated_backward": lambda ws: lib.vq_gated_backward(T, M, N, F16, 2, A, ld, B, ld, C, D, ld, E, F, ld, G, N, H, A + 64,
                                                              N, None, None, ws, n, None),
        "vq_qlinear": lambda ws: lib.vq_qlinear(ctypes.byref(q), 4, F32, 0, A, 65536, None, None, 0, B, 32, ws, n, None),
        "vq_qgated": lambda ws: lib.vq_qgated(ctypes.byref(q), ctypes.byref(q), 4, F32, 0, A, 65536, None, None, B, 32, ws, n,
                                              None),
    }
    for name, call in calls.items():
        for off in (1, 2, 4, 8, 20):
            assert call((1 << 36) + off) == vq.VQ_ERR_INVALID, (name, off)
            text = lib.vq_last_error().decode()
            assert text.startswith(name) and "16-byte aligned" in text, (name, off, text)
        assert call(None) == vq.VQ_ERR_WORKSPACE, name


def test_outputs_at_one_address_are_refused():
    """Two outputs at one address, or an output at a bias's, would be written over each other."""
    lib = vq.load()
    P = [FAKE + 4096 * k for k in range(16)]
    X, W, W2, Z, Z2, D, o1, o2, o3, o4, o5, b = P[:12]

    def lback(dX=o1, dW=o2, db=o3):
        return lib.vq_linear_backward(4, 8, 16, F16, 2, D, 8, X, 16, W, 16, Z, 8, dX, 16, dW, 16, db, None, 0, None)

    def gback(dX=o1, dWg=o2, dWu=o3, dbg=o4, dbu=o5):
        return lib.vq_gated_backward(4, 8, 16, BF16, 2, D, 8, X, 16, W, W2, 16, Z, Z2, 8, dX, 16, dWg, dWu, 16, dbg, dbu,
                                     None, 0, None)

    def refuse(st, call, kw):
        assert st == vq.VQ_ERR_INVALID, (call, kw)
        text = lib.vq_last_error().decode()
        assert text.startswith(call + ":") and "alias" in text, (kw, text)

    for kw in (dict(dX=o2), dict(db=o2), dict(db=o1)):
        refuse(lback(**kw), "vq_linear_backward", kw)
    for kw in (dict(dX=o2), dict(dX=o3), dict(dWu=o2), dict(dbu=o4), dict(dbg=o1), dict(dbu=o3)):
        refuse(gback(**kw), "vq_gated_backward", kw)
    refuse(lib.vq_linear(4, 8, 16, BF16, 0, X, 16, W, 16, b, None, 0, b, 8, None, 0, None, 0, None), "vq_linear", "Y is the bias")
    refuse(lib.vq_linear(4, 8, 16, BF16, 0, X, 16, W, 16, b, None, 0, o1, 8, b, 8, None, 0, None), "vq_linear", "Z is the bias")
    refuse(lib.vq_gated(4, 8, 16, BF16, 2, X, 16, W, W2, 16, None, b, o1, 8, o2, b, 8, None, 0, None), "vq_gated", "U is a bias")
    # apart, the calls reach the workspace's check
    for st in (lback(), gback()):
        assert st == vq.VQ_ERR_WORKSPACE


class Elsewhere:
    """Stands for a bfloat16 matrix or vector on GPU `index`; never dereferenced."""
    is_cuda = True

    def __init__(self, *shape, index=1, dtype=torch.bfloat16):
        self.shape, self.index, self.dtype = torch.Size(shape), index, dtype

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return (self.shape[-1], 1) if len(self.shape) == 2 else (1,)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return FAKE


def test_tensors_of_another_gpu_are_refused(monkeypatch):
    """The launches go to the current GPU's stream: a tensor of another one is an error, not a stray access."""
    monkeypatch.setattr(vq, "_device", lambda: 0)
    X, W, H = Elsewhere(4, 16), Elsewhere(8, 16), Elsewhere(4, 8)

    def here(*shape, **kw):
        return Elsewhere(*shape, index=0, **kw)

    for call, name in [
            (lambda: vq.linear(X, here(8, 16)), "X"), (lambda: vq.linear(here(4, 16), W), "W"),
            (lambda: vq.linear(here(4, 16), here(8, 16), bias=Elsewhere(8)), "bias"),
            (lambda: vq.linear(here(4, 16), here(8, 16), out=H), "out"),
            (lambda: vq.linear(here(4, 16), here(8, 16), out=here(4, 8), ws=Elsewhere(64, dtype=torch.uint8)), "ws"),
            (lambda: vq.gated(here(4, 16), here(8, 16), W), "W_up"),
            (lambda: vq.linear_backward(H, here(4, 16), here(8, 16)), "dY"),
            (lambda: vq.gated_backward(here(4, 8), here(4, 16), here(8, 16), here(8, 16), here(4, 8), H), "U")]:
        with pytest.raises(ValueError, match=name + " must be on the current GPU 0, is on 1"):
            call()

    f32 = dict(dtype=torch.float32)
    with pytest.raises(ValueError, match="idx1 must be on the current GPU"):
        vq.QMatrix(32, 64, 8, here(16, 8, **f32), Elsewhere(256, dtype=torch.uint16))
    Q = vq.QMatrix.__new__(vq.QMatrix)
    Q.M, Q.N, Q.d, Q._keep, Q.delta, Q.index = 32, 64, 8, (Elsewhere(16, 8, **f32),), None, 1
    for call in (lambda: vq.qlinear(Q, here(1, 64, **f32)), lambda: vq.qgated(Q, Q, here(1, 64, **f32)), Q.refresh):
        with pytest.raises(ValueError, match="on the current GPU 0, is on 1"):
            call()


def test_compressed_calls_check_residual_and_biases():
    """A residual or bias off its elements' boundary, a residual's row distance out of range, an output at a bias."""
    import ctypes
    lib = vq.load()
    q = ctypes.byref(qmatrix())
    X, Y, Z = FAKE + 8192, FAKE + 16384, FAKE + 32768
    for dt, off in ((F32, 2), (F32, 1), (BF16, 1), (F16, 1)):
        for b, R in ((Z + off, None), (None, Z + off)):
            assert lib.vq_qlinear(q, 1, dt, 0, X, 64, b, R, 32, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
            assert "not aligned" in lib.vq_last_error().decode()
        for bg, bu in ((Z + off, None), (None, Z + off)):
            assert lib.vq_qgated(q, q, 1, dt, 0, X, 64, bg, bu, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
            assert "not aligned" in lib.vq_last_error().decode()
    for ldr in (31, -1, (1 << 40) + 1):
        assert lib.vq_qlinear(q, 1, F32, 0, X, 64, None, Z, ldr, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
        assert "leading dimension of R" in lib.vq_last_error().decode()
    assert lib.vq_qlinear(q, 1, F32, 0, X, 64, Y, None, 0, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
    assert lib.vq_qgated(q, q, 1, F32, 0, X, 64, None, Y, Y, 32, None, 0, None) == vq.VQ_ERR_INVALID
    assert "bias" in lib.vq_last_error().decode()
