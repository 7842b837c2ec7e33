"""Refusals of the 8-bit calls without a GPU: every case fails validation on the host."""
import ctypes

import pytest
import torch

from hessian_weighted_vector_amd import vq

FAKE = 0x10000            # never dereferenced
BF16, F16, F32 = 0, 1, 2


def matrix(**change):
    f = dict(M=32, N=100, q=FAKE, ldq=128, scale=FAKE + 8192)
    f.update(change)
    return vq.I8MatrixStruct(*[f[k] for k, _ in vq.I8MatrixStruct._fields_])


def linear(W=None, T=4, dt=BF16, act=0, X=FAKE + 16384, ldx=100, b=None, R=None, ldr=32, Y=FAKE + 32768, ldy=32, ws=None, n=0):
    lib = vq.load()
    W = matrix() if W is None else W
    st = lib.vq_linear_i8(ctypes.byref(W) if W else None, T, dt, act, X, ldx, b, R, ldr, Y, ldy, ws, n, None)
    return st, lib.vq_last_error().decode()


@pytest.mark.parametrize("kw,msg", [
    (dict(W=False), "null"), (dict(W=matrix(M=0)), "M must"), (dict(W=matrix(N=0)), "N must"),
    (dict(W=matrix(N=(1 << 17) + 1, ldq=1 << 18), ldx=1 << 18), "N must"), (dict(W=matrix(q=None)), "null"),
    (dict(W=matrix(scale=None)), "null"), (dict(W=matrix(q=FAKE + 8)), "16-byte"), (dict(W=matrix(ldq=100)), "multiple of 64"),
    (dict(W=matrix(ldq=64)), "multiple of 64"), (dict(W=matrix(ldq=(1 << 22) + 64)), "2^22"),
    (dict(W=matrix(scale=FAKE + 2)), "scale of W"), (dict(T=-1), "T must"), (dict(dt=F32), "dtype"), (dict(act=6), "activation"),
    (dict(X=None), "null"), (dict(Y=None), "null"), (dict(X=FAKE + 16385), "aligned"), (dict(ldx=99), "leading dimension of X"),
    (dict(ldy=31), "leading dimension of Y"), (dict(R=FAKE + 65536, ldr=31), "leading dimension of R"),
    (dict(Y=FAKE + 16384), "alias"), (dict(Y=FAKE), "alias"), (dict(R=FAKE + 32768, ldr=64), "in place"),
])
def test_linear_refuses(kw, msg):
    st, text = linear(**kw)
    assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_linear_i8"), text


def test_gated_refuses():
    lib = vq.load()

    def gated(g=None, u=None, T=4, dt=F16, act=2, X=FAKE + 16384, H=FAKE + 32768, ldh=32):
        g, u = matrix() if g is None else g, matrix(q=FAKE + 4096) if u is None else u
        st = lib.vq_gated_i8(ctypes.byref(g) if g else None, ctypes.byref(u) if u else None, T, dt, act, X, 100, None, None, H, ldh,
                             None, 0, None)
        return st, lib.vq_last_error().decode()

    for kw, msg in ((dict(g=False), "null"), (dict(u=False), "null"), (dict(u=matrix(M=31)), "the same"), (dict(u=matrix(N=99)), "the same"),
                    (dict(u=matrix(ldq=192)), "the same"), (dict(T=-1), "T must"), (dict(dt=F32), "dtype"), (dict(act=-1), "activation"),
                    (dict(X=None), "null"), (dict(H=None), "null"), (dict(ldh=31), "leading dimension of H"), (dict(H=FAKE + 4096), "alias")):
        st, text = gated(**kw)
        assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_gated_i8"), kw


def test_workspaces():
    lib = vq.load()
    need = lib.vq_linear_i8_workspace_bytes(32, 100, 4)
    assert need >= 4 * 128 + 4 * 4
    assert linear(ws=FAKE + (1 << 20), n=need - 1)[0] == vq.VQ_ERR_WORKSPACE
    st, text = linear(ws=FAKE + (1 << 20) + 8, n=need)
    assert st == vq.VQ_ERR_INVALID and "16-byte" in text
    assert linear(T=0, X=None)[0] == vq.VQ_OK
    assert lib.vq_linear_i8_workspace_bytes(0, 100, 4) == lib.vq_gated_i8_workspace_bytes(32, 100, -1) == 0


def test_quantize_refuses():
    lib = vq.load()

    def quant(rows=4, cols=100, dt=F32, X=FAKE, ldx=100, q=FAKE + 8192, ldq=128, scale=FAKE + 16384):
        st = lib.vq_quantize_rows(rows, cols, dt, X, ldx, q, ldq, scale, None)
        return st, lib.vq_last_error().decode()

    for kw, msg in ((dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(cols=(1 << 20) + 1), "cols"), (dict(dt=3), "dtype"),
                    (dict(X=None), "null"), (dict(q=None), "null"), (dict(scale=None), "null"), (dict(ldx=99), "leading dimension"),
                    (dict(X=FAKE + 2), "aligned"), (dict(ldq=100), "multiple of 64"), (dict(ldq=64), "multiple of 64"),
                    (dict(q=FAKE + 8200), "16-byte"), (dict(scale=FAKE + 16386), "scale"), (dict(q=FAKE), "alias")):
        st, text = quant(**kw)
        assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_quantize_rows"), kw
    assert quant(rows=0, X=None)[0] == vq.VQ_OK


def test_python_checks():
    with pytest.raises(TypeError, match="int8 matrix"):
        vq.Int8Matrix(torch.zeros(4, 4), torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        vq.Int8Matrix(torch.zeros((4, 4), dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        vq.quantize_rows(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="matrix"):
        vq.quantize_rows(torch.zeros(4))
