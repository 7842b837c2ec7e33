"""Refusals of the AdamW calls without a GPU: every case fails validation on the host."""
import ctypes

import pytest
import torch

from hessian_weighted_vector_amd import vq

FAKE = 0x100000            # never dereferenced
BF16, F16, F32 = 0, 1, 2


def tensor(i=0, **change):
    at = FAKE + i * 0x10000
    f = dict(param=at, grad=at + 0x1000, master=at + 0x2000, m=at + 0x4000, v=at + 0x6000, m_scale=at + 0x8000,
             v_scale=at + 0x9000, n=500)
    f.update(change)
    return vq.AdamWTensor(*[f[k] for k, _ in vq.AdamWTensor._fields_])


def plan(tensors, count=None, param=BF16, grad=BF16, master=1, bits=8, table=None, size=0):
    lib = vq.load()
    rows = (vq.AdamWTensor * max(1, len(tensors)))(*tensors)
    out = vq.AdamWPlan()
    st = lib.vq_adamw_plan(rows, len(tensors) if count is None else count, param, grad, master, bits, table, size,
                           ctypes.addressof(out), None)
    return st, lib.vq_last_error().decode()


@pytest.mark.parametrize("kw,msg", [
    (dict(count=-1), "count"), (dict(param=3), "dtype"), (dict(grad=-1), "dtype"), (dict(bits=16), "state_bits"),
    (dict(param=F32, master=1), "no master"),
])
def test_plan_refuses_arguments(kw, msg):
    st, text = plan([tensor()], **kw)
    assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_adamw_plan")


@pytest.mark.parametrize("change,msg", [
    (dict(n=-1), "n must"), (dict(n=(1 << 40) + 1), "n must"), (dict(param=None), "null"), (dict(grad=None), "null"),
    (dict(m=None), "null"), (dict(v=None), "null"), (dict(master=None), "master"), (dict(m_scale=None), "m_scale"),
    (dict(v_scale=None), "m_scale"), (dict(param=FAKE + 1), "aligned"), (dict(grad=FAKE + 0x1001), "aligned"),
    (dict(master=FAKE + 0x2002), "aligned"), (dict(m_scale=FAKE + 0x8002), "aligned"),
])
def test_plan_refuses_tensors(change, msg):
    st, text = plan([tensor(0), tensor(1, **change)])
    assert st == vq.VQ_ERR_INVALID and msg in text and "tensor 1" in text


def test_plan_refuses_overlaps():
    # the same tensor twice, a moment inside a parameter, a parameter inside a gradient
    for other in (tensor(0), tensor(1, v=FAKE + 2 * 499), tensor(1, param=FAKE + 0x1000 + 998)):
        st, text = plan([tensor(0), other])
        assert st == vq.VQ_ERR_INVALID and "overlap" in text
    # gradients may overlap each other: refused only for the missing table
    st, text = plan([tensor(0), tensor(1, grad=FAKE + 0x1000)])
    assert st == vq.VQ_ERR_WORKSPACE and "table" in text
    # neighbours touch without overlapping
    st, _ = plan([tensor(0, n=256), tensor(1, param=FAKE + 512, n=256)])
    assert st == vq.VQ_ERR_WORKSPACE


def test_plan_refuses_too_many_elements():
    st, text = plan([tensor(0, n=1 << 36)])
    assert st == vq.VQ_ERR_INVALID and "chunks" in text


def test_plan_sizes():
    lib = vq.load()

    def need(*ns):
        rows = (vq.AdamWTensor * len(ns))(*[tensor(i, n=n) for i, n in enumerate(ns)])
        return lib.vq_adamw_plan_bytes(rows, len(ns))

    assert need(4096) == need(1) and need(1 << 20) > need(4096)
    assert lib.vq_adamw_plan_bytes(None, 1) == 0
    assert need(-1) == 0
    size = need(500)
    st, text = plan([tensor()], table=FAKE, size=size - 1)
    assert st == vq.VQ_ERR_WORKSPACE
    st, text = plan([tensor()], table=FAKE + 8, size=size)
    assert st == vq.VQ_ERR_INVALID and "aligned" in text
    # nothing to do: no table is needed
    assert plan([tensor(n=0)])[0] == vq.VQ_OK
    assert plan([], count=0)[0] == vq.VQ_OK


def test_step_refuses():
    lib = vq.load()
    good = vq.AdamWPlan(FAKE, 1, 1, BF16, BF16, 0, 32)

    def step(p=good, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, t=1, step_from=None, lr_from=None, scale=None):
        st = lib.vq_adamw(ctypes.addressof(p) if p else None, lr, b1, b2, eps, wd, t, step_from, lr_from, scale, None)
        return st, lib.vq_last_error().decode()

    nan = float("nan")
    for kw, msg in ((dict(p=None), "null"), (dict(lr=nan), "lr"), (dict(lr=float("inf")), "lr"), (dict(b1=1.0), "betas"),
                    (dict(b2=-0.1), "betas"), (dict(b1=nan), "betas"), (dict(eps=-1.0), "eps"), (dict(wd=nan), "eps"),
                    (dict(t=0), "step"), (dict(lr_from=FAKE), "lr_from"), (dict(scale=FAKE + 2), "aligned"),
                    (dict(step_from=FAKE + 4), "aligned"), (dict(p=vq.AdamWPlan(None, 1, 1, BF16, BF16, 0, 32)), "not made"),
                    (dict(p=vq.AdamWPlan(FAKE, 1, 1, 9, BF16, 0, 32)), "not made"),
                    (dict(p=vq.AdamWPlan(FAKE, 1, 1, BF16, BF16, 0, 16)), "not made"),
                    (dict(p=vq.AdamWPlan(None, 0, 0, BF16, BF16, 0, 32), step_from=FAKE), "elements")):
        st, text = step(**kw)
        assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_adamw:"), kw
    assert step(p=vq.AdamWPlan(None, 0, 0, BF16, BF16, 0, 32))[0] == vq.VQ_OK


def test_new_gradients_refuse():
    lib = vq.load()
    good = vq.AdamWPlan(FAKE, 2, 2, BF16, F32, 0, 32)

    def grads(ptrs, p=good, count=None):
        arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs) if ptrs is not None else None
        st = lib.vq_adamw_grads(ctypes.addressof(p) if p else None, arr, len(ptrs) if count is None else count, None)
        return st, lib.vq_last_error().decode()

    for args, msg in ((([FAKE, FAKE], None), "null"), (([FAKE],), "count"), (([FAKE, FAKE + 2],), "gradient 1"),
                      ((None, good, 2), "null"), (([FAKE, FAKE], vq.AdamWPlan(None, 2, 2, BF16, F32, 0, 32)), "not made"),
                      (([FAKE, FAKE], vq.AdamWPlan(FAKE, 2, 2, BF16, 7, 0, 32)), "not made")):
        st, text = grads(*args)
        assert st == vq.VQ_ERR_INVALID and msg in text and text.startswith("vq_adamw_grads"), args
    assert grads([], vq.AdamWPlan(None, 0, 0, BF16, F32, 0, 32))[0] == vq.VQ_OK


def test_python_checks():
    p = torch.zeros(8)
    with pytest.raises(ValueError, match="empty"):
        vq.AdamW([])
    with pytest.raises(ValueError, match="state_bits"):
        vq.AdamW([p], state_bits=4)
    with pytest.raises(ValueError, match="GPU"):
        vq.AdamW([p])
