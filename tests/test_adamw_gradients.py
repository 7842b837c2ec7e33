"""New gradients of a plan: null ones and those that overlap what a step writes are refused, as by the plan itself."""
import ctypes

import pytest
import torch

from hessian_weighted_vector_amd import vq

FAKE = 0x100000            # never dereferenced
F32 = 2


def new(plan, pointers):
    lib = vq.load()
    arr = (ctypes.c_void_p * len(pointers))(*pointers)
    return lib.vq_adamw_grads(ctypes.addressof(plan), arr, len(pointers), None), lib.vq_last_error().decode()


def test_a_plan_that_was_not_made():
    """Without the sizes nothing can be said of a gradient: refused before the GPU is asked."""
    for pointers in ([FAKE, None], [FAKE, FAKE + 64]):
        st, text = new(vq.AdamWPlan(FAKE, 2, 2, F32, F32, 0, 32), pointers)
        assert st == vq.VQ_ERR_INVALID and "not made" in text and text.startswith("vq_adamw_grads")


def test_free_of_nothing():
    lib = vq.load()
    lib.vq_adamw_plan_free(None)
    plan = vq.AdamWPlan()
    lib.vq_adamw_plan_free(ctypes.addressof(plan))
    assert plan.known is None


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_refusals(bits):
    n = 600
    params = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(3)] + [torch.zeros(0, dtype=torch.bfloat16, device="cuda")]
    masters = [torch.zeros(p.numel(), device="cuda") for p in params]
    buf = torch.ones(4 * n, device="cuda")
    good = [buf[:n], buf[n:2 * n], buf[n // 2:n // 2 + n], buf[:0]]          # may overlap each other
    opt = vq.AdamW(params, good, masters=masters, state_bits=bits, weight_decay=0.0, lr=1.0)
    good_at = [g.data_ptr() for g in good[:3]] + [None]
    assert new(opt._plan, good_at)[0] == vq.VQ_OK
    st, text = new(opt._plan, [good_at[0], None, good_at[2], None])
    assert st == vq.VQ_ERR_INVALID and "gradient 1 is null" in text
    # all that a step writes: its first and its last byte
    state = [masters[1]] + [ts[1] for ts in opt.state.values() if ts is not None] + [params[1]]
    for t in state:
        begin, end = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        for at in (begin - 4 * n + 4, begin, (end - 1) // 4 * 4):
            st, text = new(opt._plan, [good_at[0], good_at[1], at, None])
            assert st == vq.VQ_ERR_INVALID and "gradient 2 overlaps" in text
    with pytest.raises(vq.VQError, match="overlaps"):
        opt.step([masters[0]] + good[1:])
    assert opt.steps == 0 and opt.grads[0].data_ptr() == buf.data_ptr()
    opt.step()                                                # with the gradients from before
    assert opt.steps == 1 and all(bool((w < -0.9).all()) for w in masters[:3])
    # neighbours touch without overlapping
    whole = torch.zeros(3 * n, device="cuda")
    opt = vq.AdamW([whole[n:2 * n]], [whole[:n]], state_bits=bits)
    opt.step([whole[2 * n:]])
    opt.step([whole[:n]])


@pytest.mark.gpu
def test_a_freed_plan_takes_no_gradients():
    opt = vq.AdamW([torch.zeros(8, device="cuda")], [torch.ones(8, device="cuda")], weight_decay=0.0, lr=1.0)
    lib = vq.load()
    for _ in range(2):
        lib.vq_adamw_plan_free(opt._ref)
    st, text = new(opt._plan, [opt.grads[0].data_ptr()])
    assert st == vq.VQ_ERR_INVALID and "freed" in text
    opt.step()                                                # the table is still there
    assert bool((opt.params[0] < -0.9).all())


def test_release_on_another_gpu(monkeypatch):
    """Like step(), refused before anything is launched."""
    opt = object.__new__(vq.AdamW)
    opt.params, opt.index, opt._captured, opt.grads = [torch.zeros(2)], 1, [[torch.zeros(2)]], [torch.zeros(2)]
    monkeypatch.setattr(vq, "_device", lambda: 0)
    monkeypatch.setattr(opt, "_bind", lambda grads: pytest.fail("launched"), raising=False)
    with pytest.raises(ValueError, match="GPU"):
        opt.release()
    assert len(opt._captured) == 1


def test_release_puts_back_the_gradients_of_every_type(monkeypatch):
    """A graph of one type's table may replay when gradients of another type were the last ones."""
    put = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name == "vq_adamw_grads":
                    put.append((args[0], list(args[1])))
                return 0
            return call

    capturing = [False]
    monkeypatch.setattr(vq, "load", Library)
    monkeypatch.setattr(vq, "_home", lambda X, name="X": -1)
    monkeypatch.setattr(vq, "_device", lambda: -1)
    monkeypatch.setattr(vq, "_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    wide, half, own = (torch.zeros(300, dtype=t) for t in (torch.float32, torch.bfloat16, torch.float32))
    opt = vq.AdamW([torch.zeros(300)], [wide], capturable=True)
    plan_wide = opt._ref
    opt.step([half])
    plan_half = opt._ref
    capturing[0] = True
    opt.step([own])
    capturing[0] = False
    assert put == [(plan_wide, [own.data_ptr()])]
    del put[:]
    opt.release()
    assert (plan_wide, [wide.data_ptr()]) in put and put[-1] == (plan_half, [half.data_ptr()])
    assert opt._captured == [] and opt._ref == plan_half
    del put[:]
    opt.step()
    opt.release()
    assert put == []
