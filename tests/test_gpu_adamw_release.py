"""The gradients of captured steps are the optimizer's until it is told that their graphs are gone."""
import gc
import weakref

import pytest
import torch

from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu


def capture(step):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    return graph


def moved(opt, f):
    """The signs of a step from moments of nothing."""
    for k in ("m", "v"):
        opt.state[k][0].zero_()
    before = opt.params[0].clone()
    f()
    torch.cuda.synchronize()
    return torch.sign(before - opt.params[0]).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_release(dtype):
    """Captured gradients of the eager ones' type and of another."""
    opt = vq.AdamW([torch.zeros(2, device="cuda")], [torch.tensor([1.0, -1.0], dtype=dtype, device="cuda")], weight_decay=0.0,
                   capturable=True)
    opt.step([torch.tensor([1.0, -1.0], device="cuda")])      # the table of float32 gradients
    kept = []
    for _ in range(3):
        own = torch.tensor([-1.0, 1.0], dtype=dtype, device="cuda")
        graph = capture(lambda: opt.step([own]))
        kept.append(weakref.ref(own))
        del own
        gc.collect()
        assert moved(opt, graph.replay) == [-1, 1]
        assert moved(opt, opt.step) == [1, -1]
        assert moved(opt, graph.replay) == [-1, 1]
    assert len(opt._captured) >= 3 and all(r() is not None for r in kept)
    del graph
    opt.release()
    gc.collect()
    assert all(r() is None for r in kept)
    junk = [torch.full((2,), -1.0, device="cuda") for _ in range(64)]        # where they were
    for _ in range(2):
        assert moved(opt, opt.step) == [1, -1]
    opt.release()
    assert moved(opt, opt.step) == [1, -1] and len(junk) == 64
    graph = capture(opt.step)                                 # of the last gradients, none of its own
    assert opt._captured == []
    for _ in range(2):
        assert moved(opt, graph.replay) == [1, -1]
        assert moved(opt, opt.step) == [1, -1]


def test_release_in_a_capture_is_refused():
    opt = vq.AdamW([torch.zeros(2, device="cuda")], [torch.ones(2, device="cuda")], capturable=True)
    x = torch.zeros(1, device="cuda")

    def step():
        x.add_(1.0)
        with pytest.raises(ValueError, match="outside of a capture"):
            opt.release()

    capture(step).replay()
    torch.cuda.synchronize()
    assert float(x) == 1.0
    opt.release()
    opt.step()


def test_a_graph_that_stays_takes_the_gradients_of_its_type():
    """Released beside a graph without gradients of its own, of another type than the last eager ones."""
    opt = vq.AdamW([torch.zeros(2, device="cuda")], [torch.tensor([1.0, -1.0], device="cuda")], weight_decay=0.0, capturable=True)
    stays = capture(opt.step)
    own = torch.tensor([-1.0, 1.0], device="cuda")
    goes = capture(lambda: opt.step([own]))
    assert moved(opt, goes.replay) == [-1, 1] and moved(opt, stays.replay) == [-1, 1]
    assert moved(opt, lambda: opt.step([torch.tensor([1.0, 1.0], device="cuda").bfloat16()])) == [1, 1]
    del goes, own
    opt.release()
    gc.collect()
    junk = [torch.full((2,), -1.0, device="cuda") for _ in range(64)]
    for _ in range(2):
        assert moved(opt, stays.replay) == [1, -1]
        assert moved(opt, opt.step) == [1, 1]
    assert len(junk) == 64
