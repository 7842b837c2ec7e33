"""The AdamW step against its formula in float64, and its 8-bit moments against their definition.

Tolerances count roundings, u = 2^-24 each: m takes two products, two rounded
constants and a sum, v one product more; the update a root, two products, a sum, a
quotient and a product; the parameter two products and a difference.
"""
import pytest
import torch

from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
KW = dict(lr=2e-3, betas=(0.9, 0.97), eps=1e-8, weight_decay=0.1)
B = 256


def f64(t):
    return t.detach().cpu().double()


def spread(s, n):
    """A scale for each 256 elements, for each element."""
    return torch.repeat_interleave(f64(s), B)[:n]


def moments(opt, i, n):
    m, v = opt.state["m"][i].reshape(-1), opt.state["v"][i].reshape(-1)
    if opt.state_bits == 32:
        return f64(m), f64(v)
    return (f64(m.float()) * spread(opt.state["m_scale"][i], n),
            (f64(v.float()) * spread(opt.state["v_scale"][i], n)).square())


def expected(p, g, m, v, t, gs=1.0):
    """(p, m, v) after step t and the bounds on a float32 kernel's errors of them, element by element."""
    b1, b2 = KW["betas"]
    g = g * gs
    am, av = (b1 * m).abs() + ((1 - b1) * g).abs(), b2 * v + (1 - b2) * g * g
    m2, v2 = b1 * m + (1 - b1) * g, av
    em, ev = 6 * U * am + 2.0 ** -148, 8 * U * av + 2.0 ** -147
    den = v2.sqrt() / (1 - b2 ** t) ** 0.5 + KW["eps"]
    rate = KW["lr"] / (1 - b1 ** t)
    upd = rate * m2 / den
    # the root's error from v's, where v is not subnormal: half of it relatively
    eu = 14 * U * upd.abs() + rate * em / den
    p2 = p * (1 - KW["lr"] * KW["weight_decay"]) - upd
    ep = eu + 3 * U * (p.abs() + upd.abs())
    return (p2, ep), (m2, em), (v2, ev)


def check_values(got, want, bound, what):
    bad = ((got - want).abs() > bound).nonzero()
    assert len(bad) == 0, "%s: element %d: %r against %r, bound %r" % (
        what, bad[0], float(got[bad[0]]), float(want[bad[0]]), float(bound[bad[0]]))


def check_codes(opt, i, m2, v2, em, ev):
    """8-bit moments: scales of the blocks' largest, codes within half a step, no root lost."""
    n = len(m2)
    for k, x, e, floor in (("m", m2, em, False), ("v", v2.sqrt(), 8 * U * v2.sqrt() + 2.0 ** -74, True)):
        scale = f64(opt.state[k + "_scale"][i])
        pad = torch.zeros(len(scale) * B, dtype=torch.float64)
        pad[:n] = x.abs()
        top = pad.view(-1, B).amax(1)
        slack = torch.zeros_like(pad)
        slack[:n] = e
        check_values(scale, top / 448, slack.view(-1, B).amax(1) / 448 + 2 * U * top / 448 + 2.0 ** -149, k + "_scale")
        code = f64(opt.state[k][i].float().reshape(-1))
        assert bool((code.abs() <= 448).all())
        s = spread(opt.state[k + "_scale"][i], n)
        half = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s)
        if floor:
            half = torch.maximum(half, 2.0 ** -9 * s)
            assert bool((code[(x > 0) & (s > 0)] > 0).all())
        check_values(code * s, x, half * (1 + 2.0 ** -10) + 2 * e, k)


def build(sizes, param, grad, master, bits, seed, offset=0, steps=3, **kw):
    """An optimizer over tensors of these sizes after some steps, and its gradients; offset elements into their buffers."""
    g = torch.Generator().manual_seed(seed)

    def cut(dtype, scale, square=False):
        out = []
        for n in sizes:
            x = scale * torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
            buf = torch.zeros(n + offset, dtype=dtype, device="cuda")
            buf[offset:] = (x.square() if square else x).to(dtype)
            out.append(buf[offset:])
        return out

    params, grads = cut(param, 0.05), cut(grad, 1e-2)
    masters = None
    if master:
        masters = cut(torch.float32, 0.05)
        for p, w in zip(params, masters):
            p.copy_(w)
    opt = vq.AdamW(params, grads, masters=masters, state_bits=bits, steps=steps, **KW, **kw)
    if steps:
        fill(opt, g)
    return opt


def fill(opt, g):
    """Moments as after some steps."""
    for i, p in enumerate(opt.params):
        n = p.numel()
        m = 5e-3 * torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
        r = 1e-2 * torch.randn(n, generator=g).abs() * torch.exp(torch.randn(n, generator=g))
        if opt.state_bits == 32:
            opt.state["m"][i].copy_(m)
            opt.state["v"][i].copy_(r.square())
            continue
        for k, x in (("m", m), ("v", r)):
            pad = torch.zeros(-(-n // B) * B)
            pad[:n] = x
            s = pad.view(-1, B).abs().amax(1) / 448
            opt.state[k + "_scale"][i].copy_(s)
            opt.state[k][i].copy_((x / torch.repeat_interleave(s, B)[:n]).clamp(-448, 448).to(torch.float8_e4m3fn))


def snapshot(opt):
    out = []
    for i, p in enumerate(opt.params):
        src = p if opt.masters is None else opt.masters[i]
        out.append((f64(src).reshape(-1), f64(opt.grads[i]).reshape(-1)) + moments(opt, i, p.numel()))
    return out


def check_step(opt, before, t, gs=1.0):
    for i, (p, g, m, v) in enumerate(before):
        (p2, ep), (m2, em), (v2, ev) = expected(p, g, m, v, t, gs)
        dt = opt.params[i].dtype
        stored = f64(opt.params[i]).reshape(-1)
        if opt.masters is not None:
            w = f64(opt.masters[i]).reshape(-1)
            check_values(w, p2, ep + U * p2.abs(), "master %d" % i)
            assert torch.equal(opt.masters[i].to(dt).reshape(-1), opt.params[i].reshape(-1))
        else:
            check_values(stored, p2, ep + UNIT[dt] * (p2.abs() + ep) + TINY[dt], "param %d" % i)
        if opt.state_bits == 32:
            got = moments(opt, i, len(p))
            check_values(got[0], m2, em, "m %d" % i)
            check_values(got[1], v2, ev, "v %d" % i)
        else:
            check_codes(opt, i, m2, v2, em, ev)


SIZES = [1, 2, 3, 5, 255, 256, 257, 1023, 4096, 4097, 12345]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [
    (torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False), (torch.float32, torch.float16, False),
    (torch.bfloat16, torch.bfloat16, True), (torch.bfloat16, torch.float32, True), (torch.bfloat16, torch.bfloat16, False),
    (torch.float16, torch.float16, True), (torch.float16, torch.float32, False), (torch.float16, torch.bfloat16, False)])
def test_types(param, grad, master, bits):
    opt = build(SIZES, param, grad, master, bits, 1)
    for k in range(3):
        before = snapshot(opt)
        opt.step()
        assert opt.steps == 4 + k
        check_step(opt, before, 4 + k)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 3])
def test_unaligned_views_and_neighbours(bits, offset):
    """Tensors that begin at odd elements; what lies around every buffer stays as it was."""
    opt = build([1, 7, 300, 4099], torch.bfloat16, torch.bfloat16, True, bits, 2, offset=offset)
    flat = {}
    for name in ("m", "v"):                                  # moments at odd elements too, guards between
        bufs = []
        for i, t in enumerate(opt.state[name]):
            kind = torch.float32 if bits == 32 else torch.uint8
            buf = torch.full((t.numel() + 9,), 77, dtype=kind, device="cuda")
            view = buf[offset:offset + t.numel()]
            view = view if bits == 32 else view.view(torch.float8_e4m3fn)
            view.copy_(t.reshape(-1))
            bufs.append((buf, view))
        flat[name] = [b for b, _ in bufs]
        opt.state[name] = [v for _, v in bufs]
    opt = vq.AdamW(opt.params, opt.grads, masters=opt.masters, state_bits=bits, state=opt.state, steps=3, **KW)
    before = snapshot(opt)
    opt.step()
    check_step(opt, before, 4)
    for name in ("m", "v"):
        for i, buf in enumerate(flat[name]):
            n = opt.params[i].numel()
            assert bool((buf[:offset] == 77).all()) and bool((buf[offset + n:] == 77).all())
    for ts in (opt.params, opt.masters, opt.grads):
        for t in ts:
            assert t._base is None or bool((t._base[:offset] == 0).all())


def test_first_step_and_scale():
    """From zero moments, with the gradients scaled by a number on the GPU."""
    for bits in (32, 8):
        opt = build([513, 40], torch.float32, torch.float32, False, bits, 3, steps=0)
        before = snapshot(opt)
        gs = torch.tensor([0.25], device="cuda")
        opt.step(grad_scale=gs)
        check_step(opt, before, 1, 0.25)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients(bits):
    """Zero gradients and moments: parameters only decay, and nothing is divided by zero."""
    opt = build([300], torch.float32, torch.float32, False, bits, 4, steps=0)
    opt.grads[0].zero_()
    p = f64(opt.params[0])
    for _ in range(3):
        opt.step()
    want = p * (1 - KW["lr"] * KW["weight_decay"]) ** 3
    check_values(f64(opt.params[0]), want, 6 * U * want.abs(), "param")
    assert not bool(opt.state["m"][0].float().any()) and not bool(opt.state["v"][0].float().any())


def test_small_roots_keep_the_step_bounded():
    """A root far below its block's largest is stored as the smallest code, so the next step stays of its size."""
    opt = build([256], torch.float32, torch.float32, False, 8, 5, steps=0)
    g = torch.full((256,), 1e-9, device="cuda")
    g[0] = 1e3
    opt.step([g])
    assert bool((opt.state["v"][0].float() > 0).all())
    before = opt.params[0].clone()
    opt.step([g])
    assert float((opt.params[0] - before).abs().max()) <= 2 * KW["lr"]


def test_non_finite_gradients_stay_in_their_element():
    opt = build([600], torch.float32, torch.float32, False, 32, 6)
    clean = build([600], torch.float32, torch.float32, False, 32, 6)
    opt.grads[0][7], opt.grads[0][300] = float("nan"), float("inf")
    opt.step()
    clean.step()
    for a, b in ((opt.params[0], clean.params[0]), (opt.state["m"][0], clean.state["m"][0])):
        same = a == b
        same[7] = same[300] = True
        assert bool(same.all()) and not bool(torch.isfinite(a[7]))
    # in 8 bits they stay in their block of 256
    opt = build([600], torch.float32, torch.float32, False, 8, 6)
    clean = build([600], torch.float32, torch.float32, False, 8, 6)
    opt.grads[0][7] = float("nan")
    opt.grads[0][300] = float("inf")
    opt.step()
    clean.step()
    assert bool(torch.isnan(opt.state["m"][0].float()[7]))
    same = opt.state["m"][0].float() == clean.state["m"][0].float()
    assert bool(same[512:].all()) and bool(same[:7].all()) and bool(same[8:256].all())


def test_many_tensors_in_one_call():
    g = torch.Generator().manual_seed(9)
    sizes = [int(n) for n in torch.randint(1, 3000, (700,), generator=g)] + [0, 1]
    opt = build(sizes, torch.bfloat16, torch.bfloat16, True, 8, 10)
    before = snapshot(opt)
    opt.step()
    check_step(opt, before, 4)


@pytest.mark.parametrize("captured", [False, True])
def test_new_gradients_every_step(captured):
    """Gradients in new tensors at each step, of more tensors than one launch carries; captured too."""
    sizes = [5 + i % 300 for i in range(1000)]
    opt = build(sizes, torch.float32, torch.bfloat16, False, 32, 20, capturable=captured)
    g = torch.Generator().manual_seed(21)
    for k in range(3):
        grads = [(1e-2 * torch.randn(n, generator=g)).bfloat16().cuda() for n in sizes]
        opt_grads = opt.grads
        opt.grads = grads                                    # what snapshot reads; step() is given them below
        before = snapshot(opt)
        opt.grads = opt_grads
        if captured:
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                opt.step(grads)
            graph.replay()
            torch.cuda.synchronize()
        else:
            opt.step(grads)
        check_step(opt, before, 4 + k)
    # of another type: the table is made anew
    if not captured:
        grads = [x.float() for x in grads]
        opt.step(grads)
        assert opt._plan.grad_dtype == 2


def capture(step):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    return graph


def signed(opt, f):
    """The sign of a fresh element's step in f(): its gradient's, with moments of nothing."""
    for k in ("m", "v"):
        opt.state[k][0].zero_()
    before = opt.params[0].clone()
    f()
    torch.cuda.synchronize()
    return torch.sign(before - opt.params[0]).tolist()


def test_eager_steps_beside_a_captured_one_with_its_own_gradients():
    """The graph's gradients are the graph's: before and after replays step() takes those given outside of it."""
    p = torch.zeros(2, device="cuda")
    opt = vq.AdamW([p], [torch.tensor([1.0, -1.0], device="cuda")], weight_decay=0.0, capturable=True)
    own = torch.tensor([-1.0, -1.0], device="cuda")
    graph = capture(lambda: opt.step([own]))
    assert signed(opt, opt.step) == [1, -1]
    for _ in range(3):
        assert signed(opt, graph.replay) == [-1, -1]
        assert signed(opt, opt.step) == [1, -1]
    opt.step([torch.tensor([1.0, 1.0], device="cuda")])
    assert signed(opt, graph.replay) == [-1, -1]
    assert signed(opt, opt.step) == [1, 1]


def test_captured_step_keeps_its_table():
    """Gradients of another type outside of the graph leave the table that it reads, and what that points to."""
    p = torch.zeros(2, device="cuda")
    opt = vq.AdamW([p], [torch.tensor([1.0, -1.0], device="cuda").bfloat16()], weight_decay=0.0, capturable=True)
    graph = capture(opt.step)
    for _ in range(3):
        assert signed(opt, lambda: opt.step([torch.tensor([-1.0, 1.0], device="cuda")])) == [-1, 1]
        # memory that a freed table or gradient would have left
        junk = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in (16, 512, 1024, 2048) for _ in range(8)]
        assert signed(opt, graph.replay) == [1, -1]
        del junk


def test_first_gradients_in_a_capture_are_refused():
    opt = vq.AdamW([torch.zeros(2, device="cuda")], capturable=True)
    x = torch.zeros(1, device="cuda")
    g = torch.ones(2, device="cuda")

    def step():
        x.add_(1.0)
        with pytest.raises(ValueError, match="outside of a capture"):
            opt.step([g])

    capture(step).replay()
    torch.cuda.synchronize()
    assert float(x) == 1.0 and int(opt.steps) == 0
    opt.step([g])
    assert int(opt.steps) == 1


def test_capture_without_capturable_is_refused():
    p, x = torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda")
    opt = vq.AdamW([p], [torch.ones(2, device="cuda")])

    def step():
        x.add_(1.0)
        with pytest.raises(ValueError, match="capturable"):
            opt.step()

    capture(step).replay()
    torch.cuda.synchronize()
    assert float(x) == 1.0 and opt.steps == 0 and not bool(p.any())


def test_large_tensor():
    """Past 2^24 elements: chunks and blocks keep their places."""
    n = (1 << 25) + 77
    opt = vq.AdamW([torch.zeros(n, device="cuda")], lr=1e-2, weight_decay=0.0, state_bits=8)
    g = torch.zeros(n, device="cuda")
    g[n - 1], g[1 << 24] = 1.0, -1.0
    opt.step([g])
    at = opt.params[0].nonzero()[:, 0].tolist()
    assert at == [1 << 24, n - 1]
    assert abs(float(opt.params[0][n - 1]) + 1e-2) < 1e-7 and abs(float(opt.params[0][1 << 24]) - 1e-2) < 1e-7
    assert float(opt.state["m_scale"][0][-1]) == pytest.approx(0.1 / 448, rel=1e-6)


def test_same_bits_every_time_and_on_another_stream():
    ref = build(SIZES, torch.bfloat16, torch.bfloat16, True, 8, 11)
    ref.step()
    for other in (False, True):
        opt = build(SIZES, torch.bfloat16, torch.bfloat16, True, 8, 11)
        st = torch.cuda.Stream() if other else torch.cuda.current_stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            opt.step()
        st.synchronize()
        for a, b in zip(ref.masters + ref.params, opt.masters + opt.params):
            assert torch.equal(a, b)
        for k in ("m", "v"):
            for a, b in zip(ref.state[k], opt.state[k]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_count(bits):
    """Replays of a captured step are consecutive steps, with eager work between, and follow lr."""
    plain = build([300, 5000], torch.float32, torch.float32, False, bits, 12, steps=2)
    opt = build([300, 5000], torch.float32, torch.float32, False, bits, 12, steps=2, capturable=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        opt.step()
    for k in range(4):
        lr = KW["lr"] * (1 + k)
        opt.lr.fill_(lr)
        # float32 holds the GPU's learning rate: give the eager side the same number
        plain.lr = float(opt.lr)
        for a, b in zip(plain.grads, opt.grads):
            a.mul_(0.9)
            b.mul_(0.9)
        plain.step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(opt.steps) == plain.steps == 3 + k
        for a, b in zip(plain.params, opt.params):
            # the two powers of beta may differ by their last bits in double: a coefficient by one ulp
            assert torch.allclose(a, b, rtol=2.0 ** -21, atol=2.0 ** -20 * lr)


def test_refusals_on_the_gpu():
    p = torch.zeros(16, device="cuda")
    with pytest.raises(vq.VQError, match="overlap"):
        vq.AdamW([p, p], [torch.zeros(16, device="cuda")] * 2)
    with pytest.raises(ValueError, match="elements"):
        vq.AdamW([p], [torch.zeros(15, device="cuda")])
    with pytest.raises(ValueError, match="contiguous"):
        vq.AdamW([torch.zeros((4, 8), device="cuda")[:, :4]])
    with pytest.raises(TypeError, match="masters"):
        vq.AdamW([p.half()], masters=[p.half()])
    with pytest.raises(ValueError, match="no masters"):
        vq.AdamW([p], masters=[p.clone()])
    with pytest.raises(ValueError, match="grads are needed"):
        vq.AdamW([p]).step()
    with pytest.raises(ValueError, match="grad_scale"):
        vq.AdamW([p], [p.clone()]).step(grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="GPU"):
        vq.AdamW([p], [torch.zeros(16)])


def test_value_check(monkeypatch):
    opt = build([300, 9000], torch.bfloat16, torch.float32, True, 8, 13)
    monkeypatch.setenv("VQ_CHECK", "1")
    opt.step()
    opt.grads[1][8999] = float("nan")
    with pytest.raises(vq.VQError, match="gradient"):
        opt.step()
