"""The dense feed-forward calls against float64 (GPU): linear, gated, and their backward passes.

Every output element is held to the bound of ffn_reference, which follows from
the stated arithmetic.  The cases cover one token to several tiles, sizes that
are odd, aligned, below one tile and ragged past it, strided and misaligned
rows, every activation, biases and residuals, in-place residuals, empty
batches, values kept for the backward pass, and non-finite inputs.
"""
import sys

import pytest
import torch

import ffn_reference as ref
from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def tensor(g, shape, dtype, scale=1.0, layout="plain"):
    """A seeded GPU tensor; layout: plain, pitched (aligned longer rows), odd (odd
    row stride and an address one element off)."""
    v = (scale * torch.randn(shape, generator=g, dtype=torch.float64)).to(dtype)
    if layout == "plain" or len(shape) == 1:
        return v.cuda()
    r, c = shape
    ld = (c + 7) // 8 * 8 + 16 if layout == "pitched" else (c | 1) + 2
    off = 0 if layout == "pitched" else 1
    buf = torch.full((r * ld + off + 8,), float("nan"), dtype=dtype, device="cuda")
    view = buf[off:off + r * ld].view(r, ld)[:, :c]
    view.copy_(v)
    return view


def check(name, got, want):
    for k, (t, (value, bound)) in enumerate(zip(got, want)):
        t = ref.f64(t)
        assert t.shape == value.shape, (name, k)
        ratio = (t - value).abs() / bound
        worst = float(ratio.max()) if ratio.numel() else 0.0
        say("   %s[%d] max error / bound = %.3g" % (name, k, worst))
        assert worst <= 1.0, (name, k, worst)


# (T, M, N): one token; below a tile; odd; ragged past one 128 and one 256 tile; long k
SIZES = [(1, 1, 1), (1, 64, 64), (2, 40, 8), (3, 129, 72), (7, 33, 517), (16, 256, 256), (17, 100, 1000),
         (33, 260, 136), (65, 515, 200), (130, 384, 1024), (257, 300, 96), (300, 1030, 264), (5, 4104, 320),
         (64, 96, 8200)]
LAYOUTS = ["plain", "pitched", "odd"]


@pytest.mark.parametrize("size", SIZES, ids=["%dx%dx%d" % s for s in SIZES])
@pytest.mark.parametrize("dt", DT)
def test_linear(size, dt):
    T, M, N = size
    dtype = DT[dt]
    for k, layout in enumerate(LAYOUTS):
        name = ref.ACTS[(T + M + N + k) % len(ref.ACTS)]
        say("linear", size, dt, layout, name)
        g = torch.Generator().manual_seed(1000 * T + M + N + k)
        X = tensor(g, (T, N), dtype, 1.0, layout)
        W = tensor(g, (M, N), dtype, 1.0 / N ** 0.5, layout)
        b = tensor(g, (M,), dtype) if k != 1 else None
        R = tensor(g, (T, M), dtype, 1.0, layout) if k != 2 else None
        Y, Z = vq.linear(X, W, bias=b, residual=R, act=name, want_pre=True)
        want = ref.linear(X, W, b, R, name, dtype)
        check("linear", [Y, Z], want)
        # without the kept values, into a strided output
        out = tensor(g, (T, M), dtype, 1.0, layout)
        Y2 = vq.linear(X, W, bias=b, residual=R, act=name, out=out)
        assert Y2 is out
        check("linear out", [Y2], want)


@pytest.mark.parametrize("size", SIZES, ids=["%dx%dx%d" % s for s in SIZES])
@pytest.mark.parametrize("dt", DT)
def test_gated(size, dt):
    T, M, N = size
    dtype = DT[dt]
    for k, layout in enumerate(LAYOUTS):
        name = ref.ACTS[(T + M + N + k) % len(ref.ACTS)]
        say("gated", size, dt, layout, name)
        g = torch.Generator().manual_seed(2000 * T + M + N + k)
        X = tensor(g, (T, N), dtype, 1.0, layout)
        Wg = tensor(g, (M, N), dtype, 1.0 / N ** 0.5, layout)
        Wu = tensor(g, (M, N), dtype, 1.0 / N ** 0.5, layout)
        bg = tensor(g, (M,), dtype) if k != 1 else None
        bu = tensor(g, (M,), dtype) if k == 0 else None
        got = vq.gated(X, Wg, Wu, bias_gate=bg, bias_up=bu, act=name, want_pre=True)
        want = ref.gated(X, Wg, Wu, bg, bu, name, dtype)
        check("gated", got, want)
        out = tensor(g, (T, M), dtype, 1.0, layout)
        check("gated out", [vq.gated(X, Wg, Wu, bias_gate=bg, bias_up=bu, act=name, out=out)], want)


@pytest.mark.parametrize("size", SIZES, ids=["%dx%dx%d" % s for s in SIZES])
@pytest.mark.parametrize("dt", DT)
def test_linear_backward(size, dt):
    T, M, N = size
    dtype = DT[dt]
    for k, layout in enumerate(LAYOUTS):
        name = ref.ACTS[(T + M + N + k) % len(ref.ACTS)]
        say("linear_backward", size, dt, layout, name)
        g = torch.Generator().manual_seed(3000 * T + M + N + k)
        X = tensor(g, (T, N), dtype, 1.0, layout)
        W = tensor(g, (M, N), dtype, 1.0 / N ** 0.5, layout)
        Z = tensor(g, (T, M), dtype, 1.5, layout)
        dY = tensor(g, (T, M), dtype, 1.0, layout)
        want = ref.linear_backward(dY, X, W, Z, name, dtype)
        pre = None if name == "none" else Z
        check("linear_backward", vq.linear_backward(dY, X, W, pre=pre, act=name, want_db=True), want)
        dX, dW, db = vq.linear_backward(dY, X, W, pre=pre, act=name, want_dw=False)
        assert dW is None and db is None
        check("dX alone", [dX], want[:1])
        dX, dW, db = vq.linear_backward(dY, X, W, pre=pre, act=name, want_dx=False, want_dw=False, want_db=True)
        assert dX is None and dW is None
        check("db alone", [db], want[2:])


@pytest.mark.parametrize("size", SIZES, ids=["%dx%dx%d" % s for s in SIZES])
@pytest.mark.parametrize("dt", DT)
def test_gated_backward(size, dt):
    T, M, N = size
    dtype = DT[dt]
    for k, layout in enumerate(LAYOUTS):
        name = ref.ACTS[(T + M + N + k) % len(ref.ACTS)]
        say("gated_backward", size, dt, layout, name)
        g = torch.Generator().manual_seed(4000 * T + M + N + k)
        X = tensor(g, (T, N), dtype, 1.0, layout)
        Wg = tensor(g, (M, N), dtype, 1.0 / N ** 0.5, layout)
        Wu = tensor(g, (M, N), dtype, 1.0 / N ** 0.5, layout)
        G = tensor(g, (T, M), dtype, 1.5, layout)
        U = tensor(g, (T, M), dtype, 1.5, layout)
        dH = tensor(g, (T, M), dtype, 1.0, layout)
        want = ref.gated_backward(dH, X, Wg, Wu, G, U, name, dtype)
        check("gated_backward", vq.gated_backward(dH, X, Wg, Wu, G, U, act=name, want_db=True), want)
        r = vq.gated_backward(dH, X, Wg, Wu, G, U, act=name, want_dx=False)
        assert r[0] is None and r[3] is None and r[4] is None
        check("dW alone", r[1:3], want[1:3])


def test_split_sums_and_many_tiles():
    """Few output tiles under a long sum (split over workgroups), and more tiles than one round of the chip."""
    for (T, M, N) in [(48, 200, 16384), (700, 1300, 640), (1030, 2056, 264)]:
        for dt in DT:
            dtype = DT[dt]
            say("split/many", (T, M, N), dt)
            g = torch.Generator().manual_seed(T)
            X = tensor(g, (T, N), dtype)
            Wg, Wu = (tensor(g, (M, N), dtype, N ** -0.5) for _ in range(2))
            dY = tensor(g, (T, M), dtype)
            check("linear", [vq.linear(X, Wg, act="silu")], ref.linear(X, Wg, None, None, "silu", dtype))
            H, G, U = vq.gated(X, Wg, Wu, want_pre=True)
            check("gated", [H, G, U], ref.gated(X, Wg, Wu, None, None, "silu", dtype))
            check("gated_backward", vq.gated_backward(dY, X, Wg, Wu, G, U), ref.gated_backward(
                dY, X, Wg, Wu, G, U, "silu", dtype)[:3])
            check("linear_backward", vq.linear_backward(dY, X, Wg)[:2],
                  ref.linear_backward(dY, X, Wg, None, "none", dtype)[:2])


def test_few_tokens_of_a_large_matrix():
    """Enough weights for the tiled product to be taken for few tokens; unaligned rows keep the other."""
    say("few tokens, large matrix")
    g = torch.Generator().manual_seed(21)
    X = tensor(g, (20, 4096), torch.bfloat16)
    W = [tensor(g, (8192, 4096), torch.bfloat16, 0.02) for _ in range(2)]
    for Wg, Wu in (W, [torch.cat([w, w[:, :1]], 1)[:, :4096] for w in W]):
        check("linear", (vq.linear(X, Wg, act="silu"),), ref.linear(X, Wg, None, None, "silu", torch.bfloat16)[:1])
        check("gated", (vq.gated(X, Wg, Wu),), ref.gated(X, Wg, Wu, None, None, "silu", torch.bfloat16)[:1])


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: first and last rows, and gradients over all of them."""
    say("large offsets")
    T, M, N = 270000, 8192, 64
    g = torch.Generator(device="cuda").manual_seed(22)
    X = torch.randn((T, N), generator=g, device="cuda").bfloat16()
    W = (0.1 * torch.randn((M, N), generator=g, device="cuda")).bfloat16()
    Y, Z = vq.linear(X, W, act="relu", want_pre=True)
    rows = torch.tensor([0, 1, 262143, 262144, T - 2, T - 1])
    check("rows", (Y[rows], Z[rows]), ref.linear(X[rows], W, None, None, "relu", torch.bfloat16))
    # dY is zero but in those rows: the gradients are theirs alone
    Y.zero_()
    Y[rows] = torch.randn((len(rows), M), generator=g, device="cuda").bfloat16()
    dX, dW, _ = vq.linear_backward(Y, X, W, Z, "relu")
    want = ref.linear_backward(Y[rows], X[rows], W, Z[rows], "relu", torch.bfloat16)
    check("dX", (dX[rows],), want[:1])
    check("dW", (dW,), want[1:2])
    assert int((dX != 0).any(1).sum()) == len(rows)


def test_residual_in_place_and_reproducible():
    say("in place")
    g = torch.Generator().manual_seed(5)
    X, W, R = (tensor(g, s, torch.bfloat16) for s in ((20, 192), (264, 192), (20, 264)))
    want = ref.linear(X, W, None, R, "gelu", torch.bfloat16)
    a = vq.linear(X, W, residual=R, act="gelu")
    b = vq.linear(X, W, residual=R, act="gelu")
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    Y = vq.linear(X, W, residual=R, act="gelu", out=R)
    assert Y is R
    check("in place", [Y], want[:1])
    assert torch.equal(a.view(torch.int16), Y.view(torch.int16))


def test_no_tokens():
    say("T = 0")
    for dtype in DT.values():
        X = torch.empty((0, 24), dtype=dtype, device="cuda")
        W = torch.randn((40, 24), device="cuda").to(dtype)
        Y, Z = vq.linear(X, W, want_pre=True)
        assert Y.shape == Z.shape == (0, 40)
        assert vq.gated(X, W, W.clone()).shape == (0, 40)
        E = torch.empty((0, 40), dtype=dtype, device="cuda")
        dX, dW, db = vq.linear_backward(E, X, W, pre=E, act="silu", want_db=True)
        assert dX.shape == (0, 24) and not dW.any() and not db.any()
        r = vq.gated_backward(E, X, W, W.clone(), E, E, want_db=True)
        assert r[0].shape == (0, 24) and not any(t.any() for t in r[1:])


def test_non_finite_values_stay_in_their_rows():
    """An infinite or NaN input reaches the outputs whose sums it enters, no others (zero padding included)."""
    for (T, M, N) in [(5, 70, 100), (40, 300, 136)]:
        say("non-finite", (T, M, N))
        g = torch.Generator().manual_seed(9)
        X, W = tensor(g, (T, N), torch.bfloat16), tensor(g, (M, N), torch.bfloat16)
        clean = vq.linear(X, W)
        X[2, N - 1] = float("nan")
        W[M - 1, 0] = float("inf")
        Y = vq.linear(X, W)
        bad = torch.zeros((T, M), dtype=torch.bool, device="cuda")
        bad[2] = True
        bad[:, M - 1] = True
        assert bool((~torch.isfinite(Y) == bad).all())
        assert torch.equal(Y[~bad].view(torch.int16), clean[~bad].view(torch.int16))


def test_large_activations_saturate():
    """Pre-activations far outside the exponential's range: limits, not NaN."""
    z = torch.tensor([-3e38, -1e30, -1e4, -200.0, -90.0, -0.0, 0.0, 90.0, 200.0, 1e4, 1e30, 3e38])
    X = torch.eye(len(z), dtype=torch.bfloat16, device="cuda")
    W = z.to(torch.bfloat16).cuda()[None, :].contiguous()
    zz = ref.f64(W)[0]
    for name in ref.ACTS:
        Y = ref.f64(vq.linear(X, W, act=name))[:, 0]
        want = torch.where(zz > 50, {"sigmoid": torch.ones_like(zz)}.get(name, zz), torch.zeros_like(zz))
        if name == "none":
            want = zz
        if name == "sigmoid":
            want = torch.where(zz == 0, 0.5 * torch.ones_like(zz), want)
        assert torch.allclose(Y, want, rtol=2.0 ** -8, atol=1e-36), (name, Y)
        n = len(z)
        one = torch.ones((n, 1), dtype=torch.bfloat16, device="cuda")
        pre = W.reshape(n, 1).contiguous()
        dX, dW, db = vq.linear_backward(one, X, W, pre=pre, act=name, want_dx=False)
        d = ref.f64(dW)[0]
        assert bool(torch.isfinite(d).all()), (name, d)
        lim = ref.act_grad(name, zz.clamp(-60, 60)) if name != "none" else torch.ones_like(zz)
        assert torch.allclose(d, lim, rtol=2.0 ** -7, atol=1e-20), (name, d)


def test_gradients_against_differences():
    """Directional derivatives of sum(dY * forward) along random directions: central
    differences of the float64 forward against the kernels' gradients.  The
    difference quotient's own error (step 1e-5) is far below the gradients' bound."""
    g = torch.Generator().manual_seed(11)
    T, M, N = 9, 24, 40
    dtype = torch.float16
    for name in ref.ACTS:
        if name == "relu":
            continue               # not differentiable where the step crosses zero
        say("differences", name)
        X, Wg, Wu = tensor(g, (T, N), dtype), tensor(g, (M, N), dtype, 0.2), tensor(g, (M, N), dtype, 0.2)
        dY = tensor(g, (T, M), dtype)
        x, wg, wu, dy = (ref.f64(t) for t in (X, Wg, Wu, dY))

        def loss_linear(x, w):
            return float((dy * ref.act(name, x @ w.T)).sum())

        def loss_gated(x, wg, wu):
            return float((dy * ref.act(name, x @ wg.T) * (x @ wu.T)).sum())

        # pre-activations in float64 rounded to the type, as the forward call keeps them
        Zf = (x @ wg.T), (x @ wu.T)
        G, U = (z.to(dtype).cuda() for z in Zf)
        for loss, args, grads, want in [
                (loss_linear, (x, wg), vq.linear_backward(dY, X, Wg, pre=G, act=name)[:2],
                 ref.linear_backward(dY, X, Wg, G, name, dtype)),
                (loss_gated, (x, wg, wu), vq.gated_backward(dY, X, Wg, Wu, G, U, act=name)[:3],
                 ref.gated_backward(dY, X, Wg, Wu, G, U, name, dtype))]:
            for k, (a, got) in enumerate(zip(args, grads)):
                v = torch.randn(a.shape, generator=g, dtype=torch.float64)
                h = 1e-5
                up, dn = list(args), list(args)
                up[k] = a + h * v
                dn[k] = a - h * v
                fd = (loss(*up) - loss(*dn)) / (2 * h)
                # the kept values' rounding (2^-11 of each) moves the gradient's terms by at most that, twice over
                slack = float((want[k][1] * v.abs()).sum()) + 2.0 ** -9 * float((want[k][0].abs() * v.abs()).sum()) \
                    + 2.0 ** -9 * gradient_scale(k, dy, x, wg, wu, Zf, v, loss is loss_gated)
                assert abs(float((ref.f64(got) * v).sum()) - fd) <= slack, (name, k)


def gradient_scale(k, dy, x, wg, wu, Zf, v, is_gated):
    """Sum of the magnitudes of the terms of the directional derivative along v."""
    g, u = (z.abs() for z in Zf)
    dg = dy.abs() * ((u if is_gated else 1.0) * 1.2)
    du = dy.abs() * (g + 1.0)
    if k == 0:
        s = dg @ wg.abs()
        if is_gated:
            s = s + du @ wu.abs()
        return float((s * v.abs()).sum())
    d = dg if k == 1 else du
    return float(((d.T @ x.abs()) * v.abs()).sum())


def test_other_stream():
    """Work follows the current stream: a result that depends on earlier work of that stream."""
    say("stream")
    g = torch.Generator().manual_seed(13)
    X, W = tensor(g, (64, 512), torch.bfloat16), tensor(g, (256, 512), torch.bfloat16)
    want = vq.linear(X, W, act="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        X2 = torch.zeros_like(X)
        for _ in range(20):
            X2 = X2 + 0
        X2.copy_(X)
        Y = vq.linear(X2, W, act="silu")
    s.synchronize()
    assert torch.equal(Y.view(torch.int16), want.view(torch.int16))


def test_input_check_names_the_array(monkeypatch):
    say("VQ_CHECK")
    monkeypatch.setenv("VQ_CHECK", "1")
    g = torch.Generator().manual_seed(15)
    for dtype in DT.values():
        X, W = tensor(g, (4, 30), dtype, 1.0, "odd"), tensor(g, (10, 30), dtype, 1.0, "pitched")
        vq.linear(X, W)
        W[3, 29] = float("inf")
        with pytest.raises(vq.VQError, match="W holds 1 non-finite"):
            vq.linear(X, W)


def exact_to_rounding(got, want, dtype, arg):
    """Each element within its own rounding of want: u, the hardware exponential's error (2^-23 of the value for each
    unit of its argument, and a few more), or half the smallest subnormal.  No share of any other value."""
    off = (ref.f64(got) - want).abs()
    bound = want.abs() * (ref.UNIT[dtype] + (8 + arg.abs()) * 2.0 ** -23) + ref.TINY[dtype]
    say("   max error / bound = %.3g" % float((off / bound).max()))
    return bool((off <= bound).all())


@pytest.mark.parametrize("dt", DT)
def test_sigmoid_gradient_far_from_zero(dt):
    """The derivative sigma(z) sigma(-z) to its own rounding on both sides of zero, where 1 - sigma(z) has no bits left."""
    say("sigmoid gradient", dt)
    dtype = DT[dt]
    z = torch.tensor([v for a in (0.5, 4, 8, 9.5, 10, 12, 13, 14, 15, 16, 16.5, 17, 18, 20, 24) for v in (a, -a)],
                     dtype=torch.float64)
    n = len(z)
    X = torch.eye(n, dtype=dtype, device="cuda")
    W = torch.zeros((1, n), dtype=dtype, device="cuda")
    one = torch.ones((n, 1), dtype=dtype, device="cuda")
    Z = z.to(dtype).cuda()[:, None].contiguous()
    want, half = torch.sigmoid(z) * torch.sigmoid(-z), torch.full((n, 1), 0.5, dtype=dtype, device="cuda")
    # row t of dW is dZ of token t alone
    _, dW, _ = vq.linear_backward(one, X, W, pre=Z, act="sigmoid", want_dx=False)
    assert exact_to_rounding(dW[0], want, dtype, z)
    _, dWg, dWu, _, _ = vq.gated_backward(one, X, W, W.clone(), Z, half, act="sigmoid", want_dx=False)
    assert exact_to_rounding(dWg[0], 0.5 * want, dtype, z)
    assert exact_to_rounding(dWu[0], torch.sigmoid(z), dtype, z)


@pytest.mark.parametrize("name", ref.ACTS)
def test_nan_pre_activations_reach_the_gradients(name):
    """A NaN that the forward pass kept makes NaN of every gradient whose sums it enters, and of no other."""
    say("NaN pre-activation", name)
    T, M, N = 9, 40, 24
    g = torch.Generator().manual_seed(23)
    X, dY = tensor(g, (T, N), torch.bfloat16), tensor(g, (T, M), torch.bfloat16)
    Wg, Wu = (tensor(g, (M, N), torch.bfloat16) for _ in range(2))
    G, U = (tensor(g, (T, M), torch.bfloat16) for _ in range(2))
    clean = vq.gated_backward(dY, X, Wg, Wu, G, U, act=name, want_db=True)
    G[4, 7] = float("nan")
    row = torch.arange(T, device="cuda")[:, None] == 4
    col = torch.arange(M, device="cuda") == 7
    got = vq.gated_backward(dY, X, Wg, Wu, G, U, act=name, want_db=True)
    # with act "none" the derivative is 1 whatever G is: dG does not depend on it
    into_g = name != "none"
    bad = (row, col[:, None] & into_g, col[:, None], col & into_g, col)
    for k, (o, c, b) in enumerate(zip(got, clean, bad)):
        b = b.expand_as(o)
        assert torch.equal(torch.isnan(o), b), (name, k)
        assert torch.equal(o[~b].view(torch.int16), c[~b].view(torch.int16)), (name, k)
    if name != "none":
        dX, dW, db = vq.linear_backward(dY, X, Wg, pre=G, act=name, want_db=True)
        for o, b in ((dX, row), (dW, col[:, None]), (db, col)):
            assert torch.equal(torch.isnan(o), b.expand_as(o)), name


# Sizes for which the plan takes the 256 x 256 tile (mostly ragged past it: odd rows, which are
# copied, and rows of a multiple of eight, which are not), and what else it takes with it.
LARGE_TILES = [
    ("linear", 4728, 1703, 130),             # 7 x 19 tiles, each over all of k
    ("linear", 4304, 408, 4360),             # 2 x 17, sums split
    ("gated", 870, 4890, 135),               # pair of half tiles, 39 x 4
    ("gated", 152, 4368, 3512),              # split sums of a pair
    ("linear_backward", 664, 736, 6104),     # dX and dW in one launch, dX first
    ("linear_backward", 821, 569, 6124),     # dW first
    ("linear_backward", 2870, 144, 1969),    # dW's sums split
    ("linear_backward", 282, 3665, 1494),    # dX's
    ("linear_backward", 4344, 4280, 136),    # both; bias sums over 32 rows a workgroup
    ("linear_backward", 4340, 4276, 139),    # the same from odd rows
    ("linear_backward", 4340, 4277, 139),    # and from odd rows of the pre-activations
    ("gated_backward", 576, 280, 6176),      # dX of two segments, two dW
    ("gated_backward", 669, 313, 6033),      # dW first
    ("gated_backward", 3664, 2984, 152),     # both split; 32 rows a workgroup in the elementwise pass
    ("gated_backward", 3664, 2983, 151),     # the same from odd rows
    ("gated_backward", 752, 5976, 557),      # dX split, 32 rows
    ("gated_backward", 279, 5151, 1413),     # one after the other: dX by 128 x 128 split, dW by 256 x 256
    ("gated_backward", 4204, 535, 3148),     # dX by 256 x 256, dW by 128 x 128
    ("gated_backward", 440, 3506, 4487),     # both by 256 x 256, dX's sums split and both in one place of the workspace
]


@pytest.mark.parametrize("case", LARGE_TILES, ids=["%s_%dx%dx%d" % c for c in LARGE_TILES])
@pytest.mark.parametrize("dt", DT)
def test_large_tiles(case, dt):
    op, T, M, N = case
    dtype = DT[dt]
    name = ref.ACTS[(T + M + N + (dt == "f16")) % len(ref.ACTS)]
    say(op, T, M, N, dt, name)
    g = torch.Generator().manual_seed(T + M + N)
    X = tensor(g, (T, N), dtype)
    W = [tensor(g, (M, N), dtype, N ** -0.5) for _ in range(2 if op.startswith("gated") else 1)]
    b = [tensor(g, (M,), dtype) for _ in W]
    if op == "linear":
        R = tensor(g, (T, M), dtype)
        check(op, vq.linear(X, W[0], bias=b[0], residual=R, act=name, want_pre=True),
              ref.linear(X, W[0], b[0], R, name, dtype))
        return
    if op == "gated":
        check(op, vq.gated(X, *W, bias_gate=b[0], bias_up=b[1], act=name, want_pre=True),
              ref.gated(X, *W, *b, name, dtype))
        return
    dY = tensor(g, (T, M), dtype)
    Z = [tensor(g, (T, M), dtype, 1.5) for _ in W]
    if op == "linear_backward":
        want = ref.linear_backward(dY, X, W[0], Z[0], name, dtype)
        check(op, vq.linear_backward(dY, X, W[0], pre=Z[0], act=name, want_db=True), want)
        check("dX alone", vq.linear_backward(dY, X, W[0], pre=Z[0], act=name, want_dw=False)[:1], want[:1])
        check("dW alone", vq.linear_backward(dY, X, W[0], pre=Z[0], act=name, want_dx=False)[1:2], want[1:2])
    else:
        want = ref.gated_backward(dY, X, *W, *Z, name, dtype)
        check(op, vq.gated_backward(dY, X, *W, *Z, act=name, want_db=True), want)
        check("dX alone", vq.gated_backward(dY, X, *W, *Z, act=name, want_dw=False)[:1], want[:1])
        check("dW alone", vq.gated_backward(dY, X, *W, *Z, act=name, want_dx=False)[1:3], want[1:3])
