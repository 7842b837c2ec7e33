"""The 8-bit products against float64: codes equal, every output within the bound of its scales' roundings."""
import pytest
import torch

import i8_reference as ref
from ffn_reference import ACTS, f64
from hessian_weighted_vector_amd import vq

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def values(shape, dtype, g, more=0, offset=0, scale=1.0):
    """A view with rows `more` elements longer, `offset` elements into its buffer."""
    rows, cols = shape
    buf = torch.full((rows * (cols + more) + offset + 8,), 3.0, dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + more)].view(rows, cols + more)[:, :cols]
    x = scale * torch.randn(shape, generator=g)
    x[:, ::17] *= 20
    v.copy_(x)
    return v


def matrix(M, N, g, more=0):
    """(Int8Matrix, codes, scales): codes over the whole range, -128 among them."""
    buf = torch.full((M, N + more), 99, dtype=torch.int8)
    buf[:, :N] = torch.randint(-128, 128, (M, N), generator=g)
    q = buf.cuda()[:, :N]
    s = (torch.rand(M, generator=g) * 1e-2).cuda()
    return vq.Int8Matrix(q, s), q, s


def within(got, want, what):
    value, bound = want
    half = got.dtype == torch.float16
    got = f64(got)
    assert got.shape == value.shape
    bad = ~((got - value).abs() <= bound)
    if half:                                                 # fp16 rounds values from 65520 on to infinity
        bad &= ~((got == torch.copysign(torch.tensor(float("inf"), dtype=got.dtype), value)) & (value.abs() + bound >= 65520))
    wrong = int(bad.sum())
    assert wrong == 0, "%s: %d of %d, first %s: %r against %r" % (
        what, wrong, bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(value[bad][0]))


SIZES = [(1, 1, 1), (1, 16, 64), (1, 300, 4096), (2, 33, 100), (15, 17, 63), (16, 64, 65), (17, 100, 1000), (32, 257, 129),
         (33, 128, 128), (33, 1, 5), (64, 5, 700), (100, 300, 257), (129, 129, 64), (256, 512, 384), (300, 77, 1), (513, 260, 200)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,M,N", SIZES)
def test_sizes(T, M, N, dtype):
    g = torch.Generator().manual_seed(T * 7 + M)
    X = values((T, N), dtype, g)
    Q, q, s = matrix(M, N, g)
    Q2, q2, s2 = matrix(M, N, g)
    R = values((T, M), dtype, g)
    b = values((1, M), dtype, g)[0].contiguous()
    within(vq.linear_i8(Q, X), ref.linear(X, q, s, None, None, "none", dtype), "linear")
    within(vq.linear_i8(Q, X, bias=b, residual=R, act="silu"), ref.linear(X, q, s, b, R, "silu", dtype), "linear, all")
    within(vq.gated_i8(Q, Q2, X), ref.gated(X, q, s, q2, s2, None, None, "silu", dtype), "gated")
    within(vq.gated_i8(Q, Q2, X, bias_gate=b, bias_up=b, act="gelu"), ref.gated(X, q, s, q2, s2, b, b, "gelu", dtype), "gated, all")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T", [3, 40])
def test_activations(T, name):
    g = torch.Generator().manual_seed(1)
    X = values((T, 200), torch.float16, g, scale=0.05)
    Q, q, s = matrix(70, 200, g)
    Q2, q2, s2 = matrix(70, 200, g)
    within(vq.linear_i8(Q, X, act=name), ref.linear(X, q, s, None, None, name, torch.float16), name)
    within(vq.gated_i8(Q, Q2, X, act=name), ref.gated(X, q, s, q2, s2, None, None, name, torch.float16), name)


@pytest.mark.parametrize("more,offset", [(1, 0), (0, 1), (3, 5), (8, 8)])
@pytest.mark.parametrize("T", [1, 7, 60])
def test_strides_and_alignment(T, more, offset):
    g = torch.Generator().manual_seed(2)
    X = values((T, 333), torch.bfloat16, g, more, offset)
    R = values((T, 91), torch.bfloat16, g, more, offset)
    Q, q, s = matrix(91, 333, g, more)                       # copied into rows of 64
    assert Q.q.data_ptr() != q.data_ptr()
    buf = torch.zeros(T * (91 + more) + offset + 8, dtype=torch.bfloat16, device="cuda")
    out = buf[offset:offset + T * (91 + more)].view(T, 91 + more)[:, :91]
    want = ref.linear(X, q, s, None, R, "none", torch.bfloat16)
    got = vq.linear_i8(Q, X, residual=R, out=out)
    within(got, want, "linear")
    assert not bool(buf[:offset].any()) and (more == 0 or not bool(buf[offset:offset + T * (91 + more)].view(T, -1)[:, 91:].any()))
    within(vq.linear_i8(Q, X, residual=R, out=R), want, "in place of the residual")


def test_matrix_in_place():
    """Codes in rows of a multiple of 64 bytes are read where they are, with anything behind them."""
    g = torch.Generator().manual_seed(3)
    Q, q, s = matrix(50, 200, g, 56)
    assert Q.q.data_ptr() == q.data_ptr()
    for T in (2, 50):
        X = values((T, 200), torch.float16, g)
        within(vq.linear_i8(Q, X), ref.linear(X, q, s, None, None, "none", torch.float16), "linear")
    # the last row's end is not readable to the next 64 bytes: a copy
    flat = torch.zeros(49 * 256 + 200, dtype=torch.int8, device="cuda")
    short = flat.as_strided((50, 200), (256, 1))
    short.copy_(q)
    Q2 = vq.Int8Matrix(short, s)
    assert Q2.q.data_ptr() != short.data_ptr()
    assert torch.equal(vq.linear_i8(Q2, X), vq.linear_i8(Q, X))


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("N", [1, 7, 64, 1000, 4096, 4097, 9001, 20000])
def test_codes(N, dtype):
    """16-bit rows: the codes of exact arithmetic, ties to even."""
    g = torch.Generator().manual_seed(4)
    X = values((37, N), dtype, g)
    X[3] = 0
    X[4] = 0
    X[4, N - 1] = -2.0 ** -14
    X[5] = (torch.arange(N) % 255 - 127).to(dtype) / 2       # quotients on ties and on integers
    X[5, 0] = 127.0
    q, s = vq.quantize_rows(X)
    want, scale = ref.codes(X)
    assert torch.equal(q.cpu().double(), want)
    assert bool(((s.cpu().double() - scale).abs() <= 2.0 ** -24 * scale).all())
    full = q.as_strided((37, q.stride(0)), (q.stride(0), 1))
    assert not bool(full[:, N:].any())


def test_codes_of_every_pair_of_mantissas():
    """Every quotient of two bfloat16 mantissas at every distance that leaves a code, by division in float64."""
    a = torch.arange(128, 256, dtype=torch.float64)
    for shift in range(0, 8):
        X = torch.zeros((128, 129), dtype=torch.float64)
        X[:, 0] = a * 2.0 ** shift
        X[:, 1:] = a[None, :].expand(128, 128) if shift else torch.minimum(a[None, :], a[:, None])
        q, _ = vq.quantize_rows(X.bfloat16().cuda())
        assert torch.equal(q.cpu().double(), torch.round(127 * X / X[:, :1]))


def test_codes_of_float32():
    g = torch.Generator().manual_seed(5)
    for N in (100, 5000):
        X = values((20, N), torch.float32, g, 3, 1)
        q, s = vq.quantize_rows(X)
        x = f64(X)
        top = x.abs().amax(1, keepdim=True)
        # the product and the quotient are rounded once each before the integer is taken
        assert bool(((127 * x / top - q.cpu().double()).abs() <= 0.5 + 127 * 2.0 ** -23).all())
        W = vq.Int8Matrix.from_dense(X)
        assert torch.equal(W.q, q) and torch.equal(W.scale, s)


@pytest.mark.parametrize("T", [5, 70])
def test_non_finite_tokens_stay_in_their_rows(T):
    g = torch.Generator().manual_seed(6)
    X = values((T, 150), torch.bfloat16, g)
    Q, q, s = matrix(40, 150, g)
    clean = vq.linear_i8(Q, X)
    X[1, 149], X[4, 3] = float("nan"), float("-inf")
    got = vq.linear_i8(Q, X)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[1] = bad[4] = True
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], clean[~bad])


def test_zero_tokens_and_empty_batches():
    g = torch.Generator().manual_seed(7)
    Q, q, s = matrix(40, 150, g)
    b = values((1, 40), torch.bfloat16, g)[0].contiguous()
    for T in (3, 50):
        X = torch.zeros((T, 150), dtype=torch.bfloat16, device="cuda")
        assert torch.equal(vq.linear_i8(Q, X, bias=b), b.expand(T, 40))
    assert vq.linear_i8(Q, X[:0]).shape == (0, 40) and vq.gated_i8(Q, Q, X[:0]).shape == (0, 40)
    assert vq.quantize_rows(X[:0])[0].shape == (0, 150)


def test_largest_sums():
    """The longest rows with the largest codes: 127 * 128 * 2^17 fits the sum."""
    N = 1 << 17
    Q = vq.Int8Matrix(torch.full((20, N), -128, dtype=torch.int8, device="cuda"), torch.full((20,), 2.0 ** -20, device="cuda"))
    for T in (2, 40):
        X = torch.ones((T, N), dtype=torch.bfloat16, device="cuda")
        want = -128.0 * N * 2.0 ** -20
        assert bool((vq.linear_i8(Q, X).float() == want).all())


@pytest.mark.parametrize("M,N", [(1024, 16384), (100, 131072), (4096, 11008)])
def test_same_tokens_in_every_batch(M, N):
    """Few tokens, tiles of both sizes and split sums give the same bits for the same token."""
    g = torch.Generator().manual_seed(8)
    Q, q, s = matrix(M, N, g)
    X = values((520, N), torch.bfloat16, g)
    R = values((520, M), torch.bfloat16, g)
    whole = vq.linear_i8(Q, X, residual=R)
    hwhole = vq.gated_i8(Q, Q, X)
    for T in (1, 16, 20, 33, 130):
        assert torch.equal(vq.linear_i8(Q, X[:T], residual=R[:T]), whole[:T])
        assert torch.equal(vq.gated_i8(Q, Q, X[:T]), hwhole[:T])
    rows = torch.randint(0, M, (32,), generator=g).cuda()
    want = ref.linear(X[:64], q[rows], s[rows], None, R[:64, rows], "none", torch.bfloat16)
    within(whole[:64, rows], want, "rows")


@pytest.mark.parametrize("T", [2, 3, 5, 17, 31])
def test_few_tokens_of_large_matrices(T):
    """Past the size at which few tokens go through tiles; odd sizes."""
    M, N = 50001, 4099
    g = torch.Generator().manual_seed(80)
    Q, q, s = matrix(M, N, g)
    X = values((T, N), torch.float16, g, scale=0.05)
    Y, H = vq.linear_i8(Q, X), vq.gated_i8(Q, Q, X, act="none")
    rows = torch.cat([torch.arange(5), torch.randint(0, M, (100,), generator=g), torch.arange(M - 20, M)]).cuda()
    within(Y[:, rows], ref.linear(X, q[rows], s[rows], None, None, "none", torch.float16), "linear")
    within(H[:, rows], ref.gated(X, q[rows], s[rows], q[rows], s[rows], None, None, "none", torch.float16), "gated")
    assert torch.equal(vq.linear_i8(Q, X[:1]), Y[:1]) and torch.equal(vq.gated_i8(Q, Q, X[T - 1:], act="none"), H[T - 1:])


@pytest.mark.parametrize("T", [33, 100, 128])
def test_one_round_of_tiles(T):
    """Workgroups that begin at different steps: the sums of a token are those of it alone."""
    M, N = 20001, 2100
    g = torch.Generator().manual_seed(81)
    Q, q, s = matrix(M, N, g)
    X, R = values((T, N), torch.bfloat16, g), values((T, M), torch.bfloat16, g)
    Y, H = vq.linear_i8(Q, X, residual=R), vq.gated_i8(Q, Q, X)
    for t in (0, 31, T - 1):
        assert torch.equal(vq.linear_i8(Q, X[t:t + 1], residual=R[t:t + 1]), Y[t:t + 1])
        assert torch.equal(vq.gated_i8(Q, Q, X[t:t + 1]), H[t:t + 1])
    rows = torch.cat([torch.randint(0, M, (100,), generator=g), torch.arange(M - 20, M)]).cuda()
    within(Y[:, rows], ref.linear(X, q[rows], s[rows], None, R[:, rows], "none", torch.bfloat16), "linear")


@pytest.mark.parametrize("T", [1, 80])
def test_captured_graphs_and_streams(T):
    g = torch.Generator().manual_seed(9)
    Q, q, s = matrix(2000, 1000, g)
    Q2, q2, s2 = matrix(1000, 2000, g)
    X = values((T, 1000), torch.float16, g, scale=0.01)
    ws = torch.empty(max(vq.load().vq_gated_i8_workspace_bytes(2000, 1000, T), vq.load().vq_linear_i8_workspace_bytes(1000, 2000, T)),
                     dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        H = vq.gated_i8(Q, Q, X, ws=ws)                      # both calls on one workspace
        Y = vq.linear_i8(Q2, H, residual=X, ws=ws)
    for k in range(4):
        X.copy_(values((T, 1000), torch.float16, g, scale=0.01))
        graph.replay()
        torch.cuda.synchronize()
        h = vq.gated_i8(Q, Q, X)
        assert torch.equal(H, h) and torch.equal(Y, vq.linear_i8(Q2, h, residual=X))
        with torch.cuda.stream(st):
            other = vq.linear_i8(Q2, h, residual=X)
        st.synchronize()
        assert torch.equal(Y, other)


def test_refusals_and_value_check(monkeypatch):
    g = torch.Generator().manual_seed(10)
    Q, q, s = matrix(40, 150, g)
    Q2, _, _ = matrix(41, 150, g)
    X = values((3, 150), torch.bfloat16, g)
    with pytest.raises(TypeError, match="bfloat16 or torch.float16"):
        vq.linear_i8(Q, X.float())
    with pytest.raises(ValueError, match="X must be"):
        vq.linear_i8(Q, X[:, :149])
    with pytest.raises(vq.VQError, match="the same"):
        vq.gated_i8(Q, Q2, X)
    with pytest.raises(vq.VQError, match="workspace"):
        vq.linear_i8(Q, X, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="scale"):
        vq.Int8Matrix(q, s[:3])
    monkeypatch.setenv("VQ_CHECK", "1")
    vq.linear_i8(Q, X)
    s[3] = float("nan")
    with pytest.raises(vq.VQError, match="scale of W"):
        vq.linear_i8(Q, X)
