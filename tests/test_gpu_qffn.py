"""The feed-forward calls on compressed matrices against float64 (GPU).

The reference multiplies by the oracle's reconstruction in float64.  Every
output is held to the bound that include/vq.h states for the sums, carried
through the epilogue.  The cases cover every sub-vector length, one token to
more than a launch's worth, residual codebooks in LDS, in memory and absent,
rows that end inside a block of 32 sub-vectors, parts split over workgroups,
rows without and full of exact entries, misaligned codebooks and strided
tokens, and the types.
"""
import sys

import numpy as np
import pytest
import torch

import ffn_reference as ref
import oracle
from gpu_util import bits_equal, dev, host
from hessian_weighted_vector_amd import synth, vq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def make_matrix(g, M, N, d, K1, K2, scales, nnz_per_row, full_row=None):
    """A seeded compressed matrix (numpy arrays, no method arithmetic)."""
    nb = N // d
    q = dict(M=M, N=N, d=d, C1=(0.02 * g.standard_t(4.0, size=(K1, d))).astype(np.float32),
             idx1=g.integers(0, K1, M * nb).astype(np.uint16), C2=None, idx2=None, rscale=None, cscale=None,
             row_ptr=None, col=None, val=None)
    if K2:
        q["C2"] = (0.004 * g.standard_normal((K2, d))).astype(np.float32)
        q["idx2"] = g.integers(0, K2, M * nb).astype(np.uint16)
    if scales:
        q["rscale"] = g.uniform(0.5, 2.0, M).astype(np.float32)
        q["cscale"] = g.uniform(0.5, 2.0, N).astype(np.float32)
    if nnz_per_row is not None:
        per = np.minimum(g.integers(0, nnz_per_row + 1, size=M), N)
        per[0] = 0
        if full_row is not None:
            per[full_row] = N
        q["row_ptr"] = np.concatenate([[0], np.cumsum(per)]).astype(np.int32)
        q["col"] = np.concatenate([np.sort(g.choice(N, k, replace=False)) for k in per]).astype(np.int32)
        q["val"] = (0.2 * g.standard_t(3.0, size=q["col"].size)).astype(np.float32)
    return q


def on_gpu(q, misalign=False):
    t = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in q.items()}
    if misalign:
        for k in ("C1", "C2"):
            if t[k] is not None:
                buf = torch.empty(t[k].numel() + 1, dtype=torch.float32, device="cuda")
                buf[1:] = t[k].reshape(-1)
                t[k] = buf[1:].view(t[k].shape)
    return vq.QMatrix(**t)


def sums(q, X, dtype):
    """(X W^T, bound on the kernel's float32 sums) in float64."""
    rec = dict(M=q["M"], N=q["N"], d=q["d"], C1=q["C1"], idx1=q["idx1"], C2=q["C2"], idx2=q["idx2"], r=q["rscale"],
               c=q["cscale"])
    What = torch.from_numpy(oracle.reconstruct(**rec, row_ptr=q["row_ptr"], col=q["col"], val=q["val"]).astype(np.float64))
    Wd = torch.from_numpy(oracle.reconstruct(**rec, row_ptr=None, col=None, val=None).astype(np.float64))
    X = ref.f64(X)
    S = X.abs() @ Wd.abs().T + X.abs() @ (What - Wd).abs().T
    nnz = 0.0
    if q["row_ptr"] is not None:
        nnz = torch.from_numpy(np.diff(q["row_ptr"]).astype(np.float64))[None, :]
    eps = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -16
    return X @ What.T, ((q["N"] + nnz + 64) * 2.0 ** -23 + eps) * S


def check(name, got, value, error, dtype):
    bound = ref.stored(value, error, dtype)
    got = ref.f64(got)
    assert got.shape == value.shape
    ratio = (got - value).abs() / bound
    worst = float(ratio.max()) if ratio.numel() else 0.0
    say("   %s max error / bound = %.3g" % (name, worst))
    assert worst <= 1.0, (name, worst)


def add_bias(z, e, b):
    if b is None:
        return z, e
    b = ref.f64(b)
    return z + b, e + 2.0 ** -23 * (z.abs() + b.abs())


def activated(name, z, e):
    y = ref.act(name, z)
    return y, ref.LIPSCHITZ * e + ref.ACT_REL * y.abs()


def tokens(g, T, N, dtype, pad=0):
    v = torch.from_numpy(g.standard_normal((T, N + pad))).to(dtype).cuda()
    return v[:, :N] if pad else v


CASES = [
    # (M, N, d, K1, K2, T, scales, nnz_per_row)
    (1, 8, 8, 1, 0, 1, False, None),
    (16, 64, 8, 16, 0, 1, False, None),
    (37, 40, 8, 33, 5, 3, True, 3),          # a row shorter than one lane's eight sub-vectors
    (130, 264, 8, 256, 256, 8, True, 6),     # residual codebook in LDS; a row of 33 sub-vectors
    (70, 512, 8, 1000, 300, 16, True, 9),    # residual codebook in memory
    (33, 2056, 8, 4096, 256, 17, True, 40),  # two token fragments, parts split over workgroups
    (48, 8200, 8, 3000, 0, 32, False, 20),
    (20, 136, 8, 64, 16, 35, True, 4),       # two launches
    (40, 260, 4, 100, 50, 5, True, 5),       # d = 4, odd number of sub-vectors
    (33, 1028, 4, 700, 600, 19, False, 12),
    (16, 24, 3, 7, 4, 2, True, 2),
    (8, 8, 1, 5, 3, 1, True, 1),
    (50, 96, 6, 40, 0, 13, False, 4),
    (9, 700, 7, 11, 7, 4, True, 5),
    (25, 130, 5, 30, 8, 20, False, None),
    (18, 66, 2, 9, 3, 6, True, 2),
]


@pytest.mark.parametrize("case", CASES, ids=["%dx%d_d%d_T%d" % (c[0], c[1], c[2], c[5]) for c in CASES])
@pytest.mark.parametrize("dt", DT)
def test_qlinear_and_qgated(case, dt):
    M, N, d, K1, K2, T, scales, nz = case
    dtype = DT[dt]
    say("qffn", case, dt)
    g = np.random.default_rng([77, M, N, T])
    q = [make_matrix(g, M, N, d, K1, K2, scales, nz) for _ in range(2)]
    Q = [on_gpu(m) for m in q]
    name = ref.ACTS[(M + N + T) % len(ref.ACTS)]
    X = tokens(g, T, N, dtype)
    b = [tokens(g, 1, M, dtype)[0].contiguous() for _ in range(2)]
    R = tokens(g, T, M, dtype)
    z = [sums(m, X, dtype) for m in q]

    check("qlinear", vq.qlinear(Q[0], X), *z[0], dtype)
    y, e = activated(name, *add_bias(*z[0], b[0]))
    r = ref.f64(R)
    y, e = y + r, e + 2.0 ** -23 * (y.abs() + r.abs())
    got = vq.qlinear(Q[0], X, bias=b[0], residual=R, act=name)
    check("qlinear " + name, got, y, e, dtype)
    again = vq.qlinear(Q[0], X, bias=b[0], residual=R, act=name, out=R)
    assert again is R and bits_equal(host(again.view(torch.int16 if dtype != torch.float32 else torch.int32)),
                                     host(got.view(torch.int16 if dtype != torch.float32 else torch.int32)))

    for bg, bu in ((None, None), (b[0], b[1])):
        a, ea = activated(name, *add_bias(*z[0], bg))
        u, eu = add_bias(*z[1], bu)
        h = a * u
        eh = a.abs() * eu + u.abs() * ea + ea * eu + 2.0 ** -23 * h.abs()
        check("qgated " + name, vq.qgated(Q[0], Q[1], X, bias_gate=bg, bias_up=bu, act=name), h, eh, dtype)


@pytest.mark.parametrize("d", [8, 4])
def test_misaligned_codebooks_strided_tokens_full_rows(d):
    say("misaligned codebooks, d =", d)
    g = np.random.default_rng([78, d])
    q = make_matrix(g, 40, 128, d, 64, 32, True, 4, full_row=7)
    for dtype in DT.values():
        X = tokens(g, 6, 128, dtype, pad=3)
        z, e = sums(q, X, dtype)
        check("misaligned", vq.qlinear(on_gpu(q, misalign=True), X), z, e, dtype)
        check("aligned", vq.qlinear(on_gpu(q), X), z, e, dtype)
        out = tokens(g, 6, 40, dtype, pad=5)
        assert vq.qlinear(on_gpu(q), X, out=out) is out
        check("strided out", out, z, e, dtype)


@pytest.mark.parametrize("d,nb", [(8, 34), (8, 35), (4, 70), (4, 37), (6, 33), (6, 40), (7, 8), (5, 3)])
def test_indices_at_odd_addresses(d, nb):
    """Index rows that begin at odd elements, by their number or by their array's address; a codebook above and below L1's size."""
    say("odd index rows, d =", d, "nb =", nb)
    g = np.random.default_rng([83, d, nb])
    for K1 in (30, min(5000, 150 * nb)):
        q = make_matrix(g, 150, d * nb, d, K1, 20, False, 2)
        X = tokens(g, 2, d * nb, torch.float32)
        z, e = sums(q, X, torch.float32)
        t = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in q.items()}
        check("as they are", vq.qlinear(vq.QMatrix(**t), X), z, e, torch.float32)
        for k in ("idx1", "idx2"):
            buf = torch.zeros(t[k].numel() + 1, dtype=torch.uint16, device="cuda")
            buf[1:] = t[k]
            t[k] = buf[1:]
        check("shifted", vq.qlinear(vq.QMatrix(**t), X), z, e, torch.float32)


def test_matrices_of_a_pair_may_differ():
    """One with a residual stage in memory, scales and a sparse part, one without any."""
    say("differing pair")
    g = np.random.default_rng([79])
    a = make_matrix(g, 30, 320, 8, 100, 600, True, 9)
    b = make_matrix(g, 30, 320, 8, 1000, 0, False, None)
    X = tokens(g, 4, 320, torch.float32)
    for p, q in ((a, b), (b, a)):
        (z0, e0), (z1, e1) = sums(p, X, torch.float32), sums(q, X, torch.float32)
        y, ey = activated("silu", z0, e0)
        check("pair", vq.qgated(on_gpu(p), on_gpu(q), X), y * z1,
              y.abs() * e1 + z1.abs() * ey + ey * e1 + 2.0 ** -23 * (y * z1).abs(), torch.float32)


@pytest.mark.parametrize("d,K2,N", [(8, 256, 64), (8, 256, 2048), (4, 512, 8), (4, 512, 1024), (5, 250, 40)])
@pytest.mark.parametrize("T", [1, 3])
def test_residual_codebook_larger_than_the_row(d, K2, N, T):
    """The residual codebook fills its whole place in LDS; the row has fewer quads to stage."""
    say("residual codebook of", K2, "rows, d =", d, "N =", N, "T =", T)
    g = np.random.default_rng([81, d, N, T])
    p, q = (make_matrix(g, 400, N, d, 40, K2, False, 2) for _ in range(2))
    P, Q = on_gpu(p), on_gpu(q)
    for dtype in DT.values():
        X = tokens(g, T, N, dtype)
        (z0, e0), (z1, e1) = sums(p, X, dtype), sums(q, X, dtype)
        check("qlinear", vq.qlinear(P, X), z0, e0, dtype)
        y, ey = activated("silu", z0, e0)
        check("qgated", vq.qgated(P, Q, X), y * z1,
              y.abs() * e1 + z1.abs() * ey + ey * e1 + 2.0 ** -23 * (y * z1).abs(), dtype)


def test_no_tokens_reproducible_and_refresh():
    say("T = 0, reproducible, refresh")
    g = np.random.default_rng([80])
    q = make_matrix(g, 64, 1024, 8, 300, 64, True, 12)
    Q = on_gpu(q)
    for dtype in DT.values():
        E = torch.empty((0, 1024), dtype=dtype, device="cuda")
        assert vq.qlinear(Q, E).shape == (0, 64)
        assert vq.qgated(Q, Q, E).shape == (0, 64)
    X = tokens(g, 5, 1024, torch.float32)
    a, b = vq.qlinear(Q, X), vq.qlinear(Q, X)
    assert bits_equal(host(a), host(b))
    Q.val.mul_(2.0)
    Q.refresh()
    q2 = dict(q, val=q["val"] * 2)
    check("refreshed", vq.qlinear(Q, X), *sums(q2, X, torch.float32), torch.float32)


def test_served_from_a_fit():
    """fit -> QMatrix -> one token: the compressed product equals the product with the fit's reconstruction."""
    say("from a fit")
    inp = synth.small_case(31, 96, 256, d=8)
    W, h = dev(inp["W"]), dev(inp["h"])
    out = vq.fit(W, h, 8, 128, 3, 32, 2, 0.02, binorm=True, perm1=inp["perm1"], perm2=inp["perm2"])
    Q = vq.QMatrix.from_fit(out, 96, 256, 8)
    g = np.random.default_rng([81])
    X = tokens(g, 1, 256, torch.float32)
    z = ref.f64(X) @ ref.f64(out["W_hat"]).T
    S = ref.f64(X).abs() @ ref.f64(out["W_hat"]).abs().T
    # the decoded weights under the exact entries count twice over in the bound's S
    check("fit", vq.qlinear(Q, X), z, (256 + 64 + 256) * 2.0 ** -23 * 3 * S, torch.float32)
    nofit = vq.fit(W, h, 8, 128, 2, perm1=inp["perm1"])
    Q2 = vq.QMatrix.from_fit(nofit, 96, 256, 8)
    z = ref.f64(X) @ ref.f64(nofit["W_hat"]).T
    S = ref.f64(X).abs() @ ref.f64(nofit["W_hat"]).abs().T
    check("fit, one stage", vq.qlinear(Q2, X), z, (256 + 64) * 2.0 ** -23 * S + 2.0 ** -22 * S, torch.float32)


def test_out_of_range_indices_stay_in_bounds():
    """Indices at or above K read the last row; sparse columns out of range are skipped."""
    say("out-of-range indices")
    g = np.random.default_rng([82])
    for d in (8, 4, 3):
        q = make_matrix(g, 20, 24 * d, d, 40, 10, True, 3)
        bad = dict(q, idx1=q["idx1"].copy(), idx2=q["idx2"].copy())
        bad["idx1"][::5] = 65535
        bad["idx2"][::7] = 10
        fixed = dict(bad, idx1=np.minimum(bad["idx1"], 39), idx2=np.minimum(bad["idx2"], 9))
        X = tokens(g, 3, 24 * d, torch.float32)
        assert bits_equal(host(vq.qlinear(on_gpu(bad), X)), host(vq.qlinear(on_gpu(fixed), X)))


def test_input_check_names_the_array(monkeypatch):
    say("VQ_CHECK")
    monkeypatch.setenv("VQ_CHECK", "1")
    g = np.random.default_rng([83])
    q = make_matrix(g, 20, 64, 8, 16, 4, True, 3)
    Q = on_gpu(q)
    for dtype in DT.values():
        X = tokens(g, 3, 64, dtype, pad=1)
        vq.qlinear(Q, X)
        X[2, 63] = float("nan")
        with pytest.raises(vq.VQError, match="X holds 1 non-finite"):
            vq.qlinear(Q, X)


def split_left(v, n):
    """What n bfloat16 terms, each the rounding of what the ones before leave, leave of v."""
    v = v.double()
    for _ in range(n):
        v = v - v.bfloat16().double()
    return v


@pytest.mark.parametrize("d", [8, 4, 6])
@pytest.mark.parametrize("dt", DT)
def test_terms_of_same_signed_values(d, dt):
    """Weights and tokens whose bfloat16 terms leave the most, all of one sign, so that no error averages away.

    A residual of minus the rounded sum leaves the difference, which the output type holds to its own
    rounding.  Eps of the split alone: 2^-17 with 16-bit tokens, 2^-23 with float32; beside it the
    float32 sums, N + 8 additions of at most four (bf16: two, float32: six) products of terms each,
    2^-24 of the sum apiece, and the residual's subtraction.
    """
    dtype = DT[dt]
    N, M, K = 2 * d, 16, 32
    g = torch.Generator().manual_seed(24)
    cand = 1 + torch.rand(1 << 16, generator=g) * 2.0 ** -6
    worst = split_left(cand, 1).abs() + 2.0 ** 9 * split_left(cand, 2).abs()
    w = cand[worst.topk(K * d).indices].reshape(K, d)
    w = torch.where(split_left(w, 1) > 0, w, w - 2 * split_left(w, 1).float())     # second terms of one sign
    x = (1 + torch.rand(1 << 16, generator=g) * 2.0 ** -6).to(dtype).float()
    x = x[split_left(x, 1).topk(N).indices] if dtype != torch.bfloat16 else x[:N]
    idx = torch.randint(0, K, (M * 2,), generator=g).to(torch.uint16)
    Q = vq.QMatrix(M, N, d, w.cuda(), idx.cuda())
    X = x.to(dtype)[None, :]
    z = X.double() @ w.double()[idx.long()].reshape(M, N).T
    R = -z.to(dtype)
    terms = {"bf16": 2, "f16": 4, "f32": 6}[dt]
    eps = (2.0 ** -23 if dt == "f32" else 2.0 ** -17) + (N + 8) * terms * 2.0 ** -24
    say("terms", dt, d)
    check("difference", vq.qlinear(Q, X.cuda(), residual=R.cuda()), z + R.double(), eps * z, dtype)


def agree(name, got, value, error, dtype):
    """NaN and infinities where the definition has them; elsewhere within the bound."""
    g, fin = ref.f64(got), torch.isfinite(value)
    assert torch.equal(torch.isnan(g), torch.isnan(value)), name
    inf = torch.isinf(value)
    assert torch.equal(torch.isinf(g), inf) and torch.equal(g[inf], value[inf]), name
    if bool(fin.any()):
        check(name, g[fin], value[fin], error[fin], dtype)


@pytest.mark.parametrize("case", [(60, 264, 8, 100, 20, True), (33, 2056, 8, 200, 300, False), (40, 260, 4, 60, 9, True),
                                  (50, 96, 6, 40, 0, False)], ids=lambda c: "%dx%d_d%d" % c[:3])
@pytest.mark.parametrize("dt", DT)
def test_infinite_and_nan_tokens(case, dt):
    """Infinite and NaN tokens give what the definition gives (at exact entries by the exact weight); other tokens keep their bits."""
    M, N, d, K1, K2, scales = case
    dtype = DT[dt]
    say("non-finite tokens", case, dt)
    g = np.random.default_rng([85, M, N, d])
    q = [make_matrix(g, M, N, d, K1, K2, scales, 9, full_row=5) for _ in range(2)]
    Q = [on_gpu(m) for m in q]
    inf = float("inf")
    X = tokens(g, 18, N, dtype)
    clean = vq.qlinear(Q[0], X), vq.qgated(Q[0], Q[1], X, act="none")
    exact = int(q[0]["col"][0])                       # a column that some row holds exactly
    X[1, 3] = inf
    X[2, N - 1] = -inf
    X[4, exact] = inf
    X[7, 0], X[7, 9] = inf, -inf
    X[9, N // 2] = float("nan")
    X[16] = float("nan")
    X[17, exact], X[17, N - 2] = -inf, 1.0
    if dtype == torch.float32:
        X[11, 5] = 3.4e38                              # finite, and past the largest bfloat16 value
    finite = torch.where(torch.isfinite(X), X, torch.zeros_like(X))
    z = [(ref.f64(X) @ torch.from_numpy(what(m)).T, sums(m, finite, dtype)[1]) for m in q]
    # the sum is formed again where it came out infinite: N + nnz additions, as the bound has them
    same = [t for t in range(18) if t not in (1, 2, 4, 7, 9, 11, 16, 17)]
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    got = vq.qlinear(Q[0], X)
    agree("qlinear", got, *z[0], dtype)
    assert torch.equal(got[same].view(bits), clean[0][same].view(bits))
    agree("relu", vq.qlinear(Q[0], X, act="relu"), ref.act("relu", z[0][0]), z[0][1], dtype)
    got = vq.qgated(Q[0], Q[1], X, act="none")
    (a, ea), (u, eu) = z
    rows = [t for t in range(18) if t != 11]           # the square of 3.4e38 is past the type
    agree("qgated", got[rows], (a * u)[rows], (a.abs() * eu + u.abs() * ea + ea * eu + 2.0 ** -23 * (a * u).abs())[rows], dtype)
    assert torch.equal(got[same].view(bits), clean[1][same].view(bits))


def what(q):
    """The reconstruction, float64 of its float32 values."""
    return oracle.reconstruct(M=q["M"], N=q["N"], d=q["d"], C1=q["C1"], idx1=q["idx1"], C2=q["C2"], idx2=q["idx2"],
                              r=q["rscale"], c=q["cscale"], row_ptr=q["row_ptr"], col=q["col"],
                              val=q["val"]).astype(np.float64)


@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_in_float32(name):
    """Float32 results have float32's accuracy, far past the 16-bit results' 2^-16.

    One column, a token of 1: the sum is the weight itself.  Relative bound: 8 * 2^-23 for the exponential
    (or error function), the additions, products and the quotient, and twice 2^-23 for each unit of an
    exponent's argument that is itself rounded: z^2 / 2 for GELU, the cubic for its tanh form, none for the
    others.  Results below the smallest normal value may be flushed.
    """
    say("float32 activation", name)
    z = torch.linspace(-20, 20, 4001)
    n = len(z)
    Q = vq.QMatrix(n, 1, 1, z[:, None].contiguous().cuda(), torch.arange(n, dtype=torch.int32).to(torch.uint16).cuda())
    zz = z.double()
    want = ref.act(name, zz)
    if name == "gelu_tanh":
        v = 2 * (2 / np.pi) ** 0.5 * (zz + 0.044715 * zz ** 3)
        want, arg = zz * torch.sigmoid(v), v.abs()      # as ref.act, without its cancellation
    else:
        arg = zz.square() / 2 if name == "gelu" else torch.zeros_like(zz)
    X = torch.ones((1, 1), device="cuda")
    bound = want.abs() * (8 + 2 * arg) * 2.0 ** -23 + 2.0 ** -126
    off = (ref.f64(vq.qlinear(Q, X, act=name))[0] - want).abs()
    say("   max error / bound = %.3g" % float((off / bound).max()))
    assert bool((off <= bound).all())
