// The dense feed-forward calls: the product with bias, activation and residual
// (vq_linear), the gated pair of projections (vq_gated), and their backward
// passes.  The products run in vq_gemm.hip; here are the elementwise kernels
// around them and the entry points.
//
//   k_pack        a copy with 16-byte aligned rows, zero padded to a multiple
//                 of eight, for operands that are not (odd sizes, odd strides)
//   k_grad        dZ = dY act'(Z), or dG = dH U act'(G) and dU = dH act(G), and
//                 the bias gradients' partial column sums, in one pass
//                 (the copies above ride in its launch)
//   k_zero_rows   gradients of zero tokens
//
// The gradients of the pre-activations are rounded to the tensors' 16-bit type
// once, since the matrix cores read them in it: one rounding of each, independent over
// the products' sums.  In bf16 it is at most 2^-8 of the value.  In fp16 it is at most
// 2^-11 of values from 2^-14 to 65504, 2^-25 absolute below and infinite above, also
// where dX and dW themselves would be representable: fp16 callers scale their losses
// so that dY act'(Z), dH U act'(G) and dH act(G) stay in that range.  The bias
// gradients are summed from the unrounded values.
#include "vq_ffn.h"

#include <algorithm>

namespace vq {
namespace {

constexpr int64_t kMaxTokens = 1 << 28;

// blockIdx.y: the matrix.
__global__ __launch_bounds__(256) void k_pack(const Packs a) { pack_rows(a.m[blockIdx.y], blockIdx.x, gridDim.x); }

__global__ __launch_bounds__(256) void k_zero_rows(uint16_t* __restrict__ o, int64_t rows, int64_t cols, int64_t ld)
{
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * cols; e += (int64_t)gridDim.x * 256)
        o[e / cols * ld + e % cols] = 0;
}

// A workgroup's four waves take R rows each of 512 columns (eight a lane), and
// their column sums join in LDS.  GATED: D0 = dG, D1 = dU.  D0 may be null (bias
// gradient alone).  D0 and D1 have zero-padded rows of ldd.  Bound by its bytes:
// 4096 x 8192, act'(Z) from bf16, 201 MB in 48 us (4.2 TB/s; a large copy reaches
// 4.9); gated 2048 x 11008, 225 MB in 55 us.  Four rows in flight took 69 us there.
// Neighbouring workgroups take neighbouring columns: whole rows come from memory
// together (a backward call of 4096 x 8192 x 2048 279 us without, 268 with).
template <class T, bool GATED, int R, bool ODD>
__global__ __launch_bounds__(256) void k_grad(int64_t nt, int M, int act, const void* dY, int64_t ldy, const void* Z0,
                                              const void* Z1, int64_t ldz, typename T::E* D0, typename T::E* D1,
                                              int64_t ldd, float* part0, float* part1, const Packs packs)
{
    if (blockIdx.y >= (M + 511) / 512) {                     // the operands' copies, in the same launch
        const int id = (blockIdx.y - (M + 511) / 512) * gridDim.x + blockIdx.x;
        if (id < packs.blocks * packs.count) pack_rows(packs.m[id / packs.blocks], id % packs.blocks, packs.blocks);
        return;
    }
    __shared__ float sums[GATED ? 2 : 1][4][512];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int ncol = (M + 511) / 512, wid = blockIdx.y * gridDim.x + blockIdx.x, by = wid % ncol, bx = wid / ncol;
    const int m = by * 512 + lane * 8;
    const int64_t t0 = ((int64_t)bx * 4 + wave) * R;
    float c0[8] = {}, c1[8] = {};
    if (m < M) {
        constexpr int B = R < 2 ? R : 2;                     // rows whose loads are in flight together
#pragma unroll 1
        for (int r = 0; r < R; r += B) {
            float dy[B][8], z[B][8], u[B][8];
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int64_t t = t0 + r + k < nt ? t0 + r + k : nt - 1;
                load8<T, ODD>(dY, ldy, t, m, M, dy[k]);
                if (GATED || act != VQ_ACT_NONE) load8<T, ODD>(Z0, ldz, t, m, M, z[k]);
                if (GATED) load8<T, ODD>(Z1, ldz, t, m, M, u[k]);
            }
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int64_t t = t0 + r + k;
                if (t >= nt) break;
                float a[8];
                if (GATED || act != VQ_ACT_NONE) {
                    act_grad<GATED>(act, z[k], a);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        z[k][i] *= GATED ? dy[k][i] * u[k][i] : dy[k][i];
                        if (GATED) u[k][i] = dy[k][i] * a[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[k][i] = dy[k][i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c0[i] += z[k][i];
                    if (GATED) c1[i] += u[k][i];
                }
                // columns past M (loaded as zero) give zeros: the padding
                if (D0) store8<T>(D0, ldd, t, m, (int)ldd, z[k]);
                if (GATED) store8<T>(D1, ldd, t, m, (int)ldd, u[k]);
            }
        }
    }
    if (!part0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sums[0][wave][lane * 8 + i] = c0[i];
        if (GATED) sums[GATED ? 1 : 0][wave][lane * 8 + i] = c1[i];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 512; k += 256) {
        const int col = by * 512 + k;
        if (col >= M) break;
        part0[(int64_t)bx * M + col] = sums[0][0][k] + sums[0][1][k] + sums[0][2][k] + sums[0][3][k];
        if (GATED) {
            constexpr int b = GATED ? 1 : 0;
            part1[(int64_t)bx * M + col] = sums[b][0][k] + sums[b][1][k] + sums[b][2][k] + sums[b][3][k];
        }
    }
}

// Rows a workgroup takes: 32, or 4 where that leaves less than a workgroup a CU.  Gated
// bias gradients with a pass over 2048 x 11008: 43 us with 32 and 60 us with 4 (the
// partial sums' bytes); 512 x 8192: 18 and 16 us.
int grad_rows(int64_t T, int64_t M) { return (M + 511) / 512 * ((T + 31) / 32) < 256 ? 4 : 32; }

// Collects the operands that need a packed copy; each copy in the workspace takes
// its matrix's place, and one launch makes them all.
struct Packer {
    Arena& ws;
    Packs list{};
    int64_t most = 0;
    void add(Mat& m)
    {
        const int64_t ldp = round8(m.cols);
        void* o = ws.take((size_t)m.rows * ldp * 2);
        list.m[list.count++] = {static_cast<const uint16_t*>(m.p), static_cast<uint16_t*>(o), m.rows, m.ld, ldp, (int)m.cols,
                                odd_rows(m.p, m.ld)};
        most = std::max(most, m.rows * (ldp / 8));
        list.blocks = pack_blocks(most);
        m = {o, m.rows, ldp, ldp};
    }
    vq_status launch(hipStream_t st) const
    {
        return pack_launch(list, st);
    }
};

vq_status zero_matrix(void* o, int64_t rows, int64_t cols, int64_t ld, hipStream_t st)
{
    if (!o || rows * cols == 0) return VQ_OK;
    hipLaunchKernelGGL(k_zero_rows, dim3((unsigned)std::min<int64_t>((rows * cols + 255) / 256, 65536)), dim3(256), 0, st,
                       static_cast<uint16_t*>(o), rows, cols, ld);
    VQ_LAUNCHED("k_zero_rows");
    return VQ_OK;
}

// Forward product(s): nm = 1 (linear) or 2 (gated).
struct Forward {
    int64_t T, M, N;
    int dtype, nm;
    const void* X; int64_t ldx;
    const void* W[2]; int64_t ldw;
    Epilogue epi;
};

vq_status forward(const Forward& f, Arena& ws, bool run, hipStream_t st)
{
    if (f.T == 0) return VQ_OK;
    Mat x{f.X, f.T, f.N, f.ldx};
    Mat w[2] = {{f.W[0], f.M, f.N, f.ldw}, {f.W[1], f.M, f.N, f.ldw}};
    const bool packs_w = !loads_ok(w[0]) || (f.nm > 1 && !loads_ok(w[1]));
    // for few tokens a copy of the weights would cost more than the product
    if (few_tokens(f.T, f.M, f.N, f.nm) || (f.T <= 32 && packs_w)) {
        void* part = ws.take(few_workspace(f.T, f.M, f.N, f.nm));
        if (!run) return VQ_OK;
        return few_product({f.T, f.M, f.N, f.dtype, f.nm, f.X, f.ldx, {f.W[0], f.W[1]}, f.ldw, f.epi}, part, st);
    }
    Packer pk{ws};
    if (!loads_ok(x)) pk.add(x);
    // a pair shares one leading dimension: both are packed or neither
    if (packs_w)
        for (int i = 0; i < f.nm; ++i) pk.add(w[i]);
    GemmArgs g{};
    g.kind = f.nm > 1 ? GEMM_GATED : GEMM_LINEAR;
    g.dtype = f.dtype;
    g.np = (int)f.M; g.nq = (int)f.T;
    g.nseg = 1; g.nbatch = 1;
    g.kP = w[0].cols; g.kQ = x.cols;
    for (int i = 0; i < f.nm; ++i) { g.P[i] = w[i].p; }
    g.Q[0] = x.p;
    g.ldp = w[0].ld; g.ldq = x.ld;
    g.epi = f.epi;
    const size_t gb = gemm_workspace(g.kind, g.np, g.nq, f.N, 1, 1);
    void* gw = ws.take(gb);
    if (!run) return VQ_OK;
    VQ_TRY(pk.launch(st));
    return gemm_launch(g, gw, gb, st);
}

struct Backward {
    int64_t T, M, N;
    int dtype, act, nm;
    const void* dY; int64_t lddy;
    const void* X; int64_t ldx;
    const void* W[2]; int64_t ldw;
    const void* Z[2]; int64_t ldz;
    void* dX; int64_t lddx;
    void* dW[2]; int64_t lddw;
    void* db[2];
};

template <class T>
vq_status grad_launch(const Backward& b, void* const (&D)[2], int64_t ldd, float* const (&part)[2], const Packs& packs,
                      hipStream_t st)
{
    typedef typename T::E E;
    const int rows = grad_rows(b.T, b.M);
    const int64_t gx = (b.T + rows - 1) / rows, copies = ((int64_t)packs.blocks * packs.count + gx - 1) / gx;
    const dim3 grid((unsigned)gx, (unsigned)((b.M + 511) / 512 + copies));
#define VQ_GRAD(GATED_, R_, ODD_)                                                                                    \
    hipLaunchKernelGGL((k_grad<T, GATED_, R_, ODD_>), grid, dim3(256), 0, st, b.T, (int)b.M, b.act, b.dY, b.lddy, b.Z[0], \
                       b.Z[1], b.ldz, (E*)D[0], (E*)D[1], ldd, part[0], part[1], packs)
#define VQ_GRAD_ROWS(GATED_, ODD_)           \
    do {                                     \
        if (rows == 32) VQ_GRAD(GATED_, 8, ODD_); \
        else VQ_GRAD(GATED_, 1, ODD_);       \
    } while (0)
    const bool odd = odd_rows(b.dY, b.lddy) || (b.Z[0] && odd_rows(b.Z[0], b.ldz)) || (b.Z[1] && odd_rows(b.Z[1], b.ldz));
    if (b.nm > 1 && odd) VQ_GRAD_ROWS(true, true);
    else if (b.nm > 1) VQ_GRAD_ROWS(true, false);
    else if (odd) VQ_GRAD_ROWS(false, true);
    else VQ_GRAD_ROWS(false, false);
#undef VQ_GRAD_ROWS
#undef VQ_GRAD
    VQ_LAUNCHED("k_grad");
    return VQ_OK;
}

vq_status backward(const Backward& b, Arena& ws, bool run, hipStream_t st)
{
    const bool want_dw = b.dW[0] || b.dW[1], want_db = b.db[0] || b.db[1];
    if (b.T == 0) {
        if (run)
            for (int i = 0; i < b.nm; ++i) {
                VQ_TRY(zero_matrix(b.dW[i], b.M, b.N, b.lddw, st));
                VQ_TRY(zero_matrix(b.db[i], 1, b.M, b.M, st));
            }
        return VQ_OK;
    }
    // gradients of the pre-activations: the caller's dY itself where it is one
    Mat d[2] = {{b.dY, b.T, b.M, b.lddy}, {nullptr, b.T, b.M, b.lddy}};
    const bool own_d = (b.dX || want_dw) && (b.nm > 1 || b.act != VQ_ACT_NONE || !loads_ok(d[0]));
    void* D[2] = {nullptr, nullptr};
    const int64_t ldd = round8(b.M);
    if (own_d || (b.nm > 1 && want_db))
        for (int i = 0; i < b.nm; ++i) {
            D[i] = ws.take((size_t)b.T * ldd * 2);
            d[i] = {D[i], b.T, ldd, ldd};
        }
    float* part[2] = {nullptr, nullptr};
    const int rows = grad_rows(b.T, b.M);
    if (want_db)
        for (int i = 0; i < b.nm; ++i)
            part[i] = static_cast<float*>(ws.take((size_t)((b.T + rows - 1) / rows) * b.M * sizeof(float)));
    Mat x{b.X, b.T, b.N, b.ldx};
    Mat w[2] = {{b.W[0], b.M, b.N, b.ldw}, {b.W[1], b.M, b.N, b.ldw}};
    const int nb = b.dW[0] && b.dW[1] ? 2 : 1;
    const GemmSize sx{GEMM_DX, b.N, b.T, b.M, b.nm, 1}, sw{GEMM_DW, b.N, b.M, b.T, 1, nb};
    const size_t parts = b.dX && want_dw ? gemm_two_workspace(sx, sw)
                         : b.dX          ? gemm_workspace(sx.kind, sx.np, sx.nq, sx.K, sx.nseg, sx.nbatch)
                         : want_dw       ? gemm_workspace(sw.kind, sw.np, sw.nq, sw.K, sw.nseg, sw.nbatch)
                                         : 0;
    void* part_ws = ws.take(parts);
    Packer pk{ws};
    if (want_dw && !loads_ok(x)) pk.add(x);
    if (b.dX && (!loads_ok(w[0]) || (b.nm > 1 && !loads_ok(w[1]))))
        for (int i = 0; i < b.nm; ++i) pk.add(w[i]);
    if (!run) return VQ_OK;
    if (D[0] || want_db) {
        // one grid row of copies or more: a grid has fewer than 2^16 of them
        const bool ride = (b.M + 511) / 512 + (int64_t)pk.list.blocks * pk.list.count / ((b.T + rows - 1) / rows) < 65000;
        if (!ride) VQ_TRY(pk.launch(st));
        const Packs packs = ride ? pk.list : Packs{};
        VQ_TRY(b.dtype == VQ_BF16 ? grad_launch<Bf16>(b, D, ldd, part, packs, st) : grad_launch<F16>(b, D, ldd, part, packs, st));
    } else {
        VQ_TRY(pk.launch(st));
    }
    BiasSum bs{{part[0], part[1]}, {b.db[0], b.db[1]}, (b.T + rows - 1) / rows, (int)b.M, want_db ? b.nm : 0};
    if (!(b.dX && want_dw)) VQ_TRY(bias_sum_launch(b.dtype, bs, st));
    GemmArgs gx{}, gw{};
    gx.dtype = gw.dtype = b.dtype;
    gx.np = gw.np = (int)b.N;
    if (b.dX) {
        gx.kind = GEMM_DX;
        gx.nq = (int)b.T;
        gx.nseg = b.nm; gx.nbatch = 1;
        for (int i = 0; i < b.nm; ++i) { gx.P[i] = w[i].p; gx.Q[i] = d[i].p; }
        gx.ldp = w[0].ld; gx.ldq = d[0].ld;
        gx.kP = b.M; gx.kQ = d[0].cols;
        gx.wp = (int)w[0].cols;
        gx.epi.Y = b.dX; gx.epi.ldy = b.lddx;
    }
    if (want_dw) {
        const int first = b.dW[0] ? 0 : 1;
        gw.kind = GEMM_DW;
        gw.nq = (int)b.M;
        gw.nseg = 1; gw.nbatch = nb;
        gw.P[0] = gw.P[1] = x.p;
        gw.Q[0] = d[first].p; gw.Q[1] = d[1].p;
        gw.ldp = x.ld; gw.ldq = d[0].ld;
        gw.kP = gw.kQ = b.T;
        gw.wp = (int)x.cols; gw.wq = (int)d[0].cols;
        gw.epi.Y = b.dW[first]; gw.epi.ldy = b.lddw;
        gw.Y2 = b.dW[1];
    }
    if (b.dX && want_dw) return gemm_two_launch(gx, gw, bs, part_ws, parts, st);
    if (b.dX) return gemm_launch(gx, part_ws, parts, st);
    return want_dw ? gemm_launch(gw, part_ws, parts, st) : VQ_OK;
}

// ---- argument checks ------------------------------------------------------
vq_status check_sizes(const std::string& call, int64_t T, int64_t M, int64_t N, int dtype, int act)
{
    VQ_CHECK(T >= 0 && T <= kMaxTokens, call + ": T must be in [0, 2^28]");
    VQ_CHECK(M >= 1 && M <= kMaxSize && N >= 1 && N <= kMaxSize, call + ": M and N must be in [1, 2^20]");
    VQ_CHECK(T * std::max(M, N) <= ((int64_t)1 << 40), call + ": T * max(M, N) must be at most 2^40");
    VQ_CHECK(dtype == VQ_BF16 || dtype == VQ_F16, call + ": dtype must be VQ_BF16 or VQ_F16");
    VQ_CHECK(act >= VQ_ACT_NONE && act <= VQ_ACT_SIGMOID, call + ": unknown activation");
    return VQ_OK;
}


}  // namespace

vq_status pack_launch(const Packs& list, hipStream_t st)
{
    if (list.count == 0) return VQ_OK;
    hipLaunchKernelGGL(k_pack, dim3((unsigned)list.blocks, list.count), dim3(256), 0, st, list);
    VQ_LAUNCHED("k_pack");
    return VQ_OK;
}

}  // namespace vq

using namespace vq;

extern "C" {

size_t vq_linear_workspace_bytes(int64_t T, int64_t M, int64_t N, const void* X, int64_t ldx, const void* W, int64_t ldw)
{
    if (check_sizes("vq_linear", T, M, N, VQ_BF16, 0) != VQ_OK) return 0;
    Forward f{T, M, N, VQ_BF16, 1, X, ldx, {W, nullptr}, ldw, {}};
    Arena ws{nullptr};
    return forward(f, ws, false, nullptr) == VQ_OK ? ws.used : 0;
}

vq_status vq_linear(int64_t T, int64_t M, int64_t N, int dtype, int act, const void* X, int64_t ldx, const void* W,
                    int64_t ldw, const void* bias, const void* R, int64_t ldr, void* Y, int64_t ldy, void* Z, int64_t ldz,
                    void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_linear";
    VQ_TRY(check_sizes(call, T, M, N, dtype, act));
    if (T == 0) return VQ_OK;
    VQ_CHECK(X && W && Y, "vq_linear: null pointer");
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "W", W, ldw, N));
    VQ_TRY(check_ld(call, "bias", bias, M, M));
    VQ_TRY(check_ld(call, "R", R, ldr, M));
    VQ_TRY(check_ld(call, "Y", Y, ldy, M));
    VQ_TRY(check_ld(call, "Z", Z, ldz, M));
    VQ_TRY(check_apart(call, {Y, Z}, {X, W, bias}));
    VQ_CHECK(!Z || Z != R, "vq_linear: outputs may not alias inputs");
    VQ_CHECK(Y != R || ldy == ldr, "vq_linear: Y in place of R needs R's leading dimension");
    Forward f{T, M, N, dtype, 1, X, ldx, {W, nullptr}, ldw, {act, {bias, nullptr}, R, Y, {Z, nullptr}, ldr, ldy, ldz}};
    Arena a{nullptr};
    VQ_TRY(forward(f, a, false, as_stream(stream)));
    VQ_TRY(check_workspace(call, ws, ws_bytes, a.used));
    VQ_TRY(check_device());
    VQ_MATRIX(X, T, N, ldx, call, "X");
    VQ_MATRIX(W, M, N, ldw, call, "W");
    VQ_MATRIX(bias, 1, M, M, call, "bias");
    VQ_MATRIX(R, T, M, ldr, call, "R");
    TimedRegion tr("linear", 0, as_stream(stream));
    Arena w{static_cast<char*>(ws)};
    return forward(f, w, true, as_stream(stream));
}

size_t vq_gated_workspace_bytes(int64_t T, int64_t M, int64_t N, const void* X, int64_t ldx, const void* Wg,
                                const void* Wu, int64_t ldw)
{
    if (check_sizes("vq_gated", T, M, N, VQ_BF16, 0) != VQ_OK) return 0;
    Forward f{T, M, N, VQ_BF16, 2, X, ldx, {Wg, Wu}, ldw, {}};
    Arena ws{nullptr};
    return forward(f, ws, false, nullptr) == VQ_OK ? ws.used : 0;
}

vq_status vq_gated(int64_t T, int64_t M, int64_t N, int dtype, int act, const void* X, int64_t ldx, const void* Wg,
                   const void* Wu, int64_t ldw, const void* bg, const void* bu, void* H, int64_t ldh, void* G, void* U,
                   int64_t ldz, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_gated";
    VQ_TRY(check_sizes(call, T, M, N, dtype, act));
    if (T == 0) return VQ_OK;
    VQ_CHECK(X && Wg && Wu && H, "vq_gated: null pointer");
    VQ_CHECK((G == nullptr) == (U == nullptr), "vq_gated: G and U come together");
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "Wg", Wg, ldw, N));
    VQ_TRY(check_ld(call, "Wu", Wu, ldw, N));
    VQ_TRY(check_ld(call, "bg", bg, M, M));
    VQ_TRY(check_ld(call, "bu", bu, M, M));
    VQ_TRY(check_ld(call, "H", H, ldh, M));
    VQ_TRY(check_ld(call, "G", G, ldz, M));
    VQ_TRY(check_ld(call, "U", U, ldz, M));
    VQ_TRY(check_apart(call, {H, G, U}, {X, Wg, Wu, bg, bu}));
    Forward f{T, M, N, dtype, 2, X, ldx, {Wg, Wu}, ldw, {act, {bg, bu}, nullptr, H, {G, U}, 0, ldh, ldz}};
    Arena a{nullptr};
    VQ_TRY(forward(f, a, false, as_stream(stream)));
    VQ_TRY(check_workspace(call, ws, ws_bytes, a.used));
    VQ_TRY(check_device());
    VQ_MATRIX(X, T, N, ldx, call, "X");
    VQ_MATRIX(Wg, M, N, ldw, call, "Wg");
    VQ_MATRIX(Wu, M, N, ldw, call, "Wu");
    VQ_MATRIX(bg, 1, M, M, call, "bg");
    VQ_MATRIX(bu, 1, M, M, call, "bu");
    TimedRegion tr("gated", 0, as_stream(stream));
    Arena w{static_cast<char*>(ws)};
    return forward(f, w, true, as_stream(stream));
}

size_t vq_linear_backward_workspace_bytes(int64_t T, int64_t M, int64_t N, int act, const void* dY, int64_t lddy,
                                          const void* X, int64_t ldx, const void* W, int64_t ldw, int want_dx, int want_dw,
                                          int want_db)
{
    if (check_sizes("vq_linear_backward", T, M, N, VQ_BF16, act) != VQ_OK) return 0;
    void* const on = reinterpret_cast<void*>(uintptr_t(16));      // counted, never used
    Backward b{T, M, N, VQ_BF16, act, 1, dY, lddy, X, ldx, {W, nullptr}, ldw, {nullptr, nullptr}, 0,
               want_dx ? on : nullptr, N, {want_dw ? on : nullptr, nullptr}, N, {want_db ? on : nullptr, nullptr}};
    Arena ws{nullptr};
    return backward(b, ws, false, nullptr) == VQ_OK ? ws.used : 0;
}

vq_status vq_linear_backward(int64_t T, int64_t M, int64_t N, int dtype, int act, const void* dY, int64_t lddy,
                             const void* X, int64_t ldx, const void* W, int64_t ldw, const void* Z, int64_t ldz, void* dX,
                             int64_t lddx, void* dW, int64_t lddw, void* db, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_linear_backward";
    VQ_TRY(check_sizes(call, T, M, N, dtype, act));
    VQ_CHECK(T == 0 || dY, "vq_linear_backward: dY is null");
    VQ_CHECK(T == 0 || !dX || W, "vq_linear_backward: dX needs W");
    VQ_CHECK(T == 0 || !dW || X, "vq_linear_backward: dW needs X");
    VQ_CHECK(T == 0 || act == VQ_ACT_NONE || Z, "vq_linear_backward: the activation's gradient needs Z");
    VQ_TRY(check_ld(call, "dY", dY, lddy, M));
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "W", W, ldw, N));
    VQ_TRY(check_ld(call, "Z", Z, ldz, M));
    VQ_TRY(check_ld(call, "dX", dX, lddx, N));
    VQ_TRY(check_ld(call, "dW", dW, lddw, N));
    VQ_TRY(check_ld(call, "db", db, M, M));
    VQ_TRY(check_apart(call, {dX, dW, db}, {dY, X, W, Z}));
    Backward b{T, M, N, dtype, act, 1, dY, lddy, X, ldx, {W, nullptr}, ldw, {act != VQ_ACT_NONE ? Z : nullptr, nullptr}, ldz,
               dX, lddx, {dW, nullptr}, lddw, {db, nullptr}};
    Arena a{nullptr};
    VQ_TRY(backward(b, a, false, as_stream(stream)));
    VQ_TRY(check_workspace(call, ws, ws_bytes, a.used));
    if (T > 0 || dW || db) VQ_TRY(check_device());
    VQ_MATRIX(dY, T, M, lddy, call, "dY");
    if (dW) VQ_MATRIX(X, T, N, ldx, call, "X");
    if (dX) VQ_MATRIX(W, M, N, ldw, call, "W");
    if (act != VQ_ACT_NONE) VQ_MATRIX(Z, T, M, ldz, call, "Z");
    TimedRegion tr("linear_backward", 0, as_stream(stream));
    Arena w{static_cast<char*>(ws)};
    return backward(b, w, true, as_stream(stream));
}

size_t vq_gated_backward_workspace_bytes(int64_t T, int64_t M, int64_t N, int act, const void* dH, int64_t lddh,
                                         const void* X, int64_t ldx, const void* Wg, const void* Wu, int64_t ldw,
                                         int want_dx, int want_dw, int want_db)
{
    if (check_sizes("vq_gated_backward", T, M, N, VQ_BF16, act) != VQ_OK) return 0;
    void* const on = reinterpret_cast<void*>(uintptr_t(16));      // counted, never used
    void* const w = want_dw ? on : nullptr;
    void* const db = want_db ? on : nullptr;
    Backward b{T, M, N, VQ_BF16, act, 2, dH, lddh, X, ldx, {Wg, Wu}, ldw, {nullptr, nullptr}, 0,
               want_dx ? on : nullptr, N, {w, w}, N, {db, db}};
    Arena ws{nullptr};
    return backward(b, ws, false, nullptr) == VQ_OK ? ws.used : 0;
}

vq_status vq_gated_backward(int64_t T, int64_t M, int64_t N, int dtype, int act, const void* dH, int64_t lddh,
                            const void* X, int64_t ldx, const void* Wg, const void* Wu, int64_t ldw, const void* G,
                            const void* U, int64_t ldz, void* dX, int64_t lddx, void* dWg, void* dWu, int64_t lddw,
                            void* dbg, void* dbu, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_gated_backward";
    VQ_TRY(check_sizes(call, T, M, N, dtype, act));
    VQ_CHECK(T == 0 || (dH && G && U), "vq_gated_backward: null pointer");
    VQ_CHECK(T == 0 || !dX || (Wg && Wu), "vq_gated_backward: dX needs Wg and Wu");
    VQ_CHECK(T == 0 || !(dWg || dWu) || X, "vq_gated_backward: dWg and dWu need X");
    VQ_CHECK((dWg == nullptr) == (dWu == nullptr), "vq_gated_backward: dWg and dWu come together");
    VQ_CHECK((dbg == nullptr) == (dbu == nullptr), "vq_gated_backward: dbg and dbu come together");
    VQ_TRY(check_ld(call, "dH", dH, lddh, M));
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "Wg", Wg, ldw, N));
    VQ_TRY(check_ld(call, "Wu", Wu, ldw, N));
    VQ_TRY(check_ld(call, "G", G, ldz, M));
    VQ_TRY(check_ld(call, "U", U, ldz, M));
    VQ_TRY(check_ld(call, "dX", dX, lddx, N));
    VQ_TRY(check_ld(call, "dWg", dWg, lddw, N));
    VQ_TRY(check_ld(call, "dWu", dWu, lddw, N));
    VQ_TRY(check_ld(call, "dbg", dbg, M, M));
    VQ_TRY(check_ld(call, "dbu", dbu, M, M));
    VQ_TRY(check_apart(call, {dX, dWg, dWu, dbg, dbu}, {dH, X, Wg, Wu, G, U}));
    Backward b{T, M, N, dtype, act, 2, dH, lddh, X, ldx, {Wg, Wu}, ldw, {G, U}, ldz, dX, lddx, {dWg, dWu}, lddw, {dbg, dbu}};
    Arena a{nullptr};
    VQ_TRY(backward(b, a, false, as_stream(stream)));
    VQ_TRY(check_workspace(call, ws, ws_bytes, a.used));
    if (T > 0 || dWg || dbg) VQ_TRY(check_device());
    VQ_MATRIX(dH, T, M, lddh, call, "dH");
    if (dWg) VQ_MATRIX(X, T, N, ldx, call, "X");
    if (dX) VQ_MATRIX(Wg, M, N, ldw, call, "Wg");
    if (dX) VQ_MATRIX(Wu, M, N, ldw, call, "Wu");
    VQ_MATRIX(G, T, M, ldz, call, "G");
    VQ_MATRIX(U, T, M, ldz, call, "U");
    TimedRegion tr("gated_backward", 0, as_stream(stream));
    Arena w{static_cast<char*>(ws)};
    return backward(b, w, true, as_stream(stream));
}

}  // extern "C"
