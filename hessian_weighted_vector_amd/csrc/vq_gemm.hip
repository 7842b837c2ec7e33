// The tiled matrix product behind the dense feed-forward calls.
//
//   out[q, p] = sum_k P[p, k] Q[q, k],  bf16 or fp16 in, float32 sums.
//
// The loop is in vq_tile.h; here are the tile's epilogue, the split sums, the choice of
// tile and split, and dX and dW of a backward pass in one launch.
//
// What bounds it is the card's power: the pair of 28672 x 8192 by 4096 tokens takes
// 2.64 ms (1.46 PFLOP/s) with the matrix cores busy 0.80 of the cycles at 1.76 GHz, a
// gated backward pass of 2048 x 11008 x 4096 580 us (1.27 PFLOP/s; 0.67 at 1.95
// GHz, the transposing reads taking their share of LDS).  LDS has no bank conflicts
// and four of five L2 requests hit.  32 x 32 x 16 instructions were busier (0.79
// against 0.77) at a lower clock (1.57 GHz), 5 % slower; four waves of 128 x 128 moved
// sums between register files, 40 % slower.
#include "vq_tile.h"

#include <algorithm>

namespace vq {
namespace {

// One tile of one split of output `batch` of nbatch, from operands to stored outputs or parts.
template <class T, bool TRP, bool TRQ, int FP, int FQ, bool PAIR>
__device__ __forceinline__ void tile_product(const Tile& a, int id, int split, int batch, int nbatch, char* pb0, char* pb1,
                                             char* qb0, char* qb1)
{
    typedef Main<T, TRP, TRQ, FP, FQ, PAIR> L;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave / kWQ, wq = wave % kWQ;
    int tp, tq;
    pick_tile(id, a.ntp * a.ntq, a.ntp, a.ntq, tp, tq);
    const int p0 = tp * (PAIR ? L::BP / 2 : L::BP), q0 = tq * L::BQ;
    // splits in pairs of steps, as the loop takes them; past the last step come zeros
    const int pairs = (a.steps + 1) / 2;
    const int s0 = 2 * (int)((int64_t)pairs * split / a.splits), s1 = 2 * (int)((int64_t)pairs * (split + 1) / a.splits);

    f32x4 acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    L::run(a, p0, q0, batch, s0, s1, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);

    // lane l: output row l%16 of fragment j, features 4*(l/16) .. +3 of fragment i
    const int q_l = lane & 15, p_l = (lane >> 4) * 4;
    constexpr int NI = PAIR ? FP / 2 : FP;
    if (a.part) {
        const int64_t plane = (int64_t)a.nq * a.pitch;
        float* o = a.part + ((int64_t)split * (PAIR ? 2 : nbatch) + batch) * plane;
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            const int q = q0 + (wq * FQ + j) * 16 + q_l;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int p = p0 + (wp * NI + i) * 16 + p_l;
                if (q >= a.nq || p >= a.np) continue;
                *reinterpret_cast<f32x4*>(o + (int64_t)q * a.pitch + p) = acc[i][j];
                if (PAIR) *reinterpret_cast<f32x4*>(o + plane + (int64_t)q * a.pitch + p) = acc[i + NI][j];
            }
        }
        __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));          // no load into LDS outlives the workgroup
        return;
    }

    Epilogue e = a.epi;
    if (batch) e.Y = a.Y2;
    each_row<L>(acc, p0, q0, a.np, a.nq, wave, lane, pb0, pb1, qb0, qb1, [&](int q, int p, float (&v)[8], float (&u)[8]) {
        if (PAIR) epilogue_pair<T>(e, q, p, a.np, v, u);
        else epilogue_one<T>(e, q, p, a.np, v);
    });
}

template <class T, bool TRP, bool TRQ, int FP, int FQ, bool PAIR>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_gemm(const Tile a)
{
    typedef Main<T, TRP, TRQ, FP, FQ, PAIR> L;
    VQ_TILE_BUFFERS(L);
    tile_product<T, TRP, TRQ, FP, FQ, PAIR>(a, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z, pb0, pb1, qb0, qb1);
}

// Sums of the partial rows in 64 columns: a wave every eighth row, the waves' sums in
// wave order.  sh: 8 * 64 floats.
constexpr int kBiasColumns = 64;
template <class T>
__device__ __forceinline__ void bias_columns(const BiasSum& b, int id, float* sh)
{
    const int blocks = (b.M + kBiasColumns - 1) / kBiasColumns, o = id / blocks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = (id - o * blocks) * kBiasColumns + lane;
    const float* part = o ? b.part[1] : b.part[0];
    float s = 0.0f;
    if (m < b.M) {
#pragma unroll 8
        for (int64_t r = wave; r < b.n; r += kWaves) s += part[r * b.M + m];
    }
    sh[wave * 64 + lane] = s;
    __syncthreads();
    if (wave == 0 && m < b.M) {
        for (int k = 1; k < kWaves; ++k) s += sh[k * 64 + lane];
        static_cast<typename T::E*>(o ? b.db[1] : b.db[0])[m] = (typename T::E)s;
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_bias_sum(const BiasSum b)
{
    __shared__ float sh[kWaves * 64];
    bias_columns<T>(b, blockIdx.x, sh);
}

int bias_blocks(const BiasSum& b) { return (b.M + kBiasColumns - 1) / kBiasColumns * b.outputs; }

// dX and dW of a backward pass in one launch: the tiles of one fill the CUs that the
// other's last round would leave idle, and the bias gradients come last.
struct Two {
    Tile x, w;
    BiasSum bias;
    int nx, nw;                // workgroups
    int w_first, w_batch;      // whether dW's come first; its outputs
};

template <class T, int FP, int FQ>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_gemm_two(const Two a)
{
    typedef Main<T, true, true, FP, FQ, false> L;
    VQ_TILE_BUFFERS(L);
    const int id = blockIdx.x, first = a.w_first ? a.nw : a.nx;
    if (id >= a.nx + a.nw) {
        bias_columns<T>(a.bias, id - a.nx - a.nw, reinterpret_cast<float*>(pb0));
        return;
    }
    const int at = id < first ? id : id - first;
    if ((id < first) != (a.w_first != 0)) {
        const int tiles = a.x.ntp * a.x.ntq;
        tile_product<T, true, false, FP, FQ, false>(a.x, at % tiles, at / tiles, 0, 1, pb0, pb1, qb0, qb1);
    } else {
        const int tiles = a.w.ntp * a.w.ntq, batch = at / (tiles * a.w.splits), in = at - batch * tiles * a.w.splits;
        tile_product<T, true, true, FP, FQ, false>(a.w, in % tiles, in / tiles, batch, a.w_batch, pb0, pb1, qb0, qb1);
    }
}

// Adds the parts in order and applies the epilogue; eight features a thread.
// Not a pair: blockIdx.y is the output (Y[0] or Y[1]).
struct Finish {
    const float* part;         // [splits][outputs][nq][pitch]
    int splits, np, nq, pitch;
    Epilogue epi;
    void* Y2;
};

template <class T, bool PAIR>
__global__ __launch_bounds__(256) void k_gemm_finish(const Finish a)
{
    const int64_t per = a.pitch / 8;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= per * a.nq) return;
    const int64_t q = e / per;
    const int p = (int)(e - q * per) * 8;
    const int64_t plane = (int64_t)a.nq * a.pitch;
    const int b = blockIdx.y;
    const int nout = PAIR ? 2 : gridDim.y;
    const float* o = a.part + q * a.pitch + p + b * plane;
    float s[8] = {}, u[8] = {};
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {                      // four parts in flight
        const float* oz = o + (int64_t)z * nout * plane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(oz + h * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[h * 4 + i] += v[i];
            if (PAIR) {
                const f32x4 v2 = *reinterpret_cast<const f32x4*>(oz + plane + h * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) u[h * 4 + i] += v2[i];
            }
        }
    }
    if (PAIR) {
        epilogue_pair<T>(a.epi, q, p, a.np, s, u);
    } else {
        Epilogue ep = a.epi;
        if (b) ep.Y = a.Y2;
        epilogue_one<T>(ep, q, p, a.np, s);
    }
}

template <class T>
vq_status launch_finish(const Finish& f, bool pair, int nbatch, hipStream_t st)
{
    const dim3 grid(grid_for((int64_t)f.nq * (f.pitch / 8), 256), pair ? 1 : nbatch);
    if (pair) hipLaunchKernelGGL((k_gemm_finish<T, true>), grid, dim3(256), 0, st, f);
    else hipLaunchKernelGGL((k_gemm_finish<T, false>), grid, dim3(256), 0, st, f);
    VQ_LAUNCHED("k_gemm_finish");
    return VQ_OK;
}

// ---- plan ---------------------------------------------------------------
struct Plan {
    int fp, fq, ntp, ntq, splits, steps, seg_steps, pitch;
    size_t part_bytes;
    double cost;               // microseconds by the model (of two in one launch: of a tile)
};

// Tile and split by a model of the time in microseconds, fitted to 76 products
// of 64 to 28672 (mean loss against the best of all tiles and splits: 0.6 %).
// One 256 x 256 tile a CU: 1.45 a step, 10 a round for the epilogue and the
// pipeline's start.  128 x 128 tiles: 0.8 a step with one on a CU, 1.15 with two,
// 4 a round.  Split sums: 9.5 for the second launch and the parts' traffic.
// (2048 x 4096 x 11008: 156 us as 256 x 256 over two splits, 170 us as 128 x 128;
// 1024 x 2048 x 2048: 31 us and 19 us.)
Plan make_shape(GemmKind kind, int small, int64_t np, int64_t nq, int64_t K, int nseg)
{
    Plan p{};
    p.fp = small ? 4 : 8;
    p.fq = small ? 2 : 4;
    const int bp = kWP * p.fp * 16 / (kind == GEMM_GATED ? 2 : 1), bq = kWQ * p.fq * 16;
    p.ntp = (int)((np + bp - 1) / bp);
    p.ntq = (int)((nq + bq - 1) / bq);
    p.seg_steps = (int)((K + kBK - 1) / kBK);
    p.steps = p.seg_steps * nseg;
    p.pitch = (int)((np + 7) / 8 * 8);
    return p;
}

// A launch takes fewer than 2^32 threads; 256 x 256 tiles of what fits the memory stay below it.
constexpr int64_t kMostTiles = (int64_t)1 << 23;

size_t part_bytes(const Plan& p, int64_t nq, int nout)
{
    return p.splits > 1 ? align_up((size_t)p.splits * nout * nq * p.pitch * sizeof(float)) : 0;
}

Plan make_plan(GemmKind kind, int64_t np, int64_t nq, int64_t K, int nseg, int nbatch)
{
    const int nout = kind == GEMM_GATED ? 2 : nbatch;
    Plan best{};
    best.cost = 1e300;
    for (int small = 0; small < 2; ++small) {
        Plan p = make_shape(kind, small, np, nq, K, nseg);
        const int pairs = (p.steps + 1) / 2;
        if (small && (int64_t)p.ntp * p.ntq >= kMostTiles) continue;
        for (int sp = 1; sp <= 16 && sp <= pairs; ++sp) {
            const int64_t tiles = (int64_t)p.ntp * p.ntq * nbatch * sp;
            const double st = 2.0 * ((pairs + sp - 1) / sp);
            if (!small) {
                p.cost = (double)((tiles + 255) / 256) * (st * 1.45 + 10.0);
            } else {
                const int64_t rest = tiles % 512;
                p.cost = (double)(tiles / 512) * (st * 1.15 + 4.0) + (rest ? st * (rest <= 256 ? 0.8 : 1.15) + 4.0 : 0.0);
            }
            if (sp > 1) p.cost += 9.5 + 0.8e-6 * (double)np * nq * nout * (sp + 1);
            if (p.cost < best.cost) {
                best = p;
                best.splits = sp;
            }
        }
    }
    best.part_bytes = part_bytes(best, nq, nout);
    return best;
}

// Time until nl tiles of l microseconds and then ns of s <= l are done, each taken by
// the first free of `slots` places.
double fill_time(int64_t nl, double l, int64_t ns, double s, int slots)
{
    const int64_t rounds = nl / slots, late = nl % slots;       // `late` places start later by l
    const double t0 = (double)rounds * l;
    const double level = t0 + ((double)late * l + (double)ns * s) / slots;     // were tiles divisible
    double best = 1e300;
    for (int c = 0; c < 2; ++c) {                               // the last tile ends a place of either kind
        const double start = t0 + c * l;
        for (int64_t k = std::max<int64_t>(0, (int64_t)((level - start) / s)), n = 0; n < 4; ++k, ++n) {
            const double t = start + (double)k * s + 1e-9;
            const int64_t room = (int64_t)((t - t0) / s) * (slots - late) +
                                 (t >= t0 + l ? (int64_t)((t - t0 - l) / s) * late : 0);
            if (room >= ns && t < best) best = t;
        }
    }
    if (late && best < t0 + l) best = t0 + l;
    return best;
}

double split_cost(const Plan& p, int64_t np, int64_t nq, int nout)
{
    return p.splits > 1 ? 9.5 + 0.8e-6 * (double)np * nq * nout * (p.splits + 1) : 0.0;
}

// dX and dW together or apart, by the same model; apart costs 3 for its second launch.
// Fills both plans; whether together.
bool make_plans(const GemmSize& x, const GemmSize& w, Plan& px, Plan& pw)
{
    px = make_plan(x.kind, x.np, x.nq, x.K, x.nseg, x.nbatch);
    pw = make_plan(w.kind, w.np, w.nq, w.K, w.nseg, w.nbatch);
    double best = px.cost + pw.cost + 3.0;
    bool two = false;
    static const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
    for (int small = 0; small < 2; ++small) {
        Plan a = make_shape(x.kind, small, x.np, x.nq, x.K, x.nseg);
        Plan b = make_shape(w.kind, small, w.np, w.nq, w.K, w.nseg);
        const int64_t ta = (int64_t)a.ntp * a.ntq, tb = (int64_t)b.ntp * b.ntq * w.nbatch;
        const int slots = small ? 512 : 256;
        if (small && ta + tb >= kMostTiles - (1 << 20)) continue;     // the bias gradients' workgroups ride along
        for (int sa : kSplits) {
            if (sa > (a.steps + 1) / 2 || (sa > 1 && ta * sa > 2 * slots)) break;
            a.splits = sa;
            const double fa = split_cost(a, x.np, x.nq, 1);
            for (int sb : kSplits) {
                if (sb > (b.steps + 1) / 2 || (sb > 1 && tb * sb > 2 * slots)) break;
                b.splits = sb;
                const double per = small ? (ta * sa + tb * sb <= 256 ? 0.8 : 1.15) : 1.45, round = small ? 4.0 : 10.0;
                const double ca = 2.0 * (((a.steps + 1) / 2 + sa - 1) / sa) * per + round;
                const double cb = 2.0 * (((b.steps + 1) / 2 + sb - 1) / sb) * per + round;
                const double t = (ca >= cb ? fill_time(ta * sa, ca, tb * sb, cb, slots) : fill_time(tb * sb, cb, ta * sa, ca, slots)) +
                                 fa + split_cost(b, w.np, w.nq, w.nbatch);
                if (t < best) {
                    best = t;
                    two = true;
                    a.cost = ca; b.cost = cb;
                    px = a;
                    pw = b;
                }
            }
        }
    }
    if (two) {
        px.part_bytes = part_bytes(px, x.nq, 1);
        pw.part_bytes = part_bytes(pw, w.nq, w.nbatch);
    }
    return two;
}

template <class T, bool TRP, bool TRQ, bool PAIR, int FP, int FQ>
vq_status launch_shape(const Tile& t, const Plan& p, int nbatch, hipStream_t st)
{
    hipLaunchKernelGGL((k_gemm<T, TRP, TRQ, FP, FQ, PAIR>), dim3(p.ntp * p.ntq, p.splits, nbatch), dim3(kThreads), 0, st, t);
    VQ_LAUNCHED("k_gemm");
    if (p.splits > 1) VQ_TRY(launch_finish<T>({t.part, t.splits, t.np, t.nq, t.pitch, t.epi, t.Y2}, PAIR, nbatch, st));
    return VQ_OK;
}

template <class T, bool TRP, bool TRQ, bool PAIR>
vq_status launch_kind(const Tile& t, const Plan& p, int nbatch, hipStream_t st)
{
    if (p.fp == 8) return launch_shape<T, TRP, TRQ, PAIR, 8, 4>(t, p, nbatch, st);
    return launch_shape<T, TRP, TRQ, PAIR, 4, 2>(t, p, nbatch, st);
}

template <class T>
vq_status launch_type(GemmKind kind, const Tile& t, const Plan& p, int nbatch, hipStream_t st)
{
    switch (kind) {
    case GEMM_LINEAR: return launch_kind<T, false, false, false>(t, p, nbatch, st);
    case GEMM_GATED: return launch_kind<T, false, false, true>(t, p, nbatch, st);
    case GEMM_DX: return launch_kind<T, true, false, false>(t, p, nbatch, st);
    default: return launch_kind<T, true, true, false>(t, p, nbatch, st);
    }
}

}  // namespace

vq_status finish_parts(int dtype, bool pair, const float* part, int splits, int np, int nq, int pitch, const Epilogue& e,
                       hipStream_t st)
{
    const Finish f{part, splits, np, nq, pitch, e, nullptr};
    return dtype == VQ_BF16 ? launch_finish<Bf16>(f, pair, 1, st) : launch_finish<F16>(f, pair, 1, st);
}

size_t gemm_workspace(GemmKind kind, int64_t np, int64_t nq, int64_t K, int nseg, int nbatch)
{
    return make_plan(kind, np, nq, K, nseg, nbatch).part_bytes;
}

namespace {

// The kernel's arguments; parts from cv.
bool make_tile(const GemmArgs& g, const Plan& p, Carver& cv, Tile& t)
{
    t = Tile{};
    for (int i = 0; i < 2; ++i) {
        t.P[i] = static_cast<const char*>(g.P[i]);
        t.Q[i] = static_cast<const char*>(g.Q[i]);
    }
    t.ldp = (int)g.ldp; t.ldq = (int)g.ldq;
    t.kP = (int)g.kP; t.kQ = (int)g.kQ;
    t.np = g.np; t.nq = g.nq; t.wp = g.wp; t.wq = g.wq;
    t.ntp = p.ntp; t.ntq = p.ntq;
    t.seg_steps = p.seg_steps; t.steps = p.steps;
    t.splits = p.splits; t.pitch = p.pitch;
    t.epi = g.epi; t.Y2 = g.Y2;
    if (p.splits > 1) t.part = cv.take<float>(p.part_bytes / sizeof(float));
    return cv.ok;
}

GemmSize size_of(const GemmArgs& g) { return {g.kind, g.np, g.nq, std::min(g.kP, g.kQ), g.nseg, g.nbatch}; }

template <class T>
vq_status launch_two(const Two& a, const Plan& px, const Plan& pw, hipStream_t st)
{
    const int blocks = a.nx + a.nw + bias_blocks(a.bias);
    if (px.fp == 8) hipLaunchKernelGGL((k_gemm_two<T, 8, 4>), dim3(blocks), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_gemm_two<T, 4, 2>), dim3(blocks), dim3(kThreads), 0, st, a);
    VQ_LAUNCHED("k_gemm_two");
    if (px.splits > 1) VQ_TRY(launch_finish<T>({a.x.part, px.splits, a.x.np, a.x.nq, a.x.pitch, a.x.epi, nullptr}, false, 1, st));
    if (pw.splits > 1)
        VQ_TRY(launch_finish<T>({a.w.part, pw.splits, a.w.np, a.w.nq, a.w.pitch, a.w.epi, a.w.Y2}, false, a.w_batch, st));
    return VQ_OK;
}

}  // namespace

vq_status gemm_launch(const GemmArgs& g, void* ws, size_t ws_bytes, hipStream_t st)
{
    const GemmSize z = size_of(g);
    const Plan p = make_plan(z.kind, z.np, z.nq, z.K, z.nseg, z.nbatch);
    Carver cv(ws, ws_bytes);
    Tile t;
    if (!make_tile(g, p, cv, t)) return fail(VQ_ERR_WORKSPACE, "matrix product: workspace too small");
    return g.dtype == VQ_BF16 ? launch_type<Bf16>(g.kind, t, p, g.nbatch, st) : launch_type<F16>(g.kind, t, p, g.nbatch, st);
}

size_t gemm_two_workspace(const GemmSize& x, const GemmSize& w)
{
    Plan px, pw;
    return make_plans(x, w, px, pw) ? px.part_bytes + pw.part_bytes : std::max(px.part_bytes, pw.part_bytes);
}

vq_status bias_sum_launch(int dtype, const BiasSum& b, hipStream_t st)
{
    if (b.outputs == 0) return VQ_OK;
    if (dtype == VQ_BF16) hipLaunchKernelGGL((k_bias_sum<Bf16>), dim3(bias_blocks(b)), dim3(kThreads), 0, st, b);
    else hipLaunchKernelGGL((k_bias_sum<F16>), dim3(bias_blocks(b)), dim3(kThreads), 0, st, b);
    VQ_LAUNCHED("k_bias_sum");
    return VQ_OK;
}

vq_status gemm_two_launch(const GemmArgs& x, const GemmArgs& w, const BiasSum& b, void* ws, size_t ws_bytes, hipStream_t st)
{
    Plan px, pw;
    if (!make_plans(size_of(x), size_of(w), px, pw)) {          // one after the other, parts in the same place
        VQ_TRY(bias_sum_launch(x.dtype, b, st));
        VQ_TRY(gemm_launch(x, ws, ws_bytes, st));
        return gemm_launch(w, ws, ws_bytes, st);
    }
    Carver cv(ws, ws_bytes);
    Two a{};
    if (!make_tile(x, px, cv, a.x) || !make_tile(w, pw, cv, a.w))
        return fail(VQ_ERR_WORKSPACE, "matrix product: workspace too small");
    a.nx = px.ntp * px.ntq * px.splits;
    a.nw = pw.ntp * pw.ntq * pw.splits * w.nbatch;
    a.w_batch = w.nbatch;
    a.w_first = pw.cost > px.cost;
    a.bias = b;
    return x.dtype == VQ_BF16 ? launch_two<Bf16>(a, px, pw, st) : launch_two<F16>(a, px, pw, st);
}

}  // namespace vq
