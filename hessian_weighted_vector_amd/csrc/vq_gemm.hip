// The tiled matrix product behind the dense feed-forward calls.
//
//   out[q, p] = sum_k P[p, k] Q[q, k],  bf16 or fp16 in, float32 sums.
//
// A workgroup of eight waves owns a tile of BP features by BQ rows; a wave owns
// FP x FQ fragments of 16 x 16.  P fills the rows of the matrix instruction and
// Q its columns, so a lane ends with four consecutive features of one output
// row and stores them together.  A K step is 64 deep: both operands' slices go
// straight from memory into LDS (16 bytes a lane), double buffered.
//
// LDS layout.  A k-contiguous slice is [rows][64] (128 bytes a row, eight
// 16-byte chunks); chunk c of row r sits in slot c ^ (r & 7), so the eight rows
// that a fragment read touches at once are in different banks.  A k-strided
// slice is [64 k][BP] and is read through the transposing LDS read (a group of
// 16 lanes takes four k rows of 16 elements and each lane receives its
// element's column); chunk c of k row r sits in slot c ^ f(r) with f made of
// r's bits 0, 1 and 3, the bits in which the rows read together differ.  The
// swizzles are applied to the global addresses, since the direct loads fill
// LDS in lane order.
//
// Edges.  Loads go through buffer resources that end with the matrix, so rows
// and k beyond it read as zero; chunks beyond k of a k-contiguous row are
// pointed past the resource's end.
#include "vq_ffn.h"

namespace vq {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int kWP = 2, kWQ = 4;       // the waves' grid over the tile
constexpr int kBK = 64;               // k per step
constexpr uint32_t kOob = 0xC0000000u;     // past every resource's end
constexpr int64_t kMaxRecords = 0x7fffffff;

// Kernel arguments (one copy in the kernel's argument segment).
struct Tile {
    const char* P[2];
    const char* Q[2];
    float* part;               // [splits][outputs][nq][pitch] partial sums, or null
    int64_t ldp, ldq;
    int64_t kP, kQ;
    int np, nq, wp, wq;
    int ntp, ntq;              // tiles
    int seg_steps;             // K steps per segment
    int steps;                 // K steps in all
    int splits;
    int pitch;
    Epilogue epi;
    void* Y2;
};

typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ inline __amdgpu_buffer_rsrc_t resource(const char* base, int64_t bytes)
{
    const int64_t n = bytes < 0 ? 0 : (bytes > kMaxRecords ? kMaxRecords : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, (int)n, 0x00020000);
}

// Per-lane part of an operand's load addresses and its per-step resource.
// R: rows (of p or q) in the tile.  TR: k-strided.
template <int R, bool TR>
struct Slice {
    static constexpr int kBytes = R * kBK * 2;
    static constexpr int kLoads = kBytes / 1024;         // wave loads per slice
    static constexpr int kChunks = R / 8;                // 16-byte chunks of a k row (TR)
    static constexpr int kRowsPerLoad = TR ? 512 / R : 8;

    static __device__ inline int swizzle(int row)
    {
        return TR ? (2 * ((row & 3) | ((row >> 1) & 4))) & (kChunks - 1) : row & 7;
    }
};

// Loads `n` of the slice's wave loads (every kWaves-th from `wave`) into lds.
// k0: first k of the step within its segment.
template <int R, bool TR, bool PAIR>
__device__ inline void load_slice(const char* b0, const char* b1, int64_t ld, int row0, int nrows, int width, int64_t k0,
                                  int64_t K, char* lds, int wave, int lane)
{
    typedef Slice<R, TR> S;
    if (!TR) {
        const int rl = lane >> 3;
        const int chunk = (lane & 7) ^ rl;
        uint32_t v = (uint32_t)(rl * ld * 2 + chunk * 16);
        if (k0 + chunk * 8 >= K) v = kOob;
        const int64_t off = (int64_t)row0 * ld * 2;
        const int64_t bytes = ((int64_t)(nrows - row0 - 1) * ld + K) * 2;
        const __amdgpu_buffer_rsrc_t r0 = resource(b0 + off, bytes);
        const __amdgpu_buffer_rsrc_t r1 = PAIR ? resource(b1 + off, bytes) : r0;
#pragma unroll
        for (int j = 0; j < S::kLoads / kWaves; ++j) {
            const int inst = j * kWaves + wave;
            const bool second = PAIR && j >= S::kLoads / kWaves / 2;
            const int rows = (PAIR && second) ? inst * 8 - R / 2 : inst * 8;
            const uint32_t so = (uint32_t)(rows * ld * 2 + k0 * 2);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(second ? r1 : r0, (lds_ptr)(lds + inst * 1024), 16, v, so, 0, 0);
        }
    } else {
        const int rl = lane / S::kChunks;
        const __amdgpu_buffer_rsrc_t r0 =
            resource(b0 + (k0 * ld + row0) * 2, ((K - k0 - 1) * ld + (width - row0)) * 2);
#pragma unroll
        for (int j = 0; j < S::kLoads / kWaves; ++j) {
            const int inst = j * kWaves + wave;
            const int row = inst * S::kRowsPerLoad + rl;
            const int chunk = (lane % S::kChunks) ^ S::swizzle(row);
            const uint32_t v = (uint32_t)(rl * ld * 2 + chunk * 16);
            const uint32_t so = (uint32_t)(inst * S::kRowsPerLoad * ld * 2);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r0, (lds_ptr)(lds + inst * 1024), 16, v, so, 0, 0);
        }
    }
}

// Fragment (16 rows from r0, k = kk*32 .. +31): lane l holds row r0 + l%16,
// k = kk*32 + 8*(l/16) .. +7.
template <class T, int R, bool TR>
__device__ inline typename T::V8 fragment(char* lds, int r0, int kk, int lane)
{
    typedef Slice<R, TR> S;
    const int i = lane & 15, g = lane >> 4;
    if (!TR) {
        const int row = r0 + i;
        return *reinterpret_cast<const typename T::V8*>(lds + row * 128 + ((kk * 4 + g) ^ S::swizzle(row)) * 16);
    } else {
        const int row = kk * 32 + g * 8 + (i >> 2);          // second half: row + 4, same swizzle
        const int chunk = (r0 / 8 + ((i & 3) >> 1)) ^ S::swizzle(row);
        char* p = lds + row * (R * 2) + chunk * 16 + (i & 1) * 8;
        typedef __attribute__((address_space(3))) typename T::V4* tr_ptr;
        const typename T::V4 a = T::lds_tr((tr_ptr)p);
        const typename T::V4 b = T::lds_tr((tr_ptr)(p + 4 * R * 2));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}

// Work item -> tile.  Consecutive workgroup ids go to the eight dies in turn;
// each die takes a contiguous run of the tile order, and the order walks
// patches of four row tiles so that a die's concurrent tiles share operands in
// its L2.
__device__ inline void pick_tile(int id, int n, int ntp, int ntq, int& tp, int& tq)
{
    const int q = n / 8, r = n % 8, x = id % 8;
    const int t = x * q + (x < r ? x : r) + id / 8;
    constexpr int G = 4;
    const int band = t / (G * ntp);
    const int gq = ntq - band * G < G ? ntq - band * G : G;
    const int in = t - band * G * ntp;
    tp = in / gq;
    tq = band * G + in % gq;
}

// Floats per row of the epilogue's LDS tile: the pad spreads a column's rows over the banks.
constexpr int epilogue_pitch(int fp) { return fp * 16 + 4; }

template <class T, bool TRP, bool TRQ, int FP, int FQ, bool PAIR>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_gemm(const Tile a)
{
    constexpr int BP = kWP * FP * 16, BQ = kWQ * FQ * 16;
    constexpr int kBuf = (BP + BQ) * kBK * 2;
    extern __shared__ __align__(1024) char lds[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntiles = a.ntp * a.ntq;
    const int split = blockIdx.y;
    const int batch = blockIdx.z;
    int tp, tq;
    pick_tile(blockIdx.x, ntiles, a.ntp, a.ntq, tp, tq);
    const int p0 = tp * (PAIR ? BP / 2 : BP), q0 = tq * BQ;
    const int s0 = (int)((int64_t)a.steps * split / a.splits), s1 = (int)((int64_t)a.steps * (split + 1) / a.splits);

    const auto issue = [&](int s, int buf) {
        const int seg = s >= a.seg_steps ? 1 : 0;
        const int64_t k0 = (int64_t)(s - seg * a.seg_steps) * kBK;
        char* d = lds + buf * kBuf;
        load_slice<BP, TRP, PAIR>(PAIR ? a.P[0] : a.P[seg], a.P[1], a.ldp, p0, a.np, a.wp, k0, a.kP, d, wave, lane);
        load_slice<BQ, TRQ, false>(a.Q[seg + batch], nullptr, a.ldq, q0, a.nq, a.wq, k0, a.kQ, d + BP * kBK * 2, wave,
                                   lane);
    };

    f32x4 acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // rows of the tile that fragment i of this wave covers; in a pair the first
    // half of the fragments is the gate's, the second the same features of up
    const int wp = wave / kWQ, wq = wave % kWQ;
    const auto prow = [&](int i) {
        return PAIR ? (i < FP / 2 ? wp * (FP / 2) + i : FP + wp * (FP / 2) + i - FP / 2) * 16 : (wp * FP + i) * 16;
    };

    issue(s0, 0);
    for (int s = s0; s < s1; ++s) {
        const int buf = (s - s0) & 1;
        // this wave's loads of the step have landed, its reads of the other buffer are done
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        char* lp = lds + buf * kBuf;
        char* lq = lp + BP * kBK * 2;
        typename T::V8 fp[FP][2], fq[FQ][2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int i = 0; i < FP; ++i) fp[i][kk] = fragment<T, BP, TRP>(lp, prow(i), kk, lane);
#pragma unroll
            for (int j = 0; j < FQ; ++j) fq[j][kk] = fragment<T, BQ, TRQ>(lq, (wq * FQ + j) * 16, kk, lane);
        }
        if (s + 1 < s1) issue(s + 1, buf ^ 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) acc[i][j] = T::mfma(fp[i][kk], fq[j][kk], acc[i][j]);
    }

    // lane l: output row l%16 of fragment j, features 4*(l/16) .. +3 of fragment i
    const int q_l = lane & 15, p_l = (lane >> 4) * 4;
    constexpr int NI = PAIR ? FP / 2 : FP;
    if (a.part) {
        const int64_t plane = (int64_t)a.nq * a.pitch;
        float* o = a.part + ((int64_t)split * (PAIR ? 2 : gridDim.z) + batch) * plane;
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
        return;
    }

    // Epilogue: the wave turns two columns of fragments at a time around in its
    // own part of LDS, so that a lane holds eight consecutive features of a row
    // and a row's lanes write whole cache lines.
    Epilogue e = a.epi;
    if (batch) e.Y = a.Y2;
    constexpr int kPitch = epilogue_pitch(FP);
    constexpr int kLanes = NI * 2;                  // lanes per row
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    float* w = reinterpret_cast<float*>(lds) + wave * 32 * kPitch;
#pragma unroll
    for (int h = 0; h < FQ / 2; ++h) {
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int i = 0; i < FP; ++i)
                *reinterpret_cast<f32x4*>(w + (jj * 16 + q_l) * kPitch + i * 16 + p_l) = acc[i][h * 2 + jj];
#pragma unroll 1
        for (int r = 0; r < 32; r += 64 / kLanes) {
            const int row = r + lane / kLanes, c = (lane % kLanes) * 8;
            const int q = q0 + (wq * FQ + h * 2) * 16 + row;
            const int p = p0 + wp * NI * 16 + c;
            if (q < a.nq && p < a.np) {
                float v[8], u[8];
                const float* src = w + row * kPitch + c;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = src[i];
                if (PAIR) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = src[NI * 16 + i];
                    epilogue_pair<T>(e, q, p, a.np, v, u);
                } else {
                    epilogue_one<T>(e, q, p, a.np, v);
                }
            }
        }
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
    for (int z = 0; z < a.splits; ++z) {
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
};

Plan make_plan(GemmKind kind, int64_t np, int64_t nq, int64_t K, int nseg, int nbatch)
{
    const bool pair = kind == GEMM_GATED;
    Plan best{};
    double best_cost = 1e300;
    static const int shapes[][2] = {{8, 4}, {4, 2}};
    for (const auto& s : shapes) {
        Plan p;
        p.fp = s[0];
        p.fq = s[1];
        const int bp = kWP * p.fp * 16 / (pair ? 2 : 1), bq = kWQ * p.fq * 16;
        p.ntp = (int)((np + bp - 1) / bp);
        p.ntq = (int)((nq + bq - 1) / bq);
        p.seg_steps = (int)((K + kBK - 1) / kBK);
        p.steps = p.seg_steps * nseg;
        p.pitch = (int)((np + 7) / 8 * 8);
        const int64_t tiles = (int64_t)p.ntp * p.ntq * nbatch;
        for (int sp = 1; sp <= 16 && sp <= p.steps; ++sp) {
            // rounds of the chip, each as long as its share of K steps; a step of
            // the large tile costs four of the small one at twice the tiles per CU
            const double slots = p.fp == 8 ? 256.0 : 512.0;
            const double rounds = (double)((int64_t)((tiles * sp + slots - 1) / slots));
            double cost = rounds * ((p.steps + sp - 1) / sp + 6.0) * (p.fp == 8 ? 2.0 : 1.2);
            if (sp > 1) cost += 4.0 + (double)np * nq * (pair ? 2 : nbatch) * (sp + 1) * 4.0 / 4e6;
            if (cost < best_cost) {
                best_cost = cost;
                best = p;
                best.splits = sp;
            }
        }
    }
    const int nout = pair ? 2 : nbatch;
    best.part_bytes = best.splits > 1 ? align_up((size_t)best.splits * nout * nq * best.pitch * sizeof(float)) : 0;
    return best;
}

template <class T, bool TRP, bool TRQ, bool PAIR, int FP, int FQ>
vq_status launch_shape(const Tile& t, const Plan& p, int nbatch, hipStream_t st)
{
    constexpr size_t slices = 2 * (size_t)(kWP * FP + kWQ * FQ) * 16 * kBK * 2;
    constexpr size_t turned = (size_t)kWaves * 32 * epilogue_pitch(FP) * sizeof(float);
    constexpr size_t lds = slices > turned ? slices : turned;
    const auto kern = k_gemm<T, TRP, TRQ, FP, FQ, PAIR>;
    static thread_local int set_dev = -1;
    int dev = 0;
    VQ_HIP(hipGetDevice(&dev));
    if (lds > 65536 && set_dev != dev) {
        VQ_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)lds));
        set_dev = dev;
    }
    hipLaunchKernelGGL(kern, dim3(p.ntp * p.ntq, p.splits, nbatch), dim3(kThreads), lds, st, t);
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

vq_status gemm_launch(const GemmArgs& g, void* ws, size_t ws_bytes, hipStream_t st)
{
    const int64_t K = g.kP < g.kQ ? g.kP : g.kQ;
    const Plan p = make_plan(g.kind, g.np, g.nq, K, g.nseg, g.nbatch);
    Tile t{};
    for (int i = 0; i < 2; ++i) {
        t.P[i] = static_cast<const char*>(g.P[i]);
        t.Q[i] = static_cast<const char*>(g.Q[i]);
    }
    t.ldp = g.ldp; t.ldq = g.ldq;
    t.kP = g.kP; t.kQ = g.kQ;
    t.np = g.np; t.nq = g.nq; t.wp = g.wp; t.wq = g.wq;
    t.ntp = p.ntp; t.ntq = p.ntq;
    t.seg_steps = p.seg_steps; t.steps = p.steps;
    t.splits = p.splits; t.pitch = p.pitch;
    t.epi = g.epi; t.Y2 = g.Y2;
    set_vec(t.epi);
    t.epi.vec = t.epi.vec && vec8_ok(g.Y2, g.epi.ldy);
    if (p.splits > 1) {
        Carver cv(ws, ws_bytes);
        t.part = cv.take<float>(p.part_bytes / sizeof(float));
        if (!cv.ok) return fail(VQ_ERR_WORKSPACE, "matrix product: workspace too small");
    }
    return g.dtype == VQ_BF16 ? launch_type<Bf16>(g.kind, t, p, g.nbatch, st) : launch_type<F16>(g.kind, t, p, g.nbatch, st);
}

}  // namespace vq
