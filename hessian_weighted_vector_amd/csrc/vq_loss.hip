// Softmax cross entropy over a large vocabulary, its logits never kept (vq_cross_entropy,
// vq_cross_entropy_backward).
//
//   z[t, v] = x_t . w_v,  lse_t = log sum_v exp z[t, v],  loss_t = lse_t - z[t, label_t]
//   dz[t, v] = dloss_t (exp(z[t, v] - lse_t) - [v = label_t]),  dX = dz W,  dW = dz^T X
//
//   k_loss_index    the tokens that are learnt, one behind the other, and their labels
//   k_loss_gather   their rows of X, 16-byte aligned (k_loss_index_gather: both, and the copied rows
//                   of W's first piece)
//   k_loss_logits   the tiled product z; a wave's tile leaves of each token the largest
//                   logit, the sum of exponentials below it, and the label's logit
//   k_loss_few      the same for few tokens, the vocabulary read straight from memory
//   k_loss_join     joins those pairs (m, s) in a fixed order: lse = m + log s
//   k_loss_rows     a token's loss from split sums of its logits, where tiles are too few to
//                   fill the card and N is split over workgroups; k_loss_dz: dz from them
//   k_loss_grad     the tiled product z again, for one piece of the vocabulary; dz from it
//   k_loss_two      the piece's rows of dW and its part of dX in one launch
//   k_loss_dx       dX from the sums, in the caller's order; zeros for the other tokens
//
// The forward pass reads X and W once a band of tiles and writes eight bytes a token and
// 64 or 128 words of the vocabulary; the logits stay in the accumulators.  The backward
// pass forms them again rather than keep them (6 T V N operations, 4 of them dX and dW)
// and takes the vocabulary in pieces whose dz stays small enough to be read back from
// the last-level cache.  dX is summed over the pieces in float32.
//
// Tokens whose label is ignore_index take no part: they are left out before the products
// (a training batch may be half prompt), so nothing that their rows of X hold reaches a
// result.  How many are left is known on the GPU alone: the grids are those of all
// tokens, and workgroups past the count end at once.
//
// The logits and the sums of exponentials are float32; dz is rounded to the tensors'
// type once, because the matrix cores read it in it.  Before, dloss is divided by its largest
// finite magnitude, and dX and dW are multiplied by it: where every token has one weight, 1 / n say, its
// rounding would otherwise be the same in every label's term, and the gradients' own (1 / 6927
// in bf16: all of them off by 0.0025).  In fp16 dz is also multiplied by 2^13, so that
// probabilities down to 2^-27 keep the type's full precision.
//
// What bounds it: power, as the dense products.  4096 tokens of 4096 by 131072 words, bf16, 3.04
// to 3.22 ms (1.37 to 1.45 PFLOP/s, matrix cores busy 0.78); the gradient of 2048 learnt tokens of
// 2048, eight pieces of 120 us for dz (busy 0.60: the exponentials and stores of a tile are not
// hidden) and 211 us for dX and dW (1.30 PFLOP/s).  One token by 32768 x 4096 50 us, bound by W's
// bytes.
#include "vq_few.h"
#include "vq_tile.h"

#include <algorithm>
#include <cmath>

namespace vq {
namespace {

constexpr int64_t kMaxLossTokens = 1 << 20;
constexpr int64_t kCountedTokens = 2048;        // up to which each token's workgroup counts its place
constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kPieceBytes = 128 << 20;      // of dz, or of a packed piece of W

// What the index kernel leaves in front of the workspace.
struct Head {
    int count;                   // tokens learnt
    float inverse;               // what dX and dW are multiplied by
};

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// (m, s) stands for s e^m.  Where every logit was -inf, m is -inf and s 0.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2)
{
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
    s = s * exp_of(m - base) + s2 * exp_of(m2 - base);
    m = top;
}

// The magnitude where it is finite.  A dloss that is not has no part in what all are divided by.
__device__ __forceinline__ float finite_size(float x)
{
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.0f;
}

struct Index {
    const int64_t* labels;
    int64_t T, V, ignore;
    Head* head;
    int* order;                  // token of each place
    int* label;                  // of each place; -1: outside the vocabulary
    // forward
    float* loss;                 // zeroed where ignored
    float* lse;
    // backward
    int* place;                  // of each token; -1: ignored
    const float* dloss;
    const float* lse_in;
    float* g;                    // dloss and lse of each place
    float* lse_at;
    float lift = 1.0f;           // dz's power of two
};

// One workgroup; a thread takes a run of consecutive tokens.
__global__ __launch_bounds__(1024) void k_loss_index(const Index a)
{
    __shared__ int sums[16];
    __shared__ float tops[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t per = (a.T + 1023) / 1024, t0 = threadIdx.x * per, t1 = t0 + per < a.T ? t0 + per : a.T;
    int n = 0;
    float top = 0.0f;
    for (int64_t t = t0; t < t1; ++t) {
        const bool on = a.labels[t] != a.ignore;
        n += on;
        if (a.g && on) top = fmaxf(top, finite_size(a.dloss[t]));
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
        top = fmaxf(top, __shfl_xor(top, o));
    }
    if (lane == 63) sums[wave] = upto;
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    int at = upto - n, all = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < wave) at += sums[w];
        all += sums[w];
        top = fmaxf(top, tops[w]);
    }
    if (top == 0.0f) top = 1.0f;
    if (threadIdx.x == 0) *a.head = Head{all, top / a.lift};
    for (int64_t t = t0; t < t1; ++t) {
        const int64_t l = a.labels[t];
        const bool on = l != a.ignore;
        if (a.place) a.place[t] = on ? at : -1;
        if (!on) {
            if (a.loss) a.loss[t] = a.lse[t] = 0.0f;
            continue;
        }
        const bool known = l >= 0 && l < a.V;
        a.order[at] = (int)t;
        a.label[at] = known ? (int)l : -1;
        if (a.g) {
            a.g[at] = known ? a.dloss[t] / top * a.lift : NAN;
            a.lse_at[at] = a.lse_in[t];
        }
        ++at;
    }
}

// A row into the learnt tokens' matrix; columns to its pitch are zeros.
__device__ __forceinline__ void gather_row(const Pack& m, int64_t from, int64_t to)
{
    const uint16_t* row = m.s + from * m.ld;
    uint16_t* o = m.o + to * m.ldp;
    for (int c = threadIdx.x * 8; c < m.ldp; c += 256 * 8) {
        alignas(16) uint16_t v[8];
        if (c + 8 <= m.cols) {
            if (m.odd) {
                Words w;
                w.load(row + c);
                const uint4 u = w.get(row + c);
                __builtin_memcpy(v, &u, 16);
            } else {
                __builtin_memcpy(v, row + c, 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < m.cols ? row[c + i] : (uint16_t)0;
        }
        *reinterpret_cast<uint4*>(o + c) = *reinterpret_cast<const uint4*>(v);
    }
}

__global__ __launch_bounds__(256) void k_loss_gather(const Head* head, const int* __restrict__ order, const Pack m)
{
    const int q = blockIdx.x;
    if (q < head->count) gather_row(m, order[q], q);
}

// Both at once for fewer tokens: a workgroup a token, which counts the learnt ones before it itself
// (1260 tokens: a launch and about 4 us less; at 4096 the counting costs as much).  Workgroups past
// the tokens copy the first piece of W, where its rows are copied.
__global__ __launch_bounds__(256) void k_loss_index_gather(const Index a, const Pack m, const Pack w, int wblocks)
{
    if ((int)blockIdx.x >= a.T) {
        pack_rows(w, (int)(blockIdx.x - a.T), wblocks);
        return;
    }
    __shared__ int counts[4];
    __shared__ float tops[4];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, last = (int)a.T - 1;
    const int64_t l = a.labels[t];
    const bool on = l != a.ignore;
    if (!on && threadIdx.x == 0) {
        if (a.place) a.place[t] = -1;
        if (a.loss) a.loss[t] = a.lse[t] = 0.0f;
    }
    if (!on && t != last) return;                             // the last token's workgroup knows them all
    int n = 0;
    float top = 0.0f;
    const int end = a.g ? (int)a.T : t;                       // the largest |dloss| is that of all
    for (int i = threadIdx.x; i < end; i += 256) {
        const bool learnt = a.labels[i] != a.ignore;
        n += learnt && i < t;
        if (a.g && learnt) top = fmaxf(top, finite_size(a.dloss[i]));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        n += __shfl_xor(n, o);
        top = fmaxf(top, __shfl_xor(top, o));
    }
    if (lane == 0) {
        counts[wave] = n;
        tops[wave] = top;
    }
    __syncthreads();
    const int at = counts[0] + counts[1] + counts[2] + counts[3];
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    if (top == 0.0f) top = 1.0f;
    if (threadIdx.x == 0) {
        if (t == last) *a.head = Head{at + on, top / a.lift};
        if (on) {
            const bool known = l >= 0 && l < a.V;
            if (a.place) a.place[t] = at;
            a.order[at] = t;
            a.label[at] = known ? (int)l : -1;
            if (a.g) {
                a.g[at] = known ? a.dloss[t] / top * a.lift : NAN;
                a.lse_at[at] = a.lse_in[t];
            }
        }
    }
    if (on) gather_row(m, t, at);
}

// The tiled product of a piece of W (rows v0 .. of the vocabulary) and the learnt tokens.
struct Logits {
    Tile t;                      // nq: all tokens
    const Head* head;
    const int* label;
    int v0;
    int turn;                    // workgroups begin at different steps
    // forward
    float2* part;                // [waves' columns of tiles][tokens]
    int64_t pitch;               // tokens a row of it
    float* picked;               // the labels' logits
    // split sums: [t.splits][tokens][t.pitch], or null
    float* sums;
    int64_t plane;
    // backward
    const float* lse;
    const float* g;
    void* dz;                    // [places][ldz], zeros past the piece
    int64_t ldz;
};

// The tile's sums; false where the grid's place holds none.  before(): what is to be under way
// while the product runs.
template <class L, class F>
__device__ __forceinline__ bool logits_tile(const Tile& full, int turn, int n, int& p0, int& q0, int& tp, int wave, int lane, char* pb0,
                                            char* pb1, char* qb0, char* qb1, f32x4 (&acc)[L::kFP][L::kFQ], F before)
{
    Tile t = full;
    t.nq = n;
    const int ntq = (n + L::BQ - 1) / L::BQ, tiles = t.ntp * ntq;
    if ((int)blockIdx.x >= tiles) return false;
    int tq;
    pick_tile(blockIdx.x, tiles, t.ntp, ntq, tp, tq);
    p0 = tp * L::BP;
    q0 = tq * L::BQ;
    before();
    const int pairs = (t.steps + 1) / 2;
    const int s0 = 2 * (int)((int64_t)pairs * blockIdx.y / t.splits);
    int s1 = 2 * (int)((int64_t)pairs * (blockIdx.y + 1) / t.splits);
#pragma unroll
    for (int i = 0; i < L::kFP; ++i)
#pragma unroll
        for (int j = 0; j < L::kFQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (L::kFP * L::kFQ < 32) {
        const int at = turn ? turned(s0, s1) : s0;
        if (at > s0) {
            L::run(t, p0, q0, 0, at, s1, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);
            run_again();
            s1 = at;
        }
    }
    L::run(t, p0, q0, 0, s0, s1, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);
    return true;
}

template <class T, int FP, int FQ>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_loss_logits(const Logits a)
{
    typedef Main<T, false, false, FP, FQ, false> L;
    VQ_TILE_BUFFERS(L);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave / kWQ, wq = wave % kWQ;
    const int n = a.head->count;
    int p0, q0, tp;
    f32x4 acc[FP][FQ];
    __shared__ int labels[L::BQ];
    const auto stage = [&] {
        for (int i = threadIdx.x; i < L::BQ; i += kThreads) labels[i] = a.label[q0 + i < n ? q0 + i : n - 1];
    };
    if (!logits_tile<L>(a.t, a.turn, n, p0, q0, tp, wave, lane, pb0, pb1, qb0, qb1, acc, stage)) return;
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));               // no load into LDS outlives the workgroup

    // lane l: token l%16 of fragment j, words 4*(l/16) .. +3 of fragment i
    const int first = p0 + wp * FP * 16, quad = lane >> 4;
    if (a.sums) {
        float* const o = a.sums + blockIdx.y * a.plane;
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            const int q = q0 + (wq * FQ + j) * 16 + (lane & 15);
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                const int p = first + i * 16 + quad * 4;
                if (q < n && p < a.t.np) *reinterpret_cast<f32x4*>(o + (int64_t)q * a.t.pitch + p) = acc[i][j];
            }
        }
        return;
    }
    if (first + FP * 16 > a.t.np) {
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (first + i * 16 + quad * 4 + r >= a.t.np)
#pragma unroll
                    for (int j = 0; j < FQ; ++j) acc[i][j][r] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
        const int q = q0 + (wq * FQ + j) * 16 + (lane & 15);
        const int want = q < n ? labels[q - q0] - a.v0 - first : -1;
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float base = m == -INFINITY ? 0.0f : m;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) s += exp_of(acc[i][j][r] - base);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (quad == 0 && q < n) a.part[(int64_t)(tp * kWP + wp) * a.pitch + q] = make_float2(m, s);
        if (want >= 0 && want < FP * 16 && (want >> 2 & 3) == quad) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) z = want == i * 16 + quad * 4 + r ? acc[i][j][r] : z;
            a.picked[q] = z;
        }
    }
}

template <class T, int FP, int FQ>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_loss_grad(const Logits a)
{
    typedef Main<T, false, false, FP, FQ, false> L;
    VQ_TILE_BUFFERS(L);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = a.head->count;
    int p0, q0, tp;
    f32x4 acc[FP][FQ];
    // a token's values: read in the epilogue, each row of a tile would wait for them
    __shared__ int labels[L::BQ];
    __shared__ float lses[L::BQ], gs[L::BQ];
    const auto stage = [&] {
        for (int i = threadIdx.x; i < L::BQ; i += kThreads) {
            const int q = q0 + i < n ? q0 + i : n - 1;
            labels[i] = a.label[q];
            lses[i] = a.lse[q];
            gs[i] = a.g[q];
        }
    };
    if (!logits_tile<L>(a.t, a.turn, n, p0, q0, tp, wave, lane, pb0, pb1, qb0, qb1, acc, stage)) return;
    each_row<L>(acc, p0, q0, (int)a.ldz, n, wave, lane, pb0, pb1, qb0, qb1, [&](int q, int p, float (&v)[8], float (&)[8]) {
        const float lse = lses[q - q0], g = gs[q - q0];
        const int want = labels[q - q0] - a.v0 - p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = exp_of(v[i] - lse);
            v[i] = p + i < a.t.np ? (i == want ? e - 1.0f : e) * g : 0.0f;
        }
        store8<T>(a.dz, a.ldz, q, p, (int)a.ldz, v);
    });
}

// The split sums of words p .. p+3 of a place, in order.
__device__ __forceinline__ f32x4 joined_sums(const float* sums, int splits, int64_t plane, int64_t at)
{
    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < splits; ++k) z += *reinterpret_cast<const f32x4*>(sums + k * plane + at);
    return z;
}

// A workgroup a token, of as many threads as its words keep busy.
struct RowLoss {
    const float* sums;
    int splits, pitch, V;
    int64_t plane;
    const Head* head;
    const int* order;
    const int* label;
    float* loss;
    float* lse;
};

__global__ __launch_bounds__(1024) void k_loss_rows(const RowLoss a)
{
    __shared__ float2 sh[16];
    const int q = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (q >= a.head->count) return;
    const int64_t row = (int64_t)q * a.pitch;
    const int want = a.label[q], t = a.order[q];
    const f32x4 zl = joined_sums(a.sums, a.splits, a.plane, row + (want < 0 ? 0 : want & ~3));       // the label's logit is among them
    float m = -INFINITY, s = 0.0f;
    // four chunks of words in flight: one by one, each would wait for memory
    constexpr int kAhead = 4;
    const int stride = (int)blockDim.x * 4;
    for (int p0 = threadIdx.x * 4; p0 < a.V; p0 += kAhead * stride) {
        const float* at[kAhead];
        f32x4 z[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            at[j] = a.sums + row + (p0 + j * stride < a.V ? p0 + j * stride : p0);
            z[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll 2
        for (int k = 0; k < a.splits; ++k)
#pragma unroll
            for (int j = 0; j < kAhead; ++j) z[j] += *reinterpret_cast<const f32x4*>(at[j] + k * a.plane);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int p = p0 + j * stride;
            if (p >= a.V) break;
            float top = z[j][0], sum = 0.0f;
#pragma unroll
            for (int i = 1; i < 4; ++i) top = p + i < a.V ? fmaxf(top, z[j][i]) : top;
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += p + i < a.V ? exp_of(z[j][i] - base) : 0.0f;
            join(m, s, top, sum);
        }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) join(m, s, __shfl_xor(m, o), __shfl_xor(s, o));
    if (lane == 0) sh[wave] = make_float2(m, s);
    __syncthreads();
    if (wave != 0) return;
    const bool in = lane < (int)blockDim.x >> 6;
    m = in ? sh[lane & 15].x : -INFINITY;
    s = in ? sh[lane & 15].y : 0.0f;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) join(m, s, __shfl_xor(m, o), __shfl_xor(s, o));
    if (lane != 0) return;
    const float lse = m + logf(s);
    a.loss[t] = want < 0 ? NAN : lse - (want & 2 ? (want & 1 ? zl[3] : zl[2]) : (want & 1 ? zl[1] : zl[0]));
    a.lse[t] = lse;
}

template <class T>
__global__ __launch_bounds__(256) void k_loss_dz(const Logits a, int64_t places)
{
    const int per = (int)(a.ldz / 8);
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, q = e / per;
    if (q >= places || q >= a.head->count) return;
    const int p = (int)(e - q * per) * 8;
    const float lse = a.lse[q], g = a.g[q];
    const int want = a.label[q] - a.v0 - p;
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x4 z = joined_sums(a.sums, a.t.splits, a.plane, q * a.t.pitch + p + h * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = exp_of(z[i] - lse);
            v[h * 4 + i] = p + h * 4 + i < a.t.np ? (h * 4 + i == want ? x - 1.0f : x) * g : 0.0f;
        }
    }
    store8<T>(a.dz, a.ldz, q, p, (int)a.ldz, v);
}

// Few tokens, as they come: KS waves take 16 RG rows of W together, blocks of 32 H columns in
// turn; a workgroup takes 64 rows where a wave takes 16 whole.  More than 16 tokens share their
// rows of X among RG groups of rows, which would read it RG times otherwise.  Where X fits (LDS),
// it is staged there: its reads do not queue with those of W.
struct FewLogits {
    const char* W;
    const char* X;
    int64_t ldw, ldx, K;
    int V, T;
    int ldl;                     // LDS: bytes of a staged row
    const int64_t* labels;
    float2* part;                // [workgroups][T]
    float* picked;
};

constexpr int kStaged = 40 << 10;            // bytes of X in LDS: three workgroups a CU

template <class T, int NT, int H, bool ODD, bool LDS, int KS, int RG>
__global__ __launch_bounds__(KS > 4 ? KS * 64 : 256) void k_loss_few(const FewLogits a)
{
    typedef typename T::E E;
    typedef typename T::V8 V8;
    constexpr int B = 32 * H;
    extern __shared__ __align__(16) char staged[];               // [T][ldl], zeros past K
    constexpr int kGroups = KS > 1 ? 1 : 4, kThreads = KS > 4 ? KS * 64 : 256;
    __shared__ float2 sh[kGroups][NT * 16];
    __shared__ f32x4 red[KS > 1 ? KS - 1 : 1][RG][NT][KS > 1 ? 64 : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, ks = wave % KS;
    const int m0 = (blockIdx.x * kGroups + wave / KS) * 16 * RG;
    const E* w[RG];
#pragma unroll
    for (int i = 0; i < RG; ++i) {
        const int64_t row = m0 + i * 16 + r < a.V ? m0 + i * 16 + r : a.V - 1;         // rows and tokens past the last repeat it
        w[i] = reinterpret_cast<const E*>(a.W) + row * a.ldw;
    }
    const E* x[NT];
    const char* xl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = n * 16 + r < a.T ? n * 16 + r : a.T - 1;
        x[n] = reinterpret_cast<const E*>(a.X) + t * a.ldx;
        xl[n] = staged + t * a.ldl + g * 16;
    }
    f32x4 acc[RG][NT];
#pragma unroll
    for (int i = 0; i < RG; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nfull = (int)(a.K / B);
    Ahead<T, ODD> wv[RG][H], xv[LDS ? 1 : NT][LDS ? 1 : H];
    const auto load = [&](int kb, int j) {
        const int64_t c = (int64_t)kb * B + j * 32 + g * 8;
        if (!LDS)
#pragma unroll
            for (int n = 0; n < NT; ++n) xv[n][j].load(x[n], c);
#pragma unroll
        for (int i = 0; i < RG; ++i) wv[i][j].load(w[i], c);
    };
    const auto multiply = [&](int kb, int j) {
        V8 wf[RG];
#pragma unroll
        for (int i = 0; i < RG; ++i) wf[i] = wv[i][j].get(w[i]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            V8 xf;
            if (LDS) xf = *reinterpret_cast<const V8*>(xl[n] + ((int64_t)kb * B + j * 32) * 2);
            else xf = xv[LDS ? 0 : n][LDS ? 0 : j].get(x[n]);
#pragma unroll
            for (int i = 0; i < RG; ++i) acc[i][n] = T::mfma(wf[i], xf, acc[i][n]);
        }
    };
    if (ks < nfull) {
#pragma unroll
        for (int j = 0; j < H; ++j) {
            load(ks, j);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (LDS) {
        for (int t = 0; t < a.T; ++t)
            for (int c = threadIdx.x * 8; c * 2 < a.ldl; c += kThreads * 8)
                *reinterpret_cast<V8*>(staged + t * a.ldl + c * 2) =
                    chunk_tail<T>(reinterpret_cast<const E*>(a.X) + t * a.ldx, c, a.K);
        __syncthreads();
    }
    if (ks < nfull) {
        int kb = ks;
#pragma unroll 1
        for (; kb + KS < nfull; kb += KS) {
#pragma unroll
            for (int j = 0; j < H; ++j) {
                multiply(kb, j);
                __builtin_amdgcn_sched_barrier(0);
                load(kb + KS, j);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < H; ++j) multiply(kb, j);
    }
    for (int64_t c0 = (int64_t)nfull * B + ks * 32; c0 < a.K; c0 += KS * 32) {
        const int64_t c = c0 + g * 8;
        V8 wf[RG];
#pragma unroll
        for (int i = 0; i < RG; ++i) wf[i] = chunk_tail<T>(w[i], c, a.K);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const V8 xf = LDS ? *reinterpret_cast<const V8*>(xl[n] + c0 * 2) : chunk_tail<T>(x[n], c, a.K);
#pragma unroll
            for (int i = 0; i < RG; ++i) acc[i][n] = T::mfma(wf[i], xf, acc[i][n]);
        }
    }
    if (KS > 1) {                                                // the first wave adds the others' sums in order
        if (ks > 0)
#pragma unroll
            for (int i = 0; i < RG; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) red[ks > 0 ? ks - 1 : 0][i][n][lane] = acc[i][n];
        __syncthreads();
        if (ks > 0) return;
#pragma unroll
        for (int i = 0; i < RG; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < KS - 1; ++k) acc[i][n] += red[k][i][n][lane];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = n * 16 + r;
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int j = 0; j < RG; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (m0 + j * 16 + g * 4 + i < a.V) m = fmaxf(m, acc[j][n][i]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < RG; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (m0 + j * 16 + g * 4 + i < a.V) s += exp_of(acc[j][n][i] - base);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (KS > 1) {
            if (g == 0 && t < a.T) a.part[(int64_t)blockIdx.x * a.T + t] = make_float2(m, s);
        } else if (g == 0) {
            sh[wave % kGroups][t] = make_float2(m, s);
        }
        if (t < a.T) {
            const int64_t want = a.labels[t] - m0 - g * 4;
#pragma unroll
            for (int j = 0; j < RG; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (want == j * 16 + i && m0 + j * 16 + g * 4 + i < a.V) a.picked[t] = acc[j][n][i];
        }
    }
    if (KS > 1) return;
    __syncthreads();
    const int t = threadIdx.x;
    if (t < a.T) {
        float m = sh[0][t].x, s = sh[0][t].y;
#pragma unroll
        for (int k = 1; k < kGroups; ++k) join(m, s, sh[k][t].x, sh[k][t].y);
        a.part[(int64_t)blockIdx.x * a.T + t] = make_float2(m, s);
    }
}

// K tokens a workgroup: 1024 / K threads join every so many-th part of a token, then a tree.
struct Join {
    const float2* part;
    int parts;
    int64_t pitch;
    const Head* head;            // or null: every token, ignored ones among them
    const int* order;
    const int64_t* labels;
    const float* picked;
    int64_t T, V, ignore;
    float* loss;
    float* lse;
};

template <int K>
__global__ __launch_bounds__(1024) void k_loss_join(const Join a)
{
    constexpr int S = 1024 / K;
    __shared__ float2 sh[S][K];
    const int n = a.head ? a.head->count : (int)a.T;
    const int k = threadIdx.x % K, slice = threadIdx.x / K;
    const int q = blockIdx.x * K + k;
    if ((int)blockIdx.x * K >= n) return;
    float m = -INFINITY, s = 0.0f;
    if (q < n) {
#pragma unroll 4
        for (int p = slice; p < a.parts; p += S) {
            const float2 v = a.part[(int64_t)p * a.pitch + q];
            join(m, s, v.x, v.y);
        }
    }
    sh[slice][k] = make_float2(m, s);
    __syncthreads();
#pragma unroll
    for (int h = S / 2; h > 0; h >>= 1) {
        if (slice < h) {
            const float2 v = sh[slice + h][k];
            join(m, s, v.x, v.y);
            sh[slice][k] = make_float2(m, s);
        }
        __syncthreads();
    }
    if (slice != 0 || q >= n) return;
    const int64_t t = a.head ? a.order[q] : q, label = a.labels[t];
    const float lse = m + logf(s);
    const bool on = label != a.ignore;
    a.lse[t] = on ? lse : 0.0f;
    a.loss[t] = !on ? 0.0f : label >= 0 && label < a.V ? lse - a.picked[q] : NAN;
}

// dX's sums and dW's rows of a piece.
struct Grads {
    Tile x, w;                   // nq of x, k of w: all tokens
    const Head* head;
    float* sums;                 // [splits of x][tokens][pitch]
    int64_t plane;
    int add;                     // to what the pieces before left there
    void* dW;                    // the piece's rows
    int64_t lddw;
    int with_x, with_w, w_first;
};

template <class T, int FP, int FQ>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_loss_two(const Grads a)
{
    typedef Main<T, true, false, FP, FQ, false> LX;
    typedef Main<T, true, true, FP, FQ, false> LW;
    VQ_TILE_BUFFERS(LW);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = a.head->count;
    const int ntq_x = (n + LX::BQ - 1) / LX::BQ, tiles_x = a.x.ntp * ntq_x;
    const int nx = a.with_x ? tiles_x * a.x.splits : 0, nw = a.with_w ? a.w.ntp * a.w.ntq : 0;
    const int id = blockIdx.x, first = a.w_first ? nw : nx;
    if (id >= nx + nw) return;
    const int at = id < first ? id : id - first;
    f32x4 acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int tp, tq;
    if ((id < first) != (a.w_first != 0)) {
        Tile t = a.x;
        t.nq = n;
        const int split = at / tiles_x, pairs = (t.steps + 1) / 2;
        pick_tile(at % tiles_x, tiles_x, t.ntp, ntq_x, tp, tq);
        const int p0 = tp * LX::BP, q0 = tq * LX::BQ;
        const int s0 = 2 * (int)((int64_t)pairs * split / t.splits), s1 = 2 * (int)((int64_t)pairs * (split + 1) / t.splits);
        LX::run(t, p0, q0, 0, s0, s1, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);
        float* const o = a.sums + split * a.plane;
        const int wp = wave / kWQ, wq = wave % kWQ;
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            const int q = q0 + (wq * FQ + j) * 16 + (lane & 15);
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                const int p = p0 + (wp * FP + i) * 16 + (lane >> 4) * 4;
                if (q >= n || p >= t.np) continue;
                f32x4* const at = reinterpret_cast<f32x4*>(o + (int64_t)q * t.pitch + p);
                if (a.add) acc[i][j] += *at;
                *at = acc[i][j];
            }
        }
        __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));           // no load into LDS outlives the workgroup
    } else {
        Tile t = a.w;
        t.kP = t.kQ = n;
        t.steps = t.seg_steps = (n + kBK - 1) / kBK;
        pick_tile(at, nw, t.ntp, t.ntq, tp, tq);
        const int p0 = tp * LW::BP, q0 = tq * LW::BQ;
        LW::run(t, p0, q0, 0, 0, (t.steps + 1) / 2 * 2, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);
        const float scale = a.head->inverse;
        each_row<LW>(acc, p0, q0, t.np, t.nq, wave, lane, pb0, pb1, qb0, qb1, [&](int q, int p, float (&v)[8], float (&)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= scale;
            store8<T>(a.dW, a.lddw, q, p, t.np, v);
        });
    }
}

// A token's row of dX: the sums' parts in order, eight columns a thread.
struct TokenGrads {
    const float* sums;
    int splits, pitch, N;
    int64_t plane, T, ldx;
    const Head* head;
    const int* place;
    void* dX;
};

// G lanes take every G-th part of eight columns and are added in a tree: many parts of few
// tokens are in flight together.
template <class T, int G>
__global__ __launch_bounds__(256) void k_loss_dx(const TokenGrads a)
{
    const int per = a.pitch / 8, lane = threadIdx.x & 63;
    constexpr int kChunks = 64 / G;                           // of a wave
    const int64_t e = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * kChunks + lane % kChunks;
    const bool in = e < per * a.T;
    const int64_t t = in ? e / per : 0;
    const int p = in ? (int)(e - t * per) * 8 : 0, q = in ? a.place[t] : -1;
    float s[8] = {};
    if (q >= 0) {
        const float* o = a.sums + (int64_t)q * a.pitch + p;
#pragma unroll 4
        for (int z = lane / kChunks; z < a.splits; z += G) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(o + z * a.plane + h * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[h * 4 + i] += v[i];
            }
        }
    }
#pragma unroll
    for (int o = kChunks; o < 64; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += __shfl_xor(s[i], o);
    if (!in || lane >= kChunks) return;
    const float scale = a.head->inverse;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= scale;
    store8<T>(a.dX, a.ldx, t, p, a.N, s);
}

template <class T>
void dx_launch(const TokenGrads& d, hipStream_t st)
{
    const int64_t n = d.T * (d.pitch / 8);
    if (d.splits > 4) hipLaunchKernelGGL((k_loss_dx<T, 8>), dim3((unsigned)((n + 31) / 32)), dim3(256), 0, st, d);
    else hipLaunchKernelGGL((k_loss_dx<T, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, d);
}

// ---- plan -------------------------------------------------------------------
// Tiles of 256 x 256 (one on a CU) or 128 x 128 (two), by the tiled products' model of
// microseconds: 1.45 a step and 10 a tile, or 0.8 (alone on a CU) and 1.15 and 4.
struct Shape {
    int small, bp, bq;
};
Shape shape(int small) { return {small, small ? 128 : 256, small ? 128 : 256}; }
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

double tiles_cost(int small, int64_t tiles, double steps)
{
    if (!small) return (double)up(tiles, 256) * (steps * 1.45 + 10.0);
    const int64_t rest = tiles % 512;
    return (double)(tiles / 512) * (steps * 1.15 + 4.0) + (rest ? steps * (rest <= 256 ? 0.8 : 1.15) + 4.0 : 0.0);
}

// The logits of V words: the shape, and over how many workgroups N is split where the tiles are few
// (one more launch where dz comes of it; the forward pass joins parts either way).
struct LogitsPlan {
    Shape s;
    int splits;
};
LogitsPlan logits_plan(int64_t V, int64_t T, int64_t N, bool backward)
{
    LogitsPlan best{};
    double least = 1e300;
    const int64_t pairs = up(up(N, kBK), 2);
    for (int small = 0; small < 2; ++small) {
        const Shape s = shape(small);
        const int64_t tiles = up(V, s.bp) * up(T, s.bq);
        for (int sp = 1; sp <= 16 && sp <= pairs; ++sp) {
            double t = tiles_cost(small, tiles * sp, 2.0 * up(pairs, sp));
            if (sp > 1) t += (backward ? 6.0 : 2.0) + 0.9e-6 * (double)T * V * (sp + 1);
            if (t < least) {
                least = t;
                best = {s, sp};
            }
        }
    }
    return best;
}

// Both gradients of a piece in one launch: the shape, and how many parts dX's sums are in.
struct GradPlan {
    Shape s;
    int splits, w_first;
};
GradPlan grad_plan(int64_t Vp, int64_t T, int64_t N, bool with_x, bool with_w)
{
    GradPlan best{};
    double least = 1e300;
    const int64_t px = up(up(Vp, kBK), 2);
    for (int small = 0; small < 2; ++small) {
        const Shape s = shape(small);
        const int slots = small ? 512 : 256;
        const double round = small ? 4.0 : 10.0;
        for (int sx = 1; sx <= 32 && sx <= px; ++sx) {
            // half of the tokens may be ignored, which leaves dX's tiles as long and half as many
            double sum = 0.0;
            int w_first = 0;
            for (int64_t n : {T, up(T, 2)}) {
                const int64_t tx = with_x ? up(N, s.bp) * up(n, s.bq) : 0, tw = with_w ? up(N, s.bp) * up(Vp, s.bq) : 0;
                const double per = small ? (tx * sx + tw <= 256 ? 0.8 : 1.15) : 1.45;
                const double cx = tx ? 2.0 * up(px, sx) * per + round : 0.0;
                const double cw = tw ? 2.0 * up(up(n, kBK), 2) * per + round : 0.0;
                // the longer ones first, the shorter ones fill the last round
                sum += std::max((cx * tx * sx + cw * tw) / slots + 0.5 * std::min(cx, cw), std::max(cx, cw));
                sum += 1.2e-6 * (double)n * N * (with_x ? sx : 0);
                w_first = cw > cx;
            }
            if (sum < least) {
                least = sum;
                best = {s, sx, w_first};
            }
            if (!with_x) break;
        }
    }
    return best;
}

// Words of a piece: a multiple of 256, pieces of nearly one size.
int64_t piece(int64_t V, int64_t bytes_a_word)
{
    const int64_t n = up(V * bytes_a_word, kPieceBytes);
    return std::min(up(up(V, n), 256) * 256, up(V, 8) * 8);
}

// Words of one launch: fewer than 2^32 threads also in small tiles.
int64_t most_words(int64_t T) { return ((int64_t)1 << 22) / up(T, 128) * 128; }

Tile tile_of(const void* P, int64_t ldp, int64_t kP, int64_t np, int64_t wp, const void* Q, int64_t ldq, int64_t kQ, int64_t nq,
             int64_t wq, const Shape& s)
{
    Tile t{};
    t.P[0] = t.P[1] = static_cast<const char*>(P);
    t.Q[0] = t.Q[1] = static_cast<const char*>(Q);
    t.ldp = (int)ldp; t.ldq = (int)ldq;
    t.kP = (int)kP; t.kQ = (int)kQ;
    t.np = (int)np; t.nq = (int)nq;
    t.wp = (int)wp; t.wq = (int)wq;
    t.ntp = (int)up(np, s.bp); t.ntq = (int)up(nq, s.bq);
    t.steps = t.seg_steps = (int)up(std::min(kP, kQ), kBK);
    t.splits = 1;
    return t;
}

struct Loss {
    int64_t T, V, N;
    int dtype;
    const void* X; int64_t ldx;
    const void* W; int64_t ldw;
    const int64_t* labels; int64_t ignore;
    // forward
    float* loss;
    float* lse;
    // backward
    const float* dloss;
    const float* lse_in;
    void* dX; int64_t lddx;
    void* dW; int64_t lddw;
};

// The learnt tokens' order, labels and rows of X, in the workspace.
struct Tokens {
    Head* head;
    int* order;
    int* label;
    uint16_t* x;
    int64_t ldx;
    void take(Arena& ws, const Loss& a)
    {
        ldx = round8(a.N);
        head = static_cast<Head*>(ws.take(sizeof(Head)));
        order = static_cast<int*>(ws.take(a.T * sizeof(int)));
        label = static_cast<int*>(ws.take(a.T * sizeof(int)));
        x = static_cast<uint16_t*>(ws.take(a.T * ldx * 2));
    }
    // Rows v0 .. v0 + n of W into `copy`.
    static Pack piece(const Loss& a, int64_t v0, int64_t n, uint16_t* copy)
    {
        const uint16_t* p = static_cast<const uint16_t*>(a.W) + v0 * a.ldw;
        return {p, copy, n, a.ldw, round8(a.N), (int)a.N, odd_rows(p, a.ldw)};
    }
    // Also the first n rows of W into `copy` (where there is one).
    vq_status launch(const Loss& a, Index ix, int64_t n, uint16_t* copy, hipStream_t st) const
    {
        ix.labels = a.labels;
        ix.T = a.T; ix.V = a.V; ix.ignore = a.ignore;
        ix.head = head; ix.order = order; ix.label = label;
        const Pack p{static_cast<const uint16_t*>(a.X), x, a.T, a.ldx, ldx, (int)a.N, odd_rows(a.X, a.ldx)};
        if (a.T <= kCountedTokens) {
            const int blocks = copy ? pack_blocks(n * (round8(a.N) / 8)) : 0;
            hipLaunchKernelGGL(k_loss_index_gather, dim3((unsigned)(a.T + blocks)), dim3(256), 0, st, ix, p,
                               copy ? piece(a, 0, n, copy) : Pack{}, blocks);
            VQ_LAUNCHED("k_loss_index_gather");
            return VQ_OK;
        }
        hipLaunchKernelGGL(k_loss_index, dim3(1), dim3(1024), 0, st, ix);
        VQ_LAUNCHED("k_loss_index");
        hipLaunchKernelGGL(k_loss_gather, dim3((unsigned)a.T), dim3(256), 0, st, head, order, p);
        VQ_LAUNCHED("k_loss_gather");
        return copy ? copy_piece(a, 0, n, copy, st) : VQ_OK;
    }
    static vq_status copy_piece(const Loss& a, int64_t v0, int64_t n, uint16_t* copy, hipStream_t st)
    {
        Packs k{};
        k.m[0] = piece(a, v0, n, copy);
        k.count = 1;
        k.blocks = pack_blocks(n * (round8(a.N) / 8));
        return pack_launch(k, st);
    }
};

// Rows v0 .. v0 + n of W as the tiles read them: in place, or copied to `copy` (the first piece
// has been).
vq_status words(const Loss& a, int64_t v0, int64_t n, uint16_t* copy, Mat& out, hipStream_t st)
{
    out = {static_cast<const uint16_t*>(a.W) + v0 * a.ldw, n, a.N, a.ldw};
    if (!copy) return VQ_OK;
    out = {copy, n, round8(a.N), round8(a.N)};
    return v0 > 0 ? Tokens::copy_piece(a, v0, n, copy, st) : VQ_OK;
}

// Whether the vocabulary is read for few tokens straight from memory: while the products stay below
// 1.6e9, and where tiles would need a copy of its rows.  Rows from memory, straight and in tiles: 131072 x
// 4096 by two tokens 174 and 183 us, by eight 212 and 183; 65536 x 4096 by four 99 and 106, by sixteen 125 and
// 106; 32768 x 4096 by nine 61 and 63, by 32 73 and 65; 32768 x 2048 by 32 40 and 41; 4096 x 4096 by 32 20
// and 24; 2048 x 8192 by sixteen 21 and 24, by 32 32 and 25; 17513 x 4570 by 32 86 and 100.
bool few(const Loss& a)
{
    if (a.T <= 2 || a.T > 32) return a.T <= 2;
    if (a.T > 16 && a.N > a.V) return false;
    return !loads_ok({a.W, a.V, a.N, a.ldw}) || (double)a.T * (double)a.V * (double)a.N < 1.6e9;
}

// Waves that share the rows of W.  One token, by one, four and sixteen: 32768 x 4096 64, 58 and 57 us,
// 32768 x 2048 32, 35 and 34, 2048 x 8192 35, 16 and 15, 8192 x 1024 11, 10 and 10; sixteen tokens by
// 16384 x 4096 38, 44 and 42, by 8192 x 4096 34, 22 and 22.  32 tokens by four waves, with one, two and
// four groups of rows: 4096 x 4096 19, 22 and 30, 8192 x 1024 13, 12 and 14, 32768 x 4096 113, 84 and 74.
struct FewPlan {
    int waves, rows;             // groups of 16 rows a wave; a workgroup takes four where its waves share none
    int parts(int64_t V) const { return (int)up(V, waves > 1 ? 16 * rows : 64 * rows); }
};
FewPlan few_plan(int64_t T, int64_t V, int64_t N)
{
    const int64_t groups = up(V, 16);
    if (T > 16) return {4, groups < 512 ? 1 : groups < 2048 ? 2 : 4};
    if (N < 512) return {1, 1};
    if (T > 8) return {groups >= 1024 ? 1 : 4, 1};
    return {N >= 4096 ? 16 : groups >= 2048 ? 1 : 4, 1};
}

template <class T, int NT, int H, bool LDS, int KS, int RG>
void few_launch(const FewLogits& f, bool odd, const FewPlan& p, hipStream_t st)
{
    const size_t lds = LDS ? (size_t)f.T * f.ldl : 0;
    const dim3 grid((unsigned)p.parts(f.V)), wg(KS > 4 ? KS * 64 : 256);
    if (odd) hipLaunchKernelGGL((k_loss_few<T, NT, H, true, LDS, KS, RG>), grid, wg, lds, st, f);
    else hipLaunchKernelGGL((k_loss_few<T, NT, H, false, LDS, KS, RG>), grid, wg, lds, st, f);
}

template <class T, int KS>
void few_tokens_launch(FewLogits f, bool odd, const FewPlan& p, hipStream_t st)
{
    constexpr int H = KS > 1 ? 4 : 8;
    f.ldl = (int)std::min<int64_t>(up(f.K, 32) * 64 + 16, 1 << 30);          // 16 more: rows in other banks
    if ((int64_t)f.T * f.ldl <= kStaged) few_launch<T, 1, H, true, KS, 1>(f, odd, p, st);
    else few_launch<T, 1, H, false, KS, 1>(f, odd, p, st);
}

template <class T>
void few_logits(const FewLogits& f, bool odd, const FewPlan& p, hipStream_t st)
{
    if (f.T > 16) {
        if (p.rows == 1) few_launch<T, 2, 4, false, 4, 1>(f, odd, p, st);
        else if (p.rows == 2) few_launch<T, 2, 4, false, 4, 2>(f, odd, p, st);
        else few_launch<T, 2, 2, false, 4, 4>(f, odd, p, st);
        return;
    }
    if (p.waves == 1) few_tokens_launch<T, 1>(f, odd, p, st);
    else if (p.waves == 4) few_tokens_launch<T, 4>(f, odd, p, st);
    else few_tokens_launch<T, 16>(f, odd, p, st);
}

// 64 tokens by 32768 x 4096, from memory, 80.4 us and 68.4 in turns, by 65536 x 4096 131 and 107; two rounds
// of tiles, 131072 x 4096, 188 and 209.
template <class T>
void logits_launch(Logits g, const Shape& s, bool backward, hipStream_t st)
{
    const dim3 grid((unsigned)(g.t.ntp * g.t.ntq), (unsigned)g.t.splits);
    g.turn = s.small && in_turn(g.t);
    if (g.sums) backward = false;                             // dz comes of the joined sums
    if (s.small) {
        if (backward) hipLaunchKernelGGL((k_loss_grad<T, 4, 2>), grid, dim3(kThreads), 0, st, g);
        else hipLaunchKernelGGL((k_loss_logits<T, 4, 2>), grid, dim3(kThreads), 0, st, g);
    } else {
        if (backward) hipLaunchKernelGGL((k_loss_grad<T, 8, 4>), grid, dim3(kThreads), 0, st, g);
        else hipLaunchKernelGGL((k_loss_logits<T, 8, 4>), grid, dim3(kThreads), 0, st, g);
    }
}

vq_status forward(const Loss& a, Arena& ws, bool run, hipStream_t st)
{
    if (a.T == 0) return VQ_OK;
    Join j{};
    j.labels = a.labels;
    j.T = a.T; j.V = a.V; j.ignore = a.ignore;
    j.loss = a.loss; j.lse = a.lse;
    j.pitch = a.T;
    if (few(a)) {
        const FewPlan plan = few_plan(a.T, a.V, a.N);
        j.parts = plan.parts(a.V);
        float2* part = static_cast<float2*>(ws.take(j.parts * a.T * sizeof(float2)));
        float* picked = static_cast<float*>(ws.take(a.T * sizeof(float)));
        if (!run) return VQ_OK;
        const FewLogits f{static_cast<const char*>(a.W), static_cast<const char*>(a.X), a.ldw, a.ldx, a.N, (int)a.V, (int)a.T, 0,
                          a.labels, part, picked};
        const bool odd = odd_rows(a.W, a.ldw) || odd_rows(a.X, a.ldx);
        if (a.dtype == VQ_BF16) few_logits<Bf16>(f, odd, plan, st);
        else few_logits<F16>(f, odd, plan, st);
        VQ_LAUNCHED("k_loss_few");
        j.part = part; j.picked = picked;
    } else {
        Tokens tk;
        tk.take(ws, a);
        const bool copied = !loads_ok({a.W, a.V, a.N, a.ldw});
        const int64_t Vp = copied ? std::min(piece(a.V, 2 * round8(a.N)), most_words(a.T)) : std::min(a.V, most_words(a.T));
        uint16_t* copy = copied ? static_cast<uint16_t*>(ws.take(Vp * round8(a.N) * 2)) : nullptr;
        const LogitsPlan plan = logits_plan(Vp, a.T, a.N, false);
        const Shape s = plan.s;
        const int per = kWP * (int)up(Vp, s.bp);              // parts of a piece
        const int64_t pitch = round8(a.V);
        float2* part = nullptr;
        float* picked = nullptr;
        float* sums = nullptr;
        if (plan.splits > 1) {
            sums = static_cast<float*>(ws.take(plan.splits * a.T * pitch * sizeof(float)));
        } else {
            for (int64_t v0 = 0; v0 < a.V; v0 += Vp) j.parts += kWP * (int)up(std::min(Vp, a.V - v0), s.bp);
            part = static_cast<float2*>(ws.take(j.parts * a.T * sizeof(float2)));
            picked = static_cast<float*>(ws.take(a.T * sizeof(float)));
        }
        if (!run) return VQ_OK;
        Index ix{};
        ix.loss = a.loss; ix.lse = a.lse;
        VQ_TRY(tk.launch(a, ix, std::min(Vp, a.V), copy, st));
        for (int64_t v0 = 0, k = 0; v0 < a.V; v0 += Vp, ++k) {
            const int64_t n = std::min(Vp, a.V - v0);
            Mat w;
            VQ_TRY(words(a, v0, n, copy, w, st));
            Logits g{};
            g.t = tile_of(w.p, w.ld, w.cols, n, 0, tk.x, tk.ldx, tk.ldx, a.T, 0, s);
            g.head = tk.head; g.label = tk.label;
            g.v0 = (int)v0;
            if (sums) {
                g.t.splits = plan.splits;
                g.t.pitch = (int)pitch;
                g.sums = sums + v0;
                g.plane = a.T * pitch;
            } else {
                g.part = part + k * per * a.T; g.pitch = a.T; g.picked = picked;
            }
            if (a.dtype == VQ_BF16) logits_launch<Bf16>(g, s, false, st);
            else logits_launch<F16>(g, s, false, st);
            VQ_LAUNCHED("k_loss_logits");
        }
        if (sums) {
            const RowLoss r{sums, plan.splits, (int)pitch, (int)a.V, a.T * pitch, tk.head, tk.order, tk.label, a.loss, a.lse};
            hipLaunchKernelGGL(k_loss_rows, dim3((unsigned)a.T), dim3(a.V > 4096 ? 1024 : 256), 0, st, r);
            VQ_LAUNCHED("k_loss_rows");
            return VQ_OK;
        }
        j.part = part; j.picked = picked;
        j.head = tk.head; j.order = tk.order;
    }
    // one token by 32768 x 4096 (2048 parts): the call takes 49.8 us, 53.5 with 64 threads a token; 48 and
    // 128 tokens by 131072 words 9.4 and 9.2 us with 256 threads a token, 11.9 and 11.0 with 64; 512 by 32000 4.9
    // and 5.4, 2048 by 131072 15.7 and 6.1
    if (few(a)) hipLaunchKernelGGL((k_loss_join<1>), dim3((unsigned)a.T), dim3(1024), 0, st, j);
    else if (a.T <= 128) hipLaunchKernelGGL((k_loss_join<4>), dim3((unsigned)up(a.T, 4)), dim3(1024), 0, st, j);
    else hipLaunchKernelGGL((k_loss_join<16>), dim3((unsigned)up(a.T, 16)), dim3(1024), 0, st, j);
    VQ_LAUNCHED("k_loss_join");
    return VQ_OK;
}

template <class T>
void grads_launch(const Grads& g, const GradPlan& p, hipStream_t st)
{
    const dim3 grid((unsigned)((g.with_x ? g.x.ntp * g.x.ntq * g.x.splits : 0) + (g.with_w ? g.w.ntp * g.w.ntq : 0)));
    if (p.s.small) hipLaunchKernelGGL((k_loss_two<T, 4, 2>), grid, dim3(kThreads), 0, st, g);
    else hipLaunchKernelGGL((k_loss_two<T, 8, 4>), grid, dim3(kThreads), 0, st, g);
}

template <class T>
vq_status piece_launch(const Logits& l, const Shape& s, const Grads& g, const GradPlan& plan, int64_t tokens, hipStream_t st)
{
    logits_launch<T>(l, s, true, st);
    VQ_LAUNCHED("k_loss_grad");
    if (l.sums) {
        hipLaunchKernelGGL((k_loss_dz<T>), dim3((unsigned)up(tokens * (l.ldz / 8), 256)), dim3(256), 0, st, l, tokens);
        VQ_LAUNCHED("k_loss_dz");
    }
    grads_launch<T>(g, plan, st);
    VQ_LAUNCHED("k_loss_two");
    return VQ_OK;
}

__global__ __launch_bounds__(256) void k_loss_zero(uint16_t* __restrict__ o, int64_t rows, int64_t cols, int64_t ld)
{
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * cols; e += (int64_t)gridDim.x * 256)
        o[e / cols * ld + e % cols] = 0;
}

vq_status backward(const Loss& a, Arena& ws, bool run, hipStream_t st)
{
    if (!a.dX && !a.dW) return VQ_OK;
    if (a.T == 0) {
        if (run && a.dW) {
            hipLaunchKernelGGL(k_loss_zero, dim3((unsigned)std::min<int64_t>(up(a.V * a.N, 256), 65536)), dim3(256), 0, st,
                               static_cast<uint16_t*>(a.dW), a.V, a.N, a.lddw);
            VQ_LAUNCHED("k_loss_zero");
        }
        return VQ_OK;
    }
    Tokens tk;
    tk.take(ws, a);
    int* place = static_cast<int*>(ws.take(a.T * sizeof(int)));
    float* g = static_cast<float*>(ws.take(a.T * sizeof(float)));
    float* lse = static_cast<float*>(ws.take(a.T * sizeof(float)));
    const int64_t N8 = round8(a.N);
    const bool copied = !loads_ok({a.W, a.V, a.N, a.ldw});
    const int64_t Vp = piece(a.V, 2 * (copied ? std::max(a.T, N8) : a.T));
    uint16_t* copy = copied ? static_cast<uint16_t*>(ws.take(Vp * N8 * 2)) : nullptr;
    void* dz = ws.take(a.T * Vp * 2);
    const GradPlan plan = grad_plan(std::min(Vp, a.V), a.T, a.N, a.dX, a.dW);
    float* sums = a.dX ? static_cast<float*>(ws.take(plan.splits * a.T * N8 * sizeof(float))) : nullptr;
    const LogitsPlan zplan = logits_plan(std::min(Vp, a.V), a.T, a.N, true);
    const int64_t zpitch = round8(std::min(Vp, a.V));
    float* zsums = zplan.splits > 1 ? static_cast<float*>(ws.take(zplan.splits * a.T * zpitch * sizeof(float))) : nullptr;
    if (!run) return VQ_OK;
    Index ix{};
    ix.place = place;
    ix.dloss = a.dloss; ix.lse_in = a.lse_in;
    ix.g = g; ix.lse_at = lse;
    ix.lift = a.dtype == VQ_F16 ? 0x1p13f : 1.0f;
    VQ_TRY(tk.launch(a, ix, std::min(Vp, a.V), copy, st));
    for (int64_t v0 = 0; v0 < a.V; v0 += Vp) {
        const int64_t n = std::min(Vp, a.V - v0), n8 = round8(n);
        Mat w;
        VQ_TRY(words(a, v0, n, copy, w, st));
        const Shape s = zplan.s;
        Logits l{};
        l.t = tile_of(w.p, w.ld, w.cols, n, 0, tk.x, tk.ldx, tk.ldx, a.T, 0, s);
        l.t.splits = zplan.splits;
        l.t.pitch = (int)zpitch;
        l.sums = zsums;
        l.plane = a.T * zpitch;
        l.head = tk.head; l.label = tk.label;
        l.v0 = (int)v0;
        l.lse = lse; l.g = g;
        l.dz = dz; l.ldz = n8;
        Grads b{};
        // dX: sum over the piece's words of W[word, column] dz[token, word]
        b.x = tile_of(w.p, w.ld, n, a.N, w.cols, dz, n8, n8, a.T, 0, plan.s);
        b.x.pitch = (int)N8;
        b.x.splits = std::min<int>(plan.splits, (b.x.steps + 1) / 2);
        // dW: sum over the tokens of X[token, column] dz[token, word]
        b.w = tile_of(tk.x, tk.ldx, a.T, a.N, tk.ldx, dz, n8, a.T, n, n8, plan.s);
        b.head = tk.head;
        b.sums = sums;
        b.plane = a.T * N8;
        b.add = v0 > 0;
        b.dW = a.dW ? static_cast<uint16_t*>(a.dW) + v0 * a.lddw : nullptr;
        b.lddw = a.lddw;
        b.with_x = a.dX != nullptr; b.with_w = a.dW != nullptr;
        b.w_first = plan.w_first;
        if (a.dtype == VQ_BF16) VQ_TRY(piece_launch<Bf16>(l, s, b, plan, a.T, st));
        else VQ_TRY(piece_launch<F16>(l, s, b, plan, a.T, st));
    }
    if (!a.dX) return VQ_OK;
    const TokenGrads d{sums, std::min<int>(plan.splits, (int)up(up(std::min(Vp, a.V), kBK), 2)), (int)N8, (int)a.N, a.T * N8, a.T,
                       a.lddx, tk.head, place, a.dX};
    if (a.dtype == VQ_BF16) dx_launch<Bf16>(d, st);
    else dx_launch<F16>(d, st);
    VQ_LAUNCHED("k_loss_dx");
    return VQ_OK;
}

vq_status check_sizes(const std::string& call, int64_t T, int64_t V, int64_t N, int dtype)
{
    VQ_CHECK(T >= 0 && T <= kMaxLossTokens, call + ": T must be in [0, 2^20]");
    VQ_CHECK(V >= 1 && V <= kMaxSize && N >= 1 && N <= kMaxSize, call + ": V and N must be in [1, 2^20]");
    VQ_CHECK(dtype == VQ_BF16 || dtype == VQ_F16, call + ": dtype must be VQ_BF16 or VQ_F16");
    return VQ_OK;
}

vq_status check_vector(const std::string& call, const char* what, const void* p, size_t align)
{
    VQ_CHECK(reinterpret_cast<uintptr_t>(p) % align == 0, call + ": " + what + " is not aligned to its elements");
    return VQ_OK;
}

}  // namespace
}  // namespace vq

using namespace vq;

extern "C" {

size_t vq_cross_entropy_workspace_bytes(int64_t T, int64_t V, int64_t N, const void* W, int64_t ldw)
{
    if (check_sizes("vq_cross_entropy", T, V, N, VQ_BF16) != VQ_OK) return 0;
    Loss a{};
    a.T = T; a.V = V; a.N = N;
    a.W = W; a.ldw = ldw;
    Arena ws{nullptr};
    return forward(a, ws, false, nullptr) == VQ_OK ? ws.used : 0;
}

vq_status vq_cross_entropy(int64_t T, int64_t V, int64_t N, int dtype, const void* X, int64_t ldx, const void* W, int64_t ldw,
                           const int64_t* labels, int64_t ignore_index, float* loss, float* lse, void* ws, size_t ws_bytes,
                           void* stream)
{
    const char* call = "vq_cross_entropy";
    VQ_TRY(check_sizes(call, T, V, N, dtype));
    if (T == 0) return VQ_OK;
    VQ_CHECK(X && W && labels && loss && lse, "vq_cross_entropy: null pointer");
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "W", W, ldw, N));
    VQ_TRY(check_vector(call, "labels", labels, 8));
    VQ_TRY(check_vector(call, "loss", loss, 4));
    VQ_TRY(check_vector(call, "lse", lse, 4));
    VQ_TRY(check_apart(call, {loss, lse}, {X, W, labels}));
    Loss a{};
    a.T = T; a.V = V; a.N = N; a.dtype = dtype;
    a.X = X; a.ldx = ldx; a.W = W; a.ldw = ldw;
    a.labels = labels; a.ignore = ignore_index;
    a.loss = loss; a.lse = lse;
    Arena count{nullptr};
    VQ_TRY(forward(a, count, false, as_stream(stream)));
    VQ_TRY(check_workspace(call, ws, ws_bytes, count.used));
    VQ_TRY(check_device());
    VQ_MATRIX(X, T, N, ldx, call, "X");
    VQ_MATRIX(W, V, N, ldw, call, "W");
    TimedRegion tr("cross_entropy", 0, as_stream(stream));
    Arena w{static_cast<char*>(ws)};
    return forward(a, w, true, as_stream(stream));
}

size_t vq_cross_entropy_backward_workspace_bytes(int64_t T, int64_t V, int64_t N, const void* W, int64_t ldw, int want_dx,
                                                 int want_dw)
{
    if (check_sizes("vq_cross_entropy_backward", T, V, N, VQ_BF16) != VQ_OK) return 0;
    void* const on = reinterpret_cast<void*>(uintptr_t(16));      // counted, never used
    Loss a{};
    a.T = T; a.V = V; a.N = N;
    a.W = W; a.ldw = ldw;
    a.dX = want_dx ? on : nullptr; a.dW = want_dw ? on : nullptr;
    Arena ws{nullptr};
    return backward(a, ws, false, nullptr) == VQ_OK ? ws.used : 0;
}

vq_status vq_cross_entropy_backward(int64_t T, int64_t V, int64_t N, int dtype, const float* dloss, const void* X, int64_t ldx,
                                    const void* W, int64_t ldw, const int64_t* labels, int64_t ignore_index, const float* lse,
                                    void* dX, int64_t lddx, void* dW, int64_t lddw, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_cross_entropy_backward";
    VQ_TRY(check_sizes(call, T, V, N, dtype));
    VQ_CHECK(T == 0 || (!dX && !dW) || (dloss && X && W && labels && lse), "vq_cross_entropy_backward: null pointer");
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "W", W, ldw, N));
    VQ_TRY(check_ld(call, "dX", dX, lddx, N));
    VQ_TRY(check_ld(call, "dW", dW, lddw, N));
    VQ_TRY(check_vector(call, "labels", labels, 8));
    VQ_TRY(check_vector(call, "dloss", dloss, 4));
    VQ_TRY(check_vector(call, "lse", lse, 4));
    VQ_TRY(check_apart(call, {dX, dW}, {X, W, labels, dloss, lse}));
    Loss a{};
    a.T = T; a.V = V; a.N = N; a.dtype = dtype;
    a.X = X; a.ldx = ldx; a.W = W; a.ldw = ldw;
    a.labels = labels; a.ignore = ignore_index;
    a.dloss = dloss; a.lse_in = lse;
    a.dX = dX; a.lddx = lddx; a.dW = dW; a.lddw = lddw;
    Arena count{nullptr};
    VQ_TRY(backward(a, count, false, as_stream(stream)));
    VQ_TRY(check_workspace(call, ws, ws_bytes, count.used));
    if ((T > 0 && dX) || dW) VQ_TRY(check_device());
    if (dX || dW) {
        VQ_VALUES(dloss, T, false, call, "dloss");
        VQ_VALUES(lse, T, false, call, "lse");
        VQ_MATRIX(X, T, N, ldx, call, "X");
        VQ_MATRIX(W, V, N, ldw, call, "W");
    }
    TimedRegion tr("cross_entropy_backward", 0, as_stream(stream));
    Arena w{static_cast<char*>(ws)};
    return backward(a, w, true, as_stream(stream));
}

}  // extern "C"
