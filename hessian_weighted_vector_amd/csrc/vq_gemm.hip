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
//
// What bounds it is the card's power: the pair of 28672 x 8192 by 4096 tokens takes
// 2.64 ms (1.46 PFLOP/s) with the matrix cores busy 0.80 of the cycles at 1.76 GHz, a
// gated backward pass of 2048 x 11008 x 4096 580 us (1.27 PFLOP/s; 0.67 at 1.95
// GHz, the transposing reads taking their share of LDS).  LDS has no bank conflicts
// and four of five L2 requests hit.  32 x 32 x 16 instructions were busier (0.79
// against 0.77) at a lower clock (1.57 GHz), 5 % slower; four waves of 128 x 128 moved
// sums between register files, 40 % slower.
#include "vq_ffn.h"

#include <algorithm>

namespace vq {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int kWP = 2, kWQ = 4;       // the waves' grid over the tile
constexpr int kBK = 64;               // k per step
constexpr uint32_t kOob = 0xC0000000u;     // past every resource's end

// Kernel arguments (one copy in the kernel's argument segment).
struct Tile {
    const char* P[2];
    const char* Q[2];
    float* part;               // [splits][outputs][nq][pitch] partial sums, or null
    int ldp, ldq;
    int kP, kQ;
    int np, nq, wp, wq;
    int ntp, ntq;              // tiles
    int seg_steps;             // K steps per segment
    int steps;                 // K steps in all
    int splits;
    int pitch;
    Epilogue epi;
    void* Y2;
};

typedef __attribute__((address_space(3))) char* lds_ptr;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const char* base, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bytes, 0x00020000);
}

// Per-lane part of an operand's load addresses and its per-step resource.
// R: rows (of p or q) in the tile.  TR: k-strided.
template <int R, bool TR>
struct Slice {
    static constexpr int kBytes = R * kBK * 2;
    static constexpr int kLoads = kBytes / 1024;         // wave loads per slice
    static constexpr int kChunks = R / 8;                // 16-byte chunks of a k row (TR)
    static constexpr int kRowsPerLoad = TR ? 512 / R : 8;

    static __device__ __forceinline__ int swizzle(int row)
    {
        return TR ? (2 * ((row & 3) | ((row >> 1) & 4))) & (kChunks - 1) : row & 7;
    }
};

// A wave's loads (every kWaves-th of the slice) of the step that starts at k0 of
// its segment.  Everything past the matrix, a k0 past K included, arrives as
// zeros.  Offsets and sizes fit 32 bits: a slice spans at most 256 rows of 2^21
// elements.
template <int R, bool TR, bool PAIR>
struct Loader {
    typedef Slice<R, TR> S;
    static constexpr int kCount = S::kLoads / kWaves;
    const char* b0;            // the matrix from the slice on (of a pair, both)
    const char* b1;
    int bytes;                 // to the slice's end
    uint32_t v;                // lane's offset
    int so, stride;            // the wave's first load, and from one to the next

    __device__ __forceinline__ Loader(const char* m0, const char* m1, int ld, int row0, int nrows, int width, int k0, int K,
                                      int wave, unsigned lane)
    {
        if (!TR) {
            const unsigned rl = lane >> 3, chunk = (lane & 7) ^ rl;
            v = rl * ld * 2 + chunk * 16;
            if (k0 + (int)chunk * 8 >= K) v = kOob;
            const int64_t off = (int64_t)row0 * ld * 2;
            const int rows = PAIR ? R / 2 : R;
            bytes = (((nrows - row0 < rows ? nrows - row0 : rows) - 1) * ld + K) * 2;
            b0 = m0 + off;
            b1 = PAIR ? m1 + off : b0;
            so = wave * 16 * ld + k0 * 2;
            stride = kWaves * 16 * ld;
        } else {
            // a wave's loads are a multiple of 16 k rows apart, which the swizzle does not see
            static_assert(kWaves * S::kRowsPerLoad % 16 == 0, "the loads of a wave share their swizzle");
            const unsigned rl = lane / S::kChunks;
            const unsigned chunk = (lane % S::kChunks) ^ S::swizzle(wave * S::kRowsPerLoad + rl);
            v = rl * ld * 2 + chunk * 16;
            const int rows = K - k0 < kBK ? K - k0 : kBK;
            bytes = rows <= 0 ? 0 : ((rows - 1) * ld + (width - row0)) * 2;
            b0 = b1 = m0 + ((int64_t)k0 * ld + row0) * 2;
            so = wave * S::kRowsPerLoad * 2 * ld;
            stride = kWaves * S::kRowsPerLoad * 2 * ld;
        }
    }
    // Load j into its place in the slice; the second half of a pair's rows come from the second matrix.
    __device__ __forceinline__ void issue(lds_ptr slice, int wave, int j) const
    {
        typedef __attribute__((address_space(3))) void* dst;
        const bool second = PAIR && j >= kCount / 2;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(second ? b1 : b0, bytes), (dst)(slice + (j * kWaves + wave) * 1024), 16, v,
                                                 so + (second ? j - kCount / 2 : j) * stride, 0, 0);
    }
};

// Fragment i (of the wave's rows from r0) of half kk: lane l holds row r0 + 16 i + l%16,
// k = kk*32 + 8*(l/16) .. +7.  lane_base is the lane's byte offset for i = kk = 0; the
// swizzles make the other fragments' offsets an exclusive or away from it.
template <int R, bool TR>
__device__ __forceinline__ uint32_t lane_base(int r0, int lane)
{
    typedef Slice<R, TR> S;
    const int i = lane & 15, g = lane >> 4;
    if (!TR) return (uint32_t)((r0 + i) * 128 + ((g ^ S::swizzle(i)) * 16));
    const int row = g * 8 + (i >> 2);                     // the read's second half: row + 4, same swizzle
    return (uint32_t)(row * (R * 2) + (((r0 / 8 + ((i & 3) >> 1)) ^ S::swizzle(row)) * 16) + (i & 1) * 8);
}

template <class T, int R, bool TR>
__device__ __forceinline__ typename T::V8 fragment(lds_ptr lds, uint32_t base, int i, int kk)
{
    if (!TR) return *(const __attribute__((address_space(3))) typename T::V8*)(lds + (base ^ (kk * 64)) + i * 2048);
    lds_ptr p = lds + (base ^ (i * 32)) + kk * 32 * R * 2;
    typedef __attribute__((address_space(3))) typename T::V4* tr_ptr;
    const typename T::V4 a = T::lds_tr((tr_ptr)p);
    const typename T::V4 b = T::lds_tr((tr_ptr)(p + 4 * R * 2));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
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

// s_waitcnt with the given outstanding vector-memory and LDS counts.
constexpr int wait_imm(int vm, int lgkm) { return (vm & 15) | (vm >> 4) << 14 | 7 << 4 | lgkm << 8; }

template <class T, bool TRP, bool TRQ, int FP, int FQ, bool PAIR>
struct Main {
    static constexpr int BP = kWP * FP * 16, BQ = kWQ * FQ * 16;
    static constexpr int kBuf = (BP + BQ) * kBK * 2;
    static constexpr int kLoads = kBuf / 1024 / kWaves;          // a wave's loads per step
    typedef typename T::V8 V8;
    struct Frags { V8 p[FP], q[FQ]; };

    // Fragment i of P starts at row (i + skip(i)) * 16 of the wave's first: in a
    // pair the first half of the fragments is the gate's, the second the same
    // features of up, half a tile further.
    static __device__ __forceinline__ int skip(int i) { return PAIR && i >= FP / 2 ? FP / 2 : 0; }

    // Steps s0 .. s1-1 (an even count) into acc.  A step is two halves of k = 32.  While the
    // matrix cores work on one half, the next half's fragments are read from LDS,
    // so a wave waits for LDS only at the start.  One barrier a step, between the
    // halves: behind it the next step's slices are complete (each wave has waited
    // for its own loads) and this step's buffer is free (its last fragments are
    // in registers), so the loads of the step after next go out.
    static __device__ __forceinline__ void run(const Tile& a, int p0, int q0, int batch, int s0, int s1, int wave, int lane,
                                               lds_ptr pb0, lds_ptr pb1, lds_ptr qb0, lds_ptr qb1, f32x4 (&acc)[FP][FQ])
    {
        const int wp = wave / kWQ, wq = wave % kWQ;
        // pointers in registers: one read in the loop would be awaited with the fragments
        const char* const P0 = a.P[0];
        const char* const P1 = a.P[1];
        const char* const Q0 = batch ? a.Q[1] : a.Q[0];
        const char* const Q1 = a.Q[1];
        typedef Loader<BP, TRP, PAIR> LoadP;
        typedef Loader<BQ, TRQ, false> LoadQ;
        static_assert(LoadP::kCount + LoadQ::kCount == FP && kLoads == FP, "one load beside each row of products");
        uint32_t pbase = lane_base<BP, TRP>(wp * (PAIR ? FP / 2 : FP) * 16, lane);
        uint32_t qbase = lane_base<BQ, TRQ>(wq * FQ * 16, lane);
        // Piece i of a half's fragments: one of P and one of Q while there are any.
        const auto read = [&](Frags& f, lds_ptr pb, lds_ptr qb, int kk, int i) __attribute__((always_inline)) {
            if (i < FQ) f.q[i] = fragment<T, BQ, TRQ>(qb, qbase, i, kk);
            f.p[i] = fragment<T, BP, TRP>(pb, pbase, i + skip(i), kk);
        };
        const auto multiply = [&](const Frags& f, int i) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < FQ; ++j) acc[i][j] = T::mfma(f.p[i], f.q[j], acc[i][j]);
        };
        // the lane's offsets are formed anew in each half: kept, they would take the registers of the sums
        const auto renew = [&] __attribute__((always_inline)) { asm volatile("" : "+v"(pbase), "+v"(qbase)); };
        Frags f0, f1;
        const auto step = [&](int s, lds_ptr pc, lds_ptr qc, lds_ptr pn, lds_ptr qn) __attribute__((always_inline)) {
            renew();
            unsigned l = lane;
            if (TRP || TRQ) asm volatile("" : "+v"(l));
            // a step past the last stays in the last segment, past its K
            const bool second = s + 2 >= a.seg_steps && a.steps > a.seg_steps;
            const int k0 = (second ? s + 2 - a.seg_steps : s + 2) * kBK;
            const LoadP lp(!PAIR && second ? P1 : P0, P1, a.ldp, p0, a.np, a.wp, k0, a.kP, wave, l);
            const LoadQ lq(second ? Q1 : Q0, nullptr, a.ldq, q0, a.nq, a.wq, k0, a.kQ, wave, l);
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                read(f1, pc, qc, 1, i);
                multiply(f0, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
            asm volatile("s_barrier" ::: "memory");
            renew();
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                read(f0, pn, qn, 0, i);
                if (i < LoadP::kCount) lp.issue(pc, wave, i);
                else lq.issue(qc, wave, i - LoadP::kCount);
                multiply(f1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        const auto issue = [&](int s, lds_ptr pb, lds_ptr qb) __attribute__((always_inline)) {
            const bool second = s >= a.seg_steps && a.steps > a.seg_steps;
            const int k0 = (second ? s - a.seg_steps : s) * kBK;
            const LoadP lp(!PAIR && second ? P1 : P0, P1, a.ldp, p0, a.np, a.wp, k0, a.kP, wave, lane);
            const LoadQ lq(second ? Q1 : Q0, nullptr, a.ldq, q0, a.nq, a.wq, k0, a.kQ, wave, lane);
#pragma unroll
            for (int j = 0; j < LoadP::kCount; ++j) lp.issue(pb, wave, j);
#pragma unroll
            for (int j = 0; j < LoadQ::kCount; ++j) lq.issue(qb, wave, j);
        };
        issue(s0, pb0, qb0);
        issue(s0 + 1, pb1, qb1);
        __builtin_amdgcn_s_waitcnt(wait_imm(kLoads, 0));
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int i = 0; i < FP; ++i) read(f0, pb0, qb0, 0, i);
        // loads past s1 go out too (zeros past the matrix): the body stays one block
#pragma unroll 1
        for (int s = s0; s < s1; s += 2) {
            step(s, pb0, qb0, pb1, qb1);
            step(s + 1, pb1, qb1, pb0, qb0);
        }
    }
};

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

    // Epilogue: the wave turns two columns of fragments at a time around in its
    // own part of LDS, so that a lane holds eight consecutive features of a row
    // and a row's lanes write whole cache lines.
    Epilogue e = a.epi;
    if (batch) e.Y = a.Y2;
    constexpr int kRow = FP * 16;                   // floats per row of the tile
    constexpr int kLanes = NI * 2;                  // lanes per row
    constexpr int kSmall = (L::BP < L::BQ ? L::BP : L::BQ) * kBK * 2;            // bytes of the smaller buffer
    constexpr int J = 2 * 32 * kRow * 4 <= kSmall ? 2 : 1;     // columns of fragments at a time: two waves a buffer
    static_assert(2 * J * 16 * kRow * 4 <= kSmall && FQ % J == 0, "two waves' tiles fit one operand buffer");
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));     // the last loads into LDS too
    asm volatile("s_barrier" ::: "memory");
    char* const w = (wave & 4 ? (wave & 2 ? qb1 : qb0) : (wave & 2 ? pb1 : pb0)) + (wave & 1) * J * 16 * kRow * 4;
    // 16-byte chunk c of row r sits in slot c ^ (r & 7)
    const auto at = [&](int row, int chunk) { return reinterpret_cast<f32x4*>(w + row * kRow * 4 + (chunk ^ (row & 7)) * 16); };
#pragma unroll
    for (int h = 0; h < FQ / J; ++h) {
#pragma unroll
        for (int jj = 0; jj < J; ++jj)
#pragma unroll
            for (int i = 0; i < FP; ++i) *at(jj * 16 + q_l, i * 4 + (lane >> 4)) = acc[i][h * J + jj];
#pragma unroll 1
        for (int r = 0; r < J * 16; r += 64 / kLanes) {
            const int row = r + lane / kLanes, c = (lane % kLanes) * 2;
            const int q = q0 + (wq * FQ + h * J) * 16 + row;
            const int p = p0 + wp * NI * 16 + c * 4;
            if (q < a.nq && p < a.np) {
                const auto take = [&](int chunk, float (&v)[8]) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const f32x4 t = *at(row, chunk + k);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[k * 4 + i] = t[i];
                    }
                };
                float v[8], u[8];
                take(c, v);
                if (PAIR) {
                    take(NI * 4 + c, u);
                    epilogue_pair<T>(e, q, p, a.np, v, u);
                } else {
                    epilogue_one<T>(e, q, p, a.np, v);
                }
            }
        }
    }
}

// The tile's operands in LDS, double buffered.  Four arrays, not one: the compiler
// then knows that a fragment is never read from a buffer that is being filled, and
// does not wait for those loads.
#define VQ_TILE_BUFFERS(L) \
    __shared__ __align__(1024) char pb0[L::BP * kBK * 2], pb1[L::BP * kBK * 2], qb0[L::BQ * kBK * 2], qb1[L::BQ * kBK * 2]

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
