// The loop of the tiled matrix products: operands from memory through LDS into
// matrix-core fragments, and the sums' way back.
//
//   sum[q, p] = sum_k P[p, k] Q[q, k],  16-bit elements (or pairs of 8-bit ones) in,
//               32-bit sums.
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
#pragma once

#include "vq_ffn.h"

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
    if constexpr (!TR) {
        return *(const __attribute__((address_space(3))) typename T::V8*)(lds + (base ^ (kk * 64)) + i * 2048);
    } else {
        lds_ptr p = lds + (base ^ (i * 32)) + kk * 32 * R * 2;
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

// s_waitcnt with the given outstanding vector-memory and LDS counts.
constexpr int wait_imm(int vm, int lgkm) { return (vm & 15) | (vm >> 4) << 14 | 7 << 4 | lgkm << 8; }

template <class T, bool TRP, bool TRQ, int FP, int FQ, bool PAIR>
struct Main {
    typedef typename T::Acc Acc;                                 // four sums
    static constexpr int kFP = FP, kFQ = FQ;
    static constexpr bool kPair = PAIR;
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
                                               lds_ptr pb0, lds_ptr pb1, lds_ptr qb0, lds_ptr qb1, Acc (&acc)[FP][FQ])
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

// Few tokens against a matrix that is read once, by one round of workgroups (two small tiles a CU): all
// of them walk its rows in step and ask a few memory channels at a time.  They begin at one of eight
// places of their steps instead and come to the steps before it last.  The second start costs about as
// much as a step or two, so runs of less than 16 steps are left as they are.
__device__ __forceinline__ int turned(int s0, int s1)
{
    return s0 + 2 * ((s1 - s0) / 2 * (int)(((blockIdx.x + blockIdx.y * 3) / 8 + blockIdx.x) & 7) / 8);
}
inline bool in_turn(const Tile& t)
{
    return t.ntq == 1 && (int64_t)t.ntp * t.splits <= 512 && t.steps >= 16 * t.splits;
}

// Between two runs: every wave has read the buffers, and its last loads into them are there.
__device__ __forceinline__ void run_again()
{
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
    asm volatile("s_barrier" ::: "memory");
}

// The finished sums, eight consecutive features of a row at a time: f(q, p, v, u) for
// features p .. p+7 of output row q (u: the second matrix's, of a pair), rows and
// features past the last left out.  The wave turns two columns of fragments at a time
// around in its own part of LDS, so that a row's lanes write whole cache lines.
template <class L, class F>
__device__ __forceinline__ void each_row(const typename L::Acc (&acc)[L::kFP][L::kFQ], int p0, int q0, int np, int nq, int wave,
                                         int lane, char* pb0, char* pb1, char* qb0, char* qb1, F f)
{
    typedef typename L::Acc Acc;
    constexpr int FP = L::kFP, FQ = L::kFQ;
    constexpr bool PAIR = L::kPair;
    const int wp = wave / kWQ, wq = wave % kWQ;
    const int q_l = lane & 15;                      // lane l: output row l%16 of fragment j, features 4*(l/16) .. +3 of fragment i
    constexpr int NI = PAIR ? FP / 2 : FP;
    constexpr int kRow = FP * 16;                   // sums per row of the tile
    constexpr int kLanes = NI * 2;                  // lanes per row
    constexpr int kSmall = (L::BP < L::BQ ? L::BP : L::BQ) * kBK * 2;            // bytes of the smaller buffer
    constexpr int J = 2 * 32 * kRow * 4 <= kSmall ? 2 : 1;     // columns of fragments at a time: two waves a buffer
    static_assert(2 * J * 16 * kRow * 4 <= kSmall && FQ % J == 0, "two waves' tiles fit one operand buffer");
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));     // the last loads into LDS too
    asm volatile("s_barrier" ::: "memory");
    char* const w = (wave & 4 ? (wave & 2 ? qb1 : qb0) : (wave & 2 ? pb1 : pb0)) + (wave & 1) * J * 16 * kRow * 4;
    // 16-byte chunk c of row r sits in slot c ^ (r & 7)
    const auto at = [&](int row, int chunk) { return reinterpret_cast<Acc*>(w + row * kRow * 4 + (chunk ^ (row & 7)) * 16); };
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
            if (q < nq && p < np) {
                typedef decltype(Acc{}[0] + Acc{}[0]) S;
                const auto take = [&](int chunk, S (&v)[8]) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const Acc t = *at(row, chunk + k);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[k * 4 + i] = t[i];
                    }
                };
                S v[8], u[8];
                take(c, v);
                if (PAIR) take(NI * 4 + c, u);
                f(q, p, v, u);
            }
        }
    }
}

// The tile's operands in LDS, double buffered.  Four arrays, not one: the compiler
// then knows that a fragment is never read from a buffer that is being filled, and
// does not wait for those loads.
#define VQ_TILE_BUFFERS(L) \
    __shared__ __align__(1024) char pb0[L::BP * kBK * 2], pb1[L::BP * kBK * 2], qb0[L::BQ * kBK * 2], qb1[L::BQ * kBK * 2]

}  // namespace
}  // namespace vq
