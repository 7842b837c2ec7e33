// Feed-forward calls that read the compressed matrices, for few tokens:
//   vq_qlinear  Y = act(X W^T + bias) + R
//   vq_qgated   H = act(X Wg^T + bg) * (X Wu^T + bu), both matrices in one launch
// with W = decoded codebook rows, scaled, with the sparse correction; W is
// never written.
//
// The product runs on the matrix cores with exact operands.  A lane's share of
// a 16 x 16 x 32 instruction is eight consecutive k of one row, which is one
// sub-vector of d = 8 (two of d = 4; one of another length padded with zeros):
// the lane gathers its centroid row, adds the residual row, multiplies by the
// column scales and splits the float32 values into bf16 terms hi + lo (+
// lowest), each the rounding of what the terms before leave; the tokens are split
// alike (bf16 tokens are one term, fp16 two, float32 three, without a remainder).
// Of a value v the second term is at most 2^-8 v and the third 2^-17 v; two terms
// leave at most 2^-17 v, three nothing (24 bits).  With 16-bit tokens every
// product of a token's and a weight's terms is summed, in float32: what is missing
// is at most 2^-17 |w x|.  With float32 tokens the products of the second with the
// third terms and of the third terms are left out, at most 2^-23 |w x|.  Sixteen
// tokens cost the gathers of one.
//
// What bounds it is the requests from L1 to L2 that a CU keeps in flight: each
// sub-vector is one, to a random line, L2 hits of 237 cycles, and about 65 are in flight
// (0.28 a clock and CU; the L2 channels, 16 for a die of 32 CUs, take 0.56 of one each
// a clock).  So the tokens' terms and the column scales of a
// slab of columns are staged in LDS once a workgroup, indices are read 16 bytes
// (eight sub-vectors) a lane, a block ahead, and neighbouring lanes fetch the two
// halves of one centroid row in one instruction (one request, not two) and swap
// them.  4096 x 11008, one float32 token, all parts: 36 to 40 us; without residual,
// scales and exact entries 33, the gathers alone; a pair of 8192 x 2048, one
// token, 30 us; of 11008 x 4096, eight tokens, 95 us.  The body has one copy:
// unrolled over a block's groups it was 28 KB of code and its sums went through
// scratch memory, 14 to 20 % slower.  Seventeen to 32 float32 tokens still keep 11
// registers there (d = 8 and 4).
//
// A workgroup owns 16 rows; its waves (of a pair, the even ones gate and the odd
// ones up) take blocks of 32 sub-vectors in turn and their sums are added in wave
// order.  Where the rows alone leave CUs idle the
// blocks are split over workgroups too, and a second kernel adds the parts in
// order.  The sparse correction adds sum_e delta_e x[col_e] per row, delta
// being the exact value less the decoded weight, made once per matrix.
#include "vq_ffn.h"

#include <algorithm>
#include <cstring>
#include <string>

namespace vq {
namespace {

typedef Bf16::V8 V8;

constexpr int kQRows = 16;
constexpr int kBlock = 32;                 // sub-vectors of a row that a wave takes at a time
constexpr int kC2Floats = 2048;            // residual codebooks up to 8 KB are held in LDS
constexpr int kQTokens = 32;               // tokens per launch

struct QMat {
    const float* C1;
    const uint16_t* idx1;
    const float* C2;
    const uint16_t* idx2;
    const float* rs;
    const float* cs;
    const int32_t* row_ptr;
    const int32_t* col;
    const float* delta;
    int K1, K2;
};

struct QArgs {
    QMat q[2];
    int64_t M, N, nb;
    int d, T, nm, splits;
    int slab;                  // sub-vectors per slab, a multiple of kBlock
    const void* X;
    int64_t ldx;
    int dtype, act;
    const void* bias[2];
    const void* R;
    int64_t ldr;
    void* Y;
    int64_t ldy;
    float* part;               // [splits][matrices][T][M], or null
};

// kOrders: products of term p of a weight and term k of a token are summed for p + k below it.
template <int XT> struct XType;
template <> struct XType<VQ_BF16> { typedef __bf16 E; static constexpr int kTerms = 1, kWTerms = 2, kOrders = 2; };
template <> struct XType<VQ_F16> { typedef _Float16 E; static constexpr int kTerms = 2, kWTerms = 2, kOrders = 3; };
template <> struct XType<VQ_F32> { typedef float E; static constexpr int kTerms = 3, kWTerms = 3, kOrders = 3; };

__device__ inline int swap_pair(int v) { return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true); }
__device__ inline float swap_pair(float v) { return __int_as_float(swap_pair(__float_as_int(v))); }

// v = t[0] + t[1] + ... in bf16 terms, each rounded to nearest.  What a term leaves
// is exact, and formed by the two-element dot product, (t0, t1) . (-1, 0) + v0, which
// takes the packed terms as they are: 12 instructions a term and chunk, not 20.
template <int NTERM>
__device__ inline void split(const float (&v)[8], V8 (&t)[NTERM])
{
    typedef __bf16 V2 __attribute__((ext_vector_type(2)));
    // -1 in the low and in the high half, in registers: as a constant of the instruction
    // the compiler writes -1.0 for either, which is read as the high half's
    uint32_t low = 0x0000bf80u, high = 0xbf800000u;
    asm("" : "+s"(low), "+s"(high));
    const V2 first = __builtin_bit_cast(V2, low), second = __builtin_bit_cast(V2, high);
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
    for (int k = 0; k < NTERM; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[k][i] = (__bf16)rest[i];
        if (k + 1 == NTERM) break;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const V2 p = {t[k][i], t[k][i + 1]};
            rest[i] = __builtin_amdgcn_fdot2_f32_bf16(p, first, rest[i], false);
            rest[i + 1] = __builtin_amdgcn_fdot2_f32_bf16(p, second, rest[i + 1], false);
        }
    }
}

template <class E> __device__ inline float load_x(const void* p, int64_t i) { return (float)static_cast<const E*>(p)[i]; }

__device__ inline float load_any(const void* p, int64_t i, int dtype)
{
    return dtype == VQ_F32 ? load_x<float>(p, i) : dtype == VQ_BF16 ? load_x<__bf16>(p, i) : load_x<_Float16>(p, i);
}

__device__ inline void store_any(void* p, int64_t i, int dtype, float v)
{
    if (dtype == VQ_F32) static_cast<float*>(p)[i] = v;
    else if (dtype == VQ_BF16) static_cast<__bf16*>(p)[i] = (__bf16)v;
    else static_cast<_Float16*>(p)[i] = (_Float16)v;
}

// Eight indices from sub-vector s of a row of nb, as they are loaded ahead; past the
// row's end 0.  odd: whether some rows begin at an odd index.
__device__ inline void load_indices(const uint16_t* row, int64_t s, int64_t nb, bool odd, Words& k)
{
    if (s + 8 <= nb && !odd) {
        __builtin_memcpy(k.q, row + s, 16);
    } else if (s + 8 <= nb) {
        k.load(row + s);
    } else {
        uint16_t v[9] = {};                            // as Words: from the word that holds the first
        const bool from = odd && (reinterpret_cast<uintptr_t>(row) & 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t e = s + i < nb ? row[s + i] : (uint16_t)0;
            v[i] = from ? v[i] : e;
            v[i + 1] = from ? e : v[i + 1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) k.q[i] = v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
        k.last = v[8];
    }
}

// They, two to a register, at most top (two copies of K - 1).
__device__ inline void take_indices(const Words& w, const uint16_t* row, bool odd, uint32_t top, uint32_t (&k)[4])
{
    typedef uint16_t U2 __attribute__((ext_vector_type(2)));
    uint32_t v[4] = {w.q[0], w.q[1], w.q[2], w.q[3]};
    if (odd) {
        const uint4 u = w.get(row);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        k[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(U2, v[i]), __builtin_bit_cast(U2, top)));
}

// Index j of them.
__device__ inline uint32_t index_of(const uint32_t (&k)[4], int j) { return j & 1 ? k[j >> 1] >> 16 : k[j >> 1] & 0xffffu; }

// Elements 4 .. 7 of a row of d >= 4, zeros past it, from its last four.
__device__ inline void tail_of(const float (&last)[4], int d, float (&w)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = 0.0f;                              // element 4 + i is last[8 - d + i]
#pragma unroll
        for (int q = i; q < 4; ++q) v = q - i == 8 - d ? last[q] : v;
        w[4 + i] = v;
    }
}

// Row k of a codebook of any d <= 8, zero padded to eight: two (overlapping)
// four-element loads inside the row for d >= 4.
__device__ inline void load_row(const float* C, uint32_t k, int d, float (&w)[8])
{
    const float* row = C + k * (uint32_t)d;
    if (d >= 4) {
        float a[4], b[4];
        __builtin_memcpy(a, row, 16);
        __builtin_memcpy(b, row + d - 4, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = a[i];
        tail_of(b, d, w);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const float v = row[i < d ? i : d - 1];
            w[i] = i < d ? v : 0.0f;
        }
#pragma unroll
        for (int i = 3; i < 8; ++i) w[i] = 0.0f;
    }
}

// One sum from the definition, in plain float32.  Infinite values cannot be split
// (inf - inf), and inf times a term of zero is NaN, so a sum that comes out infinite
// or NaN is formed again by this: rare, so one lane takes a row (4096 x 11008, one
// token with an infinity in its last column, 2.9 ms).  An infinite token value meets an
// exact entry's whole weight, not the decoded one and the difference.  Finite calls pay
// for the test with 0 to 1 % (fp16, 17 to 32 tokens, 3 %).
template <class E>
__device__ inline float defined_sum(const QMat& q, const E* x, int64_t row, int64_t nb, int d)
{
    const int e0 = q.row_ptr ? q.row_ptr[row] : 0, e1 = q.row_ptr ? q.row_ptr[row + 1] : 0;
    const float rs = q.rs ? q.rs[row] : 1.0f;
    const int64_t N = nb * d;
    float s = 0.0f;
#pragma unroll 1
    for (int64_t b = 0; b < nb; ++b) {
        const uint32_t i1 = q.idx1[row * nb + b], i2 = q.C2 ? q.idx2[row * nb + b] : 0;
        const float* const c1 = q.C1 + (int64_t)min(i1, (uint32_t)q.K1 - 1) * d;
        const float* const c2 = q.C2 ? q.C2 + (int64_t)min(i2, (uint32_t)q.K2 - 1) * d : nullptr;
#pragma unroll 1
        for (int i = 0; i < d; ++i) {
            const int64_t j = b * d + i;
            float w = c2 ? c1[i] + c2[i] : c1[i];
            if (q.cs) w *= q.cs[j];
            w *= rs;
            const float v = (float)x[j];
            if (__builtin_isinf(v)) {
#pragma unroll 1
                for (int e = e0; e < e1; ++e)
                    if (q.col[e] == j) w += q.delta[e];
            }
            s += w * v;
        }
        if (__builtin_isnan(s)) return s;
    }
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
        const int64_t j = q.col[e];
        if (j < 0 || j >= N) continue;
        const float v = (float)x[j];
        if (__builtin_isfinite(v)) s += q.delta[e] * v;
    }
    return s;
}

// Columns of LDS per sub-vector: d = 8 and 4 as they are, others padded to eight.
__host__ __device__ constexpr int slots_of(int D) { return D ? D : 8; }
// Elements between tokens in LDS: 16 bytes past a multiple of 128, so that eight
// tokens' reads of one column are in different banks.
__host__ __device__ constexpr int token_pitch(int columns) { return columns + 8; }

// D = 8 or 4: sub-vectors of that length in 16-byte aligned codebooks (4: an even
// number of them in a row).  D = 0: any d, one sub-vector per chunk of eight k slots.
template <int D, int XT, int NT>
__global__ __launch_bounds__(1024) void k_qffn(const QArgs a)
{
    typedef typename XType<XT>::E E;
    constexpr int XTERMS = XType<XT>::kTerms, WTERMS = XType<XT>::kWTerms, ORDERS = XType<XT>::kOrders;
    constexpr int U = D == 4 ? 2 : 1;                  // sub-vectors per chunk
    constexpr int S = slots_of(D);
    constexpr int H = 2;                               // chunks whose gathers are in flight together
    extern __shared__ __align__(16) float lds[];
    const int d = D ? D : a.d;
    const int nm = a.nm;
    const int nthreads = blockDim.x, nwaves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * kQRows;
    const int64_t row = row0 + r < a.M ? row0 + r : a.M - 1;
    // this wave's matrix, its place among the matrix's waves and their number
    const int mm = nm > 1 ? wave & 1 : 0, turn = nm > 1 ? wave >> 1 : wave, turns = nm > 1 ? nwaves >> 1 : nwaves;

    // LDS: corrections [nm][NT * 16][16], residual codebooks (rows of S floats), column
    // scales [scaled][slab * S], token terms [XTERMS][T][pitch]; the sums' exchange takes
    // the last two's place
    const int columns = a.slab * S, pitch = token_pitch(columns);
    float* const cor = lds;
    int used = nm * NT * 16 * kQRows, cs_rows = 0;
    int c2_of[2] = {-1, -1}, cs_of[2] = {-1, -1};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (m >= nm) break;
        if (a.q[m].C2 && a.q[m].K2 * S <= kC2Floats) {
            c2_of[m] = used;
            used += a.q[m].K2 * S;
        }
        if (a.q[m].cs) cs_of[m] = cs_rows++ * columns;
    }
    const int c2_at = c2_of[mm], cs_at = cs_of[mm];
    float* const cs = lds + used;
    __bf16* const xs = reinterpret_cast<__bf16*>(cs + cs_rows * columns);
    const QMat q = a.q[mm];

    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Sparse corrections: a wave has one, two or four rows (16 of each matrix over its
    // waves) and gives each as many lanes; a row's lanes are tp tokens, times entries.
    const bool sparse = a.q[0].row_ptr || (nm > 1 && a.q[1].row_ptr);
    const int own = nm * kQRows / nwaves, per_row = 64 / own;
    int tp = 1;
    while (tp < a.T && tp < per_row) tp *= 2;
    const int sparse_id = lane / per_row * nwaves + wave;      // matrix * 16 + row

    const int nkb = (int)((a.nb + kBlock - 1) / kBlock);
    const int kb0 = (int)((int64_t)nkb * blockIdx.y / a.splits), kb1 = (int)((int64_t)nkb * (blockIdx.y + 1) / a.splits);
    const int slab_blocks = a.slab / kBlock;
    const uint32_t top1 = (uint32_t)(q.K1 - 1) * 0x10001u, top2 = q.C2 ? (uint32_t)(q.K2 - 1) * 0x10001u : 0;
    const bool odd1 = (reinterpret_cast<uintptr_t>(q.idx1) & 2) || (a.nb & 1);
    const bool odd2 = (reinterpret_cast<uintptr_t>(q.idx2) & 2) || (a.nb & 1);
    // d = 5 to 7: whether neighbouring lanes share rows (one request each, more
    // instructions).  One token by 4096 x 11010, d = 6, K1 = 65536: 48 us shared,
    // 52 not; two by 1133 x 14616, K1 = 197 (in L1): 28 and 26 us.
    const bool share = D == 0 && d >= 5 && q.K1 * d > 16384;
    Words i1, i2 = {};
    const auto load_block = [&](int kb) {
        const int64_t s = (int64_t)kb * kBlock + g * 8;
        load_indices(q.idx1 + row * a.nb, s, a.nb, odd1, i1);
        if (q.C2) load_indices(q.idx2 + row * a.nb, s, a.nb, odd2, i2);
    };

    const int item = threadIdx.x;
    int e0 = 0, e1 = 0;                                        // the lane's row's entries
    if (sparse) {
        const int64_t i = row0 + sparse_id % kQRows;
        const int32_t* rp = sparse_id < kQRows ? a.q[0].row_ptr : a.q[1].row_ptr;
        if (rp && i < a.M) {
            e0 = rp[i];
            e1 = rp[i + 1];
        }
    }
    f32x4 c2_v[2];                                             // D: at most one quad a thread
    if (D) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (c2_of[m] >= 0 && item < a.q[m].K2 * S / 4) c2_v[m] = reinterpret_cast<const f32x4*>(a.q[m].C2)[item];
    }

    for (int sb = kb0; sb < kb1; sb += slab_blocks) {
        const int se = sb + slab_blocks < kb1 ? sb + slab_blocks : kb1;
        const int64_t sv0 = (int64_t)sb * kBlock;
        const int cols = (se - sb) * kBlock * S;               // of this slab
        if (sb + turn < se) load_block(sb + turn);
        if (sb != kb0) __syncthreads();
        if (D) {
            // quads of column scales and chunks of eight columns of the tokens, two
            // of each a thread in flight; columns past the row are zeros
            const int quads = cs_rows ? cols / 4 : 0, per = cols / 8, total = per * a.T;
            constexpr int kFlight = 2;
            const int most = max(max(quads, total), nthreads);    // every thread passes once
            for (int i0 = item; i0 < most; i0 += nthreads * kFlight) {
                E e[kFlight][8];
                f32x4 c[2][kFlight];
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const int i = i0 + u * nthreads;
                    const int ix = i < total ? i : total - 1, t = ix / per;
                    const int64_t j = sv0 * d + (ix - t * per) * 8;
                    __builtin_memcpy(e[u], static_cast<const E*>(a.X) + t * a.ldx + (j < a.N ? j : a.N - 8), sizeof(e[u]));
                    const int64_t jc = sv0 * d + (i < quads ? i : 0) * 4;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        if (cs_of[m] >= 0) __builtin_memcpy(&c[m][u], a.q[m].cs + (jc < a.N ? jc : a.N - 4), 16);
                }
                if (sb == kb0 && i0 == item) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        if (c2_of[m] >= 0 && item < a.q[m].K2 * S / 4) reinterpret_cast<f32x4*>(lds + c2_of[m])[item] = c2_v[m];
                }
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const int i = i0 + u * nthreads;
                    if (i < total) {
                        const int t = i / per, cx = (i - t * per) * 8;
                        const bool in = sv0 * d + cx < a.N;
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = in ? (float)e[u][k] : 0.0f;
                        V8 w[XTERMS];
                        split<XTERMS>(v, w);
#pragma unroll
                        for (int k = 0; k < XTERMS; ++k) *reinterpret_cast<V8*>(xs + (k * a.T + t) * pitch + cx) = w[k];
                    }
                    if (i < quads) {
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            if (cs_of[m] >= 0) {
                                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                                *reinterpret_cast<f32x4*>(cs + cs_of[m] + i * 4) = sv0 * d + i * 4 < a.N ? c[m][u] : zero;
                            }
                    }
                }
            }
        } else {
            // column c of the slab: element c % 8 of sub-vector sv0 + c / 8; zero past the row and past d
            const auto source = [&](int c) -> int64_t {
                const int64_t sv = sv0 + c / S;
                const int e = c % S;
                return sv < a.nb && e < d ? sv * d + e : -1;
            };
            for (int m = 0; m < nm; ++m) {
                if (c2_of[m] >= 0 && sb == kb0)
                    for (int i = item; i < a.q[m].K2 * S; i += nthreads)
                        lds[c2_of[m] + i] = i % S < d ? a.q[m].C2[i / S * d + i % S] : 0.0f;
                if (cs_of[m] >= 0)
                    for (int c = item; c < cols; c += nthreads) {
                        const int64_t j = source(c);
                        cs[cs_of[m] + c] = j >= 0 ? a.q[m].cs[j] : 0.0f;
                    }
            }
            const int per = cols / 8, total = per * a.T;
            for (int i = item; i < total; i += nthreads) {
                const int t = i / per, c = (i - t * per) * 8;
                const E* x = static_cast<const E*>(a.X) + t * a.ldx;
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int64_t j = source(c + k);
                    const float f = (float)x[j >= 0 ? j : 0];
                    v[k] = j >= 0 ? f : 0.0f;
                }
                V8 w[XTERMS];
                split<XTERMS>(v, w);
#pragma unroll
                for (int k = 0; k < XTERMS; ++k) *reinterpret_cast<V8*>(xs + (k * a.T + t) * pitch + c) = w[k];
            }
        }
        __syncthreads();

#pragma unroll 1
        for (int kb = sb + turn; kb < se; kb += turns) {
            uint32_t k1[4], k2[4];
            take_indices(i1, q.idx1 + row * a.nb, odd1, top1, k1);       // blocks keep the row's parity
            take_indices(i2, q.idx2 + row * a.nb, odd2, top2, k2);
            if (kb + turns < se) load_block(kb + turns);
            int c0 = ((kb - sb) * kBlock + g * 8) * S;         // the lane's first column in the slab
#pragma unroll 1
            for (int h = 0; h < 8 / U / H; ++h) {              // one copy of the body: the code stays in its cache
                float w[H][8];
                if (D == 8) {
                    const f32x4* C = reinterpret_cast<const f32x4*>(q.C1);
                    const int odd = lane & 1;
                    f32x4 ga[H], gb[H];
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const int mine = index_of(k1, j), other = swap_pair(mine);
                        ga[j] = C[2 * (odd ? other : mine) + odd];
                        gb[j] = C[2 * (odd ? mine : other) + odd];
                    }
#pragma unroll
                    for (int j = 0; j < H; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float other = swap_pair(odd ? ga[j][i] : gb[j][i]);
                            w[j][i] = odd ? other : ga[j][i];
                            w[j][4 + i] = odd ? gb[j][i] : other;
                        }
                } else if (D == 4) {
                    const f32x4* C = reinterpret_cast<const f32x4*>(q.C1);
#pragma unroll
                    for (int j = 0; j < H; ++j)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const f32x4 v = C[index_of(k1, j * 2 + u)];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[j][u * 4 + i] = v[i];
                        }
                } else if (share) {
                    // as with d = 8, by the row's first and last four elements
                    const int odd = lane & 1;
                    float ga[H][4], gb[H][4];
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const int mine = index_of(k1, j), other = swap_pair(mine);
                        __builtin_memcpy(ga[j], q.C1 + (uint32_t)((odd ? other : mine) * d + odd * (d - 4)), 16);
                        __builtin_memcpy(gb[j], q.C1 + (uint32_t)((odd ? mine : other) * d + odd * (d - 4)), 16);
                    }
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        float last[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float other = swap_pair(odd ? ga[j][i] : gb[j][i]);
                            w[j][i] = odd ? other : ga[j][i];
                            last[i] = odd ? gb[j][i] : other;
                        }
                        tail_of(last, d, w[j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < H; ++j) load_row(q.C1, index_of(k1, j), d, w[j]);
                }
                if (q.C2) {
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        if (D == 0 && c2_at < 0) {
                            float v[8];
                            load_row(q.C2, index_of(k2, j), d, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[j][i] += v[i];
                        } else {
                            const float* c2 = c2_at >= 0 ? lds + c2_at : q.C2;
#pragma unroll
                            for (int u = 0; u < 2; ++u) {        // halves of one row, or two rows
                                const int k = index_of(k2, j * U + (D == 4 ? u : 0));
                                const f32x4 v = *reinterpret_cast<const f32x4*>(c2 + k * S + (D == 4 ? 0 : u * 4));
#pragma unroll
                                for (int i = 0; i < 4; ++i) w[j][u * 4 + i] += v[i];
                            }
                        }
                    }
                }
                if (cs_at >= 0) {
#pragma unroll
                    for (int j = 0; j < H; ++j)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const f32x4 v = *reinterpret_cast<const f32x4*>(cs + cs_at + c0 + j * 8 + u * 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[j][u * 4 + i] *= v[i];
                        }
                }
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    V8 wt[WTERMS];
                    split<WTERMS>(w[j], wt);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        // tokens past the last read the last: their sums are not stored
                        const int t = n * 16 + r < a.T ? n * 16 + r : a.T - 1;
                        V8 xt[XTERMS];
#pragma unroll
                        for (int k = 0; k < XTERMS; ++k)
                            xt[k] = *reinterpret_cast<const V8*>(xs + (k * a.T + t) * pitch + c0 + j * 8);
#pragma unroll
                        for (int p = 0; p < WTERMS; ++p)
#pragma unroll
                            for (int k = 0; k < XTERMS; ++k)
                                if (p + k < ORDERS) acc[n] = Bf16::mfma(wt[p], xt[k], acc[n]);
                    }
                }
                c0 += H * 8;
#pragma unroll
                for (int i = 0; i + U * H / 2 < 4; ++i) {
                    k1[i] = k1[i + U * H / 2];
                    k2[i] = k2[i + U * H / 2];
                }
            }
        }

        // exact entries whose column lies in the slab: x from its terms
        if (sparse) {
            const int64_t col0 = sv0 * d, col1 = (int64_t)se * kBlock < a.nb ? (int64_t)se * kBlock * d : a.N;
            const int32_t* const col = sparse_id < kQRows ? a.q[0].col : a.q[1].col;
            const float* const delta = sparse_id < kQRows ? a.q[0].delta : a.q[1].delta;
            const int place = lane % per_row, step = per_row / tp;
#pragma unroll 1
            for (int t0 = 0; t0 < a.T; t0 += tp) {
                const int t = t0 + (place & (tp - 1)), tx = t < a.T ? t : a.T - 1;
                float c = 0.0f;
#pragma unroll 1
                for (int e = e0 + place / tp; e < e1; e += step * 4) {
                    int j[4];
                    float v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {              // four entries in flight
                        const int k = e + u * step < e1 ? e + u * step : e1 - 1;
                        j[u] = col[k];
                        v[u] = delta[k];
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (e + u * step >= e1 || j[u] < col0 || j[u] >= col1) continue;
                        const int cl = (int)(j[u] - col0);
                        const int at = D ? cl : cl / d * S + cl % d;
                        float x = 0.0f;
#pragma unroll
                        for (int k = 0; k < XTERMS; ++k) x += (float)xs[(k * a.T + tx) * pitch + at];
                        c = fmaf(v[u], x, c);
                    }
                }
                for (int o = per_row / 2; o >= tp; o >>= 1) c += __shfl_xor(c, o, 64);
                float* const sum = cor + (sparse_id / kQRows * NT * 16 + t) * kQRows + sparse_id % kQRows;
                if (place < tp && t < a.T) *sum = sb == kb0 ? c : *sum + c;
            }
        }
    }

    // Item threadIdx.x of the sums is fragment n, lane l, element e -> token, row; what
    // its end needs is loaded ahead of the exchange.
    const int item_t = (item >> 8) * 16 + ((item >> 2) & 15), item_r = ((item >> 6) & 3) * 4 + (item & 3);
    const int64_t out_row = row0 + item_r;
    const bool stores = item < NT * 256 && item_t < a.T && out_row < a.M;
    float rs_v[2] = {1.0f, 1.0f}, bias_v[2] = {0.0f, 0.0f}, res_v = 0.0f;
    if (stores) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (m >= nm) break;
            if (a.q[m].rs) rs_v[m] = a.q[m].rs[out_row];
            if (a.bias[m]) bias_v[m] = load_any(a.bias[m], out_row, XT);
        }
        if (a.R) res_v = load_any(a.R, item_t * a.ldr + out_row, XT);
    }

    // sums over the waves, in wave order, and the corrections
    __syncthreads();
    float* red = lds + used;                                   // [nwaves][NT][64] of four rows
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(red + ((wave * NT + n) * 64 + lane) * 4) = acc[n];
    __syncthreads();
    if (!stores) return;
    float z[2] = {0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (m >= nm) break;
        const float* p = red + m * NT * 256 + (item >> 8) * 256 + (item & 255);
        float v = 0.0f;
        for (int w = 0; w < turns; w += 4) {                   // 4, 8 or 16 waves a matrix
            float f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) f[u] = p[(w + u) * nm * NT * 256];
#pragma unroll
            for (int u = 0; u < 4; ++u) v += f[u];
        }
        if (a.q[m].rs) v *= rs_v[m];
        z[m] = sparse ? v + cor[(m * NT * 16 + item_t) * kQRows + item_r] : v;
        if (__builtin_expect(!a.part && !__builtin_isfinite(z[m]), 0))
            z[m] = defined_sum(a.q[m], static_cast<const E*>(a.X) + item_t * a.ldx, out_row, a.nb, d);
        if (a.part) a.part[(((int64_t)blockIdx.y * nm + m) * a.T + item_t) * a.M + out_row] = z[m];
        z[m] += bias_v[m];
    }
    if (a.part) return;
    float y = act_full(a.act, z[0]);
    if (nm > 1) y *= z[1];
    if (a.R) y += res_v;
    store_any(a.Y, item_t * a.ldy + out_row, XT, y);
}

// Adds the parts in order and applies the epilogue.
template <int XT>
__global__ __launch_bounds__(256) void k_qffn_finish(const QArgs a)
{
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = (int64_t)a.T * a.M;
    if (e >= n) return;
    const int64_t t = e / a.M, row = e - t * a.M;
    float z[2] = {0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (m >= a.nm) break;
        float v = 0.0f;
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) v += a.part[((int64_t)s * a.nm + m) * n + e];
        if (__builtin_expect(!__builtin_isfinite(v), 0))
            v = defined_sum(a.q[m], static_cast<const typename XType<XT>::E*>(a.X) + t * a.ldx, row, a.nb, a.d);
        z[m] = a.bias[m] ? v + load_any(a.bias[m], row, XT) : v;
    }
    float y = act_full(a.act, z[0]);
    if (a.nm > 1) y *= z[1];
    if (a.R) y += load_any(a.R, t * a.ldr + row, XT);
    store_any(a.Y, t * a.ldy + row, XT, y);
}

// delta_e = val_e - decoded weight at e (each step rounded as the
// reconstruction rounds it, then the difference).
__global__ __launch_bounds__(256) void k_sparse_delta(int64_t M, int64_t N, int64_t nb, int d, const float* __restrict__ C1,
                                                      int K1, const uint16_t* __restrict__ idx1,
                                                      const float* __restrict__ C2, int K2,
                                                      const uint16_t* __restrict__ idx2, const float* __restrict__ rs,
                                                      const float* __restrict__ cs, const int32_t* __restrict__ row_ptr,
                                                      const int32_t* __restrict__ col, const float* __restrict__ val,
                                                      float* __restrict__ delta)
{
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= M) return;
    const int e1 = row_ptr[i + 1];
    for (int e = row_ptr[i] + lane; e < e1; e += 64) {
        const int64_t j = col[e];
        float w = 0.0f;
        if (j >= 0 && j < N) {
            const int64_t s = j / d;
            const int t = (int)(j - s * d);
            const int k1 = idx1[i * nb + s];
            w = C1[(int64_t)(k1 < K1 ? k1 : K1 - 1) * d + t];
            if (C2) {
                const int k2 = idx2[i * nb + s];
                w = w + C2[(int64_t)(k2 < K2 ? k2 : K2 - 1) * d + t];
            }
            if (cs) w = w * cs[j];
            if (rs) w = w * rs[i];
        }
        delta[e] = val[e] - w;
    }
}

// ---- plan ---------------------------------------------------------------
constexpr size_t kLdsTwo = 72 * 1024, kLdsOne = 144 * 1024;      // a workgroup's LDS with two or one on a CU

int64_t q_groups(int64_t M) { return (M + kQRows - 1) / kQRows; }
int64_t q_blocks(int64_t nb) { return (nb + kBlock - 1) / kBlock; }

// Each row's blocks are split over up to 16 workgroups while the workgroups stay
// one a CU and have four blocks or more.  179 x 15720, one token: 17 us over 8 or
// 16, 37 us over one, 22 us over 32; 512 x 4096, pair: 17 us over 4, 31 us over
// one; 256 x 1024: 10 us over one, 13 us over two.
int q_splits(int64_t M, int64_t nb)
{
    int s = 1;
    while (s < 16 && q_groups(M) * s * 2 <= 256 && q_blocks(nb) >= s * 8) s *= 2;
    return s;
}

// Eight waves a workgroup where its tokens and scales fit in half a CU's LDS at
// once, so that two share a CU and one gathers while the other stages or sums;
// else sixteen.  Pair of 8192 x 2048, one token: 31 us with eight, 39 us with
// sixteen; of 11008 x 4096, one token 74 and 87 us, but 16 tokens (more slabs)
// 145 and 124 us.  Many tokens' exact entries are shared among sixteen where the
// rows leave one workgroup a CU: pair of 512 x 4096, 24 tokens, 31 and 26 us;
// without exact entries 19.0 and 19.6 us.  lds: bytes staged at once.
int q_waves(const QArgs& a, size_t lds)
{
    if (q_blocks(a.nb) * a.nm < 16) return 8;
    const bool sparse = a.q[0].row_ptr || (a.nm > 1 && a.q[1].row_ptr);
    return lds > kLdsTwo || (sparse && a.T > 8 && q_groups(a.M) * a.splits < 512) ? 16 : 8;
}

size_t q_workspace(int64_t M, int64_t nb, int64_t T, int nm)
{
    const int splits = q_splits(M, nb);
    const int64_t t = T < kQTokens ? T : kQTokens;
    return splits > 1 ? align_up((size_t)splits * nm * t * M * sizeof(float)) : 0;
}

template <int D, int XT, int NT>
vq_status q_launch(QArgs a, hipStream_t st)
{
    constexpr int S = slots_of(D);
    size_t c2 = (size_t)a.nm * NT * 16 * kQRows * sizeof(float);   // the corrections and the residual codebooks
    int scales = 0;
    for (int m = 0; m < a.nm; ++m) {
        if (a.q[m].C2 && a.q[m].K2 * S <= kC2Floats) c2 += (size_t)a.q[m].K2 * S * sizeof(float);
        scales += a.q[m].cs != nullptr;
    }
    const size_t per_token = XType<XT>::kTerms * 2 * (size_t)a.T;
    const auto slab_bytes = [&](int64_t sv) {
        return (size_t)scales * sv * S * sizeof(float) + per_token * token_pitch((int)(sv * S));
    };
    const int64_t mine = (q_blocks(a.nb) + a.splits - 1) / a.splits;
    const int waves = q_waves(a, c2 + slab_bytes(mine * kBlock));
    // balanced slabs of whole blocks
    const size_t cap = waves == 16 ? kLdsOne : kLdsTwo;
    int64_t slabs = 1;
    while (slabs < mine && c2 + slab_bytes((mine + slabs - 1) / slabs * kBlock) > cap) ++slabs;
    a.slab = (int)((mine + slabs - 1) / slabs * kBlock);
    const size_t sums = (size_t)waves * NT * 256 * sizeof(float);
    const size_t lds = c2 + std::max(slab_bytes(a.slab), sums);
    const auto kern = k_qffn<D, XT, NT>;
    if (lds > 64 * 1024) {
        static thread_local int set_dev = -1;
        int dev = 0;
        VQ_HIP(hipGetDevice(&dev));
        if (set_dev != dev) {
            VQ_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       160 * 1024));
            set_dev = dev;
        }
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)q_groups(a.M), a.splits), dim3(waves * 64), lds, st, a);
    VQ_LAUNCHED("k_qffn");
    return VQ_OK;
}

template <int D, int XT>
vq_status q_tokens(const QArgs& a, hipStream_t st)
{
    return a.T > 16 ? q_launch<D, XT, 2>(a, st) : q_launch<D, XT, 1>(a, st);
}

template <int D>
vq_status q_type(const QArgs& a, hipStream_t st)
{
    switch (a.dtype) {
    case VQ_BF16: return q_tokens<D, VQ_BF16>(a, st);
    case VQ_F16: return q_tokens<D, VQ_F16>(a, st);
    default: return q_tokens<D, VQ_F32>(a, st);
    }
}

vq_status q_run(QArgs a, int64_t T, int nm, void* ws, hipStream_t st)
{
    a.nm = nm;
    a.splits = q_splits(a.M, a.nb);
    a.part = a.splits > 1 ? static_cast<float*>(ws) : nullptr;
    bool vec = a.d == 8 || (a.d == 4 && a.nb % 2 == 0);          // chunks of eight columns
    for (int m = 0; m < nm; ++m) vec = vec && aligned16(a.q[m].C1) && (!a.q[m].C2 || aligned16(a.q[m].C2));
    const size_t e = a.dtype == VQ_F32 ? 4 : 2;
    const char* X = static_cast<const char*>(a.X);
    const char* R = static_cast<const char*>(a.R);
    char* Y = static_cast<char*>(a.Y);
    for (int64_t t0 = 0; t0 < T; t0 += kQTokens) {
        a.T = (int)(T - t0 < kQTokens ? T - t0 : kQTokens);
        a.X = X + t0 * a.ldx * e;
        a.R = R ? R + t0 * a.ldr * e : nullptr;
        a.Y = Y + t0 * a.ldy * e;
        VQ_TRY(vec && a.d == 8 ? q_type<8>(a, st) : vec ? q_type<4>(a, st) : q_type<0>(a, st));
        if (a.part) {
            const auto finish = a.dtype == VQ_BF16 ? k_qffn_finish<VQ_BF16>
                                : a.dtype == VQ_F16 ? k_qffn_finish<VQ_F16>
                                                    : k_qffn_finish<VQ_F32>;
            hipLaunchKernelGGL(finish, dim3(grid_for((int64_t)a.T * a.M, 256)), dim3(256), 0, st, a);
            VQ_LAUNCHED("k_qffn_finish");
        }
    }
    return VQ_OK;
}

vq_status check_qmatrix(const std::string& call, const vq_qmatrix* Q)
{
    VQ_CHECK(Q != nullptr, call + ": matrix is null");
    VQ_TRY(check_shape(Q->M, Q->N, Q->d));
    const int64_t n_sub = Q->M * Q->N / Q->d;
    VQ_TRY(check_K(Q->K1, n_sub));
    VQ_CHECK(Q->C1 && Q->idx1, call + ": null pointer");
    if (Q->C2) {
        VQ_TRY(check_K(Q->K2, n_sub));
        VQ_CHECK(Q->idx2 != nullptr, call + ": idx2 is null");
    }
    return VQ_OK;
}

vq_status check_call(const std::string& call, const vq_qmatrix* Q, int64_t T, int dtype, int act, const void* X, int64_t ldx,
                     const void* Y, int64_t ldy, const void* bias, const void* R, int64_t ldr)
{
    VQ_TRY(check_qmatrix(call, Q));
    VQ_CHECK(!Q->row_ptr || (Q->col && Q->delta), call + ": the sparse part needs col and delta");
    VQ_CHECK(T >= 0 && T <= (1 << 28), call + ": T must be in [0, 2^28]");
    VQ_CHECK(dtype >= VQ_BF16 && dtype <= VQ_F32, call + ": dtype must be VQ_BF16, VQ_F16 or VQ_F32");
    VQ_CHECK(act >= VQ_ACT_NONE && act <= VQ_ACT_SIGMOID, call + ": unknown activation");
    if (T == 0) return VQ_OK;
    VQ_CHECK(X && Y, call + ": null pointer");
    VQ_CHECK(ldx >= Q->N && ldx <= ((int64_t)1 << 40), call + ": leading dimension of X is out of range");
    VQ_CHECK(ldy >= Q->M && ldy <= ((int64_t)1 << 40), call + ": leading dimension of the output is out of range");
    VQ_CHECK(!R || (ldr >= Q->M && ldr <= ((int64_t)1 << 40)), call + ": leading dimension of R is out of range");
    const uintptr_t mis = dtype == VQ_F32 ? 3 : 1;
    for (const void* p : {X, Y, bias, R})
        VQ_CHECK((reinterpret_cast<uintptr_t>(p) & mis) == 0, call + ": a tensor is not aligned to its elements");
    VQ_CHECK(X != Y, call + ": the output may not alias X");
    VQ_CHECK(bias != Y, call + ": the output may not alias a bias");
    VQ_CHECK(Y != R || ldy == ldr, call + ": Y in place of R needs R's leading dimension");
    return VQ_OK;
}

vq_status check_qvalues(const char* call, const vq_qmatrix* Q, hipStream_t stream)
{
    VQ_VALUES(Q->C1, (int64_t)Q->K1 * Q->d, false, call, "C1");
    VQ_VALUES(Q->C2, (int64_t)Q->K2 * Q->d, false, call, "C2");
    VQ_VALUES(Q->rscale, Q->M, false, call, "rscale");
    VQ_VALUES(Q->cscale, Q->N, false, call, "cscale");
    return VQ_OK;
}

QMat device_matrix(const vq_qmatrix* Q)
{
    return {Q->C1, Q->idx1, Q->C2, Q->idx2, Q->rscale, Q->cscale, Q->row_ptr, Q->col, Q->delta, Q->K1, Q->C2 ? Q->K2 : 0};
}

}  // namespace
}  // namespace vq

using namespace vq;

extern "C" {

vq_status vq_sparse_delta(const vq_qmatrix* Q, const float* val, float* delta, void* stream)
{
    const char* call = "vq_sparse_delta";
    VQ_TRY(check_qmatrix(call, Q));
    VQ_CHECK(Q->row_ptr && Q->col && val && delta, "vq_sparse_delta: null pointer");
    VQ_TRY(check_device());
    VQ_TRY(check_qvalues(call, Q, as_stream(stream)));
    hipLaunchKernelGGL(k_sparse_delta, dim3(grid_for(Q->M, 4)), dim3(256), 0, as_stream(stream), Q->M, Q->N, Q->N / Q->d, Q->d,
                       Q->C1, Q->K1, Q->idx1, Q->C2, Q->K2, Q->idx2, Q->rscale, Q->cscale, Q->row_ptr, Q->col, val, delta);
    VQ_LAUNCHED("k_sparse_delta");
    return VQ_OK;
}

size_t vq_qlinear_workspace_bytes(int64_t M, int64_t N, int d, int64_t T)
{
    if (T <= 0 || check_shape(M, N, d) != VQ_OK) return 0;
    return q_workspace(M, N / d, T, 1);
}

vq_status vq_qlinear(const vq_qmatrix* Q, int64_t T, int dtype, int act, const void* X, int64_t ldx, const void* bias,
                     const void* R, int64_t ldr, void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_qlinear";
    VQ_TRY(check_call(call, Q, T, dtype, act, X, ldx, Y, ldy, bias, R, ldr));
    if (T == 0) return VQ_OK;
    const size_t need = q_workspace(Q->M, Q->N / Q->d, T, 1);
    VQ_TRY(check_workspace(call, ws, ws_bytes, need));
    VQ_TRY(check_device());
    VQ_TRY(check_qvalues(call, Q, as_stream(stream)));
    VQ_TRY(check_matrix(X, T, Q->N, ldx, dtype, call, "X", as_stream(stream)));
    VQ_TRY(check_matrix(bias, 1, Q->M, Q->M, dtype, call, "bias", as_stream(stream)));
    VQ_TRY(check_matrix(R, T, Q->M, ldr, dtype, call, "R", as_stream(stream)));
    QArgs a{};
    a.q[0] = device_matrix(Q);
    a.M = Q->M; a.N = Q->N; a.nb = Q->N / Q->d; a.d = Q->d;
    a.X = X; a.ldx = ldx;
    a.dtype = dtype; a.act = act;
    a.bias[0] = bias;
    a.R = R; a.ldr = ldr;
    a.Y = Y; a.ldy = ldy;
    TimedRegion tr("qlinear", 0, as_stream(stream));
    return q_run(a, T, 1, ws, as_stream(stream));
}

size_t vq_qgated_workspace_bytes(int64_t M, int64_t N, int d, int64_t T)
{
    if (T <= 0 || check_shape(M, N, d) != VQ_OK) return 0;
    return q_workspace(M, N / d, T, 2);
}

vq_status vq_qgated(const vq_qmatrix* Qg, const vq_qmatrix* Qu, int64_t T, int dtype, int act, const void* X, int64_t ldx,
                    const void* bg, const void* bu, void* H, int64_t ldh, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_qgated";
    VQ_TRY(check_call(call, Qg, T, dtype, act, X, ldx, H, ldh, bg, nullptr, 0));
    VQ_TRY(check_call(call, Qu, T, dtype, act, X, ldx, H, ldh, bu, nullptr, 0));
    VQ_CHECK(Qg->M == Qu->M && Qg->N == Qu->N && Qg->d == Qu->d, "vq_qgated: the matrices differ in M, N or d");
    if (T == 0) return VQ_OK;
    const size_t need = q_workspace(Qg->M, Qg->N / Qg->d, T, 2);
    VQ_TRY(check_workspace(call, ws, ws_bytes, need));
    VQ_TRY(check_device());
    VQ_TRY(check_qvalues(call, Qg, as_stream(stream)));
    VQ_TRY(check_qvalues(call, Qu, as_stream(stream)));
    VQ_TRY(check_matrix(X, T, Qg->N, ldx, dtype, call, "X", as_stream(stream)));
    VQ_TRY(check_matrix(bg, 1, Qg->M, Qg->M, dtype, call, "bg", as_stream(stream)));
    VQ_TRY(check_matrix(bu, 1, Qg->M, Qg->M, dtype, call, "bu", as_stream(stream)));
    QArgs a{};
    a.q[0] = device_matrix(Qg);
    a.q[1] = device_matrix(Qu);
    a.M = Qg->M; a.N = Qg->N; a.nb = Qg->N / Qg->d; a.d = Qg->d;
    a.X = X; a.ldx = ldx;
    a.dtype = dtype; a.act = act;
    a.bias[0] = bg; a.bias[1] = bu;
    a.Y = H; a.ldy = ldh;
    TimedRegion tr("qgated", 0, as_stream(stream));
    return q_run(a, T, 2, ws, as_stream(stream));
}

}  // extern "C"
