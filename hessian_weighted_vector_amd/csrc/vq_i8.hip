// Products in 8-bit integers with a scale for each token and each row of the matrix
// (vq_quantize_rows, vq_linear_i8, vq_gated_i8).
//
//   q[t, j] = nearest(127 x[t, j] / top_t), top_t = max_j |x[t, j]|, s_t = top_t / 127
//   z[t, m] = s_t w_m sum_j q[t, j] Q[m, j] + bias,  Y = act(z) + R, or H = act(g) u
//
//   k_i8_rows       the tokens' codes and scales: one read of X
//   k_i8_gemm       the tiled product: its loop takes pairs of 8-bit elements where the
//                   16-bit products take one, so tiles, LDS layout and steps are theirs
//                   and a step is 128 columns
//   k_i8_few        few tokens: the matrix straight from memory into matrix-core operands
//   k_i8_finish     adds split sums
//
// The sums are exact in 32 bits (127 * 128 * 2^17 < 2^31), whatever the order and the
// split; they are converted to float32, scaled and go through the epilogue of the dense calls.
// For 16-bit tokens the codes are those of exact arithmetic: a quotient that is no
// tie is at least 2^-19 of its value away from one, and the arithmetic rounds by 2^-23.
//
// What bounds it: a step of the tile loop takes as many cycles of LDS as of the matrix cores.
// 4096 tokens by a pair of 28672 x 8192 1.38 to 1.46 ms (2.6 to 2.8 POP/s, matrix cores busy 0.72 at 1.8
// GHz; 1.29 ms with zeros, so power is a tenth of it); 2048 by 4096 x 11008 101 to 111 us, 14 of
// them the codes; one token 12 us, matrices from memory 14.4 (45 MB at the rate of a large read: 7.3).
#include "vq_tile.h"

#include <algorithm>

namespace vq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Sixteen 8-bit elements a lane; the tile loop sees eight 16-bit ones.
struct I8 {
    typedef i32x4 Acc;
    typedef i32x4 V8;
    static __device__ __forceinline__ i32x4 mfma(i32x4 a, i32x4 b, i32x4 c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }
};

constexpr int64_t kMaxColumns = 1 << 17;      // the sums stay below 2^31
constexpr int64_t kMaxI8Tokens = 1 << 28;
constexpr int64_t kRowBytes = 64;             // rows of codes begin and end on these

inline int64_t round64(int64_t n) { return (n + 63) / 64 * 64; }

// ---- codes of rows ------------------------------------------------------------
struct Rows {
    const void* X;
    int64_t rows, ldx;
    int cols;
    int8_t* q;
    int64_t ldq;                 // zeros from cols on
    float* scale;
    int odd;
};

// Eight elements from column c on (those below cols, else 0), in their own type.
template <class E>
struct Eight {
    typedef E V __attribute__((ext_vector_type(8)));
    V v;
    __device__ __forceinline__ void load(const E* row, int c, int cols, int odd)
    {
        if (c + 8 <= cols) {
            if (sizeof(E) == 2 && odd) {
                Words w;
                w.load(row + c);
                const uint4 u = w.get(row + c);
                __builtin_memcpy(&v, &u, 16);
            } else {
                __builtin_memcpy(&v, row + c, sizeof(v));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? row[c + i] : (E)0.0f;
        }
    }
};

// The largest magnitude as bits of a float32: NaN and infinities are above every number.
// Bits without the sign order as the magnitudes do, two of 16 bits at a time.
template <class E>
struct Top {
    typedef unsigned short U2 __attribute__((ext_vector_type(2)));
    U2 m = {0, 0};
    __device__ __forceinline__ void add(const Eight<E>& e)
    {
        uint32_t w[4];
        __builtin_memcpy(w, &e.v, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(U2, w[i] & 0x7fff7fffu));
    }
    __device__ __forceinline__ uint32_t bits() const
    {
        const unsigned short t = m[0] > m[1] ? m[0] : m[1];
        return __float_as_uint((float)__builtin_bit_cast(E, t));
    }
};
template <>
struct Top<float> {
    uint32_t m = 0;
    __device__ __forceinline__ void add(const Eight<float>& e)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(e.v[i]) & 0x7fffffffu;
            m = b > m ? b : m;
        }
    }
    __device__ __forceinline__ uint32_t bits() const { return m; }
};

// Codes of a row whose largest magnitude has these bits; all zero where that is 0 or not finite.
//
// 16-bit elements: y = x (127 / top) in place of 127 x / top, at a fifth of a division's
// instructions.  y is within 2^-23 of the quotient relatively, two units in its last place.  A
// tie, k + 1/2 with k < 127, has eight bits, and any other quotient is 2^-19 of itself away from
// one; so y with its last three bits rounded off is the tie where the quotient is one and on
// the quotient's side of it elsewhere.  Adding 1.5 2^23 then rounds to an integer, ties to even,
// whose low byte is the code.  Below 2^-90, where 127 / top could overflow, and for float32
// elements, each is divided: 127 x rounded, then the quotient rounded.  Rows above 2^120, where 127 x
// could overflow, are taken 2^-7 times as large, which changes no code.
template <class E>
struct Coder {
    float top, r, shrink;
    bool divide;
    __device__ __forceinline__ explicit Coder(uint32_t bits)
    {
        top = bits < 0x7f800000u ? __uint_as_float(bits) : 0.0f;
        shrink = sizeof(E) == 4 && top > 0x1p120f ? 0x1p-7f : 1.0f;
        top *= shrink;
        divide = sizeof(E) == 4 || (top > 0.0f && top < 0x1p-90f);
        r = top > 0.0f && !divide ? 127.0f / top : 0.0f;
    }
    static __device__ __forceinline__ float scale(uint32_t bits) { return bits < 0x7f800000u ? __uint_as_float(bits) / 127.0f : NAN; }
    __device__ __forceinline__ uint2 codes(const Eight<E>& e) const
    {
        uint32_t k[8];
        if (divide) {
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = top > 0.0f ? (uint32_t)__float2int_rn(127.0f * ((float)e.v[i] * shrink) / top) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = (float)e.v[i];
                // of a row that is not finite: 0, not NaN
                const uint32_t y = __float_as_uint(r > 0.0f ? x * r : 0.0f);
                k[i] = __float_as_uint(__uint_as_float((y + 4u) & ~7u) + 0x1.8p23f);
            }
        }
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // bytes: v_perm takes the second operand's as 0..3, the first's as 4..7
            const uint32_t lo = __builtin_amdgcn_perm(k[h * 4 + 1], k[h * 4], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(k[h * 4 + 3], k[h * 4 + 2], 0x04000c0cu);
            w[h] = lo | hi;
        }
        return make_uint2(w[0], w[1]);
    }
};

__device__ __forceinline__ uint32_t wave_max(uint32_t t)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = (uint32_t)__shfl_xor((int)t, o);
        t = v > t ? v : t;
    }
    return t;
}

// WAVES waves a row (1 or 4), four waves a workgroup.  The first R chunks of a lane stay
// in registers, those of longer rows are read again.
template <class E, int WAVES, int R>
__global__ __launch_bounds__(256) void k_i8_rows(const Rows a)
{
    __shared__ uint32_t tops[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r = WAVES == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (r >= a.rows) return;                                  // whole waves; with four a row, whole workgroups
    const int first = (WAVES == 1 ? lane : threadIdx.x) * 8, stride = WAVES * 64 * 8;
    const E* row = static_cast<const E*>(a.X) + r * a.ldx;
    Eight<E> v[R];
    Top<E> most;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (first + i * stride < a.cols) v[i].load(row, first + i * stride, a.cols, a.odd);
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (first + i * stride < a.cols) most.add(v[i]);
    for (int c = first + R * stride; c < a.cols; c += stride) {
        Eight<E> w;
        w.load(row, c, a.cols, a.odd);
        most.add(w);
    }
    uint32_t top = wave_max(most.bits());
    if (WAVES > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) top = tops[k] > top ? tops[k] : top;
    }
    const Coder<E> coder(top);
    int8_t* const q = a.q + r * a.ldq;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (first + i * stride < a.cols) *reinterpret_cast<uint2*>(q + first + i * stride) = coder.codes(v[i]);
    for (int c = first + R * stride; c < a.cols; c += stride) {
        Eight<E> w;
        w.load(row, c, a.cols, a.odd);
        *reinterpret_cast<uint2*>(q + c) = coder.codes(w);
    }
    // columns past the last chunk
    for (int64_t c = (a.cols + 7) / 8 * 8 + first; c < a.ldq; c += stride) *reinterpret_cast<uint2*>(q + c) = make_uint2(0, 0);
    if (first == 0) a.scale[r] = Coder<E>::scale(top);
}

// A launch takes fewer than 2^32 threads.
template <class E>
void rows_launch(const Rows& all, hipStream_t st)
{
    constexpr int64_t kRows = 1 << 23;
    for (int64_t r = 0; r < all.rows; r += kRows) {
        Rows a = all;
        a.X = static_cast<const E*>(all.X) + r * all.ldx;
        a.rows = std::min(all.rows - r, kRows);
        a.q += r * all.ldq;
        a.scale += r;
        // a wave a row up to 4096 columns (eight chunks of 64 lanes)
        if (a.cols <= 4096) hipLaunchKernelGGL((k_i8_rows<E, 1, 8>), dim3((unsigned)((a.rows + 3) / 4)), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_i8_rows<E, 4, 8>), dim3((unsigned)a.rows), dim3(256), 0, st, a);
    }
}

vq_status rows_codes(const Rows& a, int dtype, hipStream_t st)
{
    if (dtype == VQ_BF16) rows_launch<__bf16>(a, st);
    else if (dtype == VQ_F16) rows_launch<_Float16>(a, st);
    else rows_launch<float>(a, st);
    VQ_LAUNCHED("k_i8_rows");
    return VQ_OK;
}

// ---- scaled sums ----------------------------------------------------------------
struct Scales {
    const float* x;              // a token's
    const float* w[2];           // a row's of each matrix
};

// Features m .. m+7 of token t: the epilogue of the dense calls from exact sums; w0, w1:
// these features' scales.
template <class T, bool PAIR>
__device__ __forceinline__ void finish(const Epilogue& e, const float (&w0)[8], const float (&w1)[8], float sx, int64_t t, int m,
                                       int M, const int (&v)[8], const int (&u)[8])
{
    float z[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z[i] = (float)v[i] * sx * w0[i];
        if (PAIR) y[i] = (float)u[i] * sx * w1[i];
    }
    if (PAIR) epilogue_pair<T>(e, t, m, M, z, y);
    else epilogue_one<T>(e, t, m, M, z);
}

// Scales m .. m+7 (0 from M on).
__device__ __forceinline__ void eight_scales(const float* s, int m, int M, float (&w)[8])
{
    if (m + 8 <= M) {
        __builtin_memcpy(w, s + m, 32);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = m + i < M ? s[m + i] : 0.0f;
    }
}

// ---- the tiled product -------------------------------------------------------------
struct I8Tile {
    Tile t;                      // part: int32 sums
    int turn;                    // workgroups begin at different steps
    Scales s;
};

template <class T, int FP, int FQ, bool PAIR>
__global__ __launch_bounds__(kThreads, FP * FQ >= 32 ? 2 : 4) void k_i8_gemm(const I8Tile a)
{
    typedef Main<I8, false, false, FP, FQ, PAIR> L;
    constexpr int kP = PAIR ? L::BP / 2 : L::BP;              // features of the tile
    VQ_TILE_BUFFERS(L);
    // the tile's scales, read in front of the product and kept: in the epilogue a row's would be waited for each time
    __shared__ __align__(16) float scale_q[L::BQ], scale_p[PAIR ? 2 : 1][kP];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave / kWQ, wq = wave % kWQ, split = blockIdx.y;
    int tp, tq;
    pick_tile(blockIdx.x, a.t.ntp * a.t.ntq, a.t.ntp, a.t.ntq, tp, tq);
    const int p0 = tp * kP, q0 = tq * L::BQ;
    static_assert(L::BQ <= kThreads && kP <= kThreads, "a scale a thread");
    const int i_q = q0 + (int)threadIdx.x < a.t.nq ? q0 + (int)threadIdx.x : a.t.nq - 1;
    const int i_p = p0 + (int)threadIdx.x < a.t.np ? p0 + (int)threadIdx.x : a.t.np - 1;
    const float my_q = a.s.x[i_q], my_p = a.s.w[0][i_p], my_p2 = PAIR ? a.s.w[1][i_p] : 0.0f;
    const int pairs = (a.t.steps + 1) / 2;
    const int s0 = 2 * (int)((int64_t)pairs * split / a.t.splits);
    int s1 = 2 * (int)((int64_t)pairs * (split + 1) / a.t.splits);
    i32x4 acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    if constexpr (FP * FQ < 32) {
        const int at = a.turn ? turned(s0, s1) : s0;
        if (at > s0) {
            L::run(a.t, p0, q0, 0, at, s1, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);
            run_again();
            s1 = at;
        }
    }
    L::run(a.t, p0, q0, 0, s0, s1, wave, lane, (lds_ptr)pb0, (lds_ptr)pb1, (lds_ptr)qb0, (lds_ptr)qb1, acc);
    if (a.t.part) {
        constexpr int NI = PAIR ? FP / 2 : FP;
        const int64_t plane = (int64_t)a.t.nq * a.t.pitch;
        int* o = reinterpret_cast<int*>(a.t.part) + (int64_t)split * (PAIR ? 2 : 1) * plane;
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            const int q = q0 + (wq * FQ + j) * 16 + (lane & 15);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int p = p0 + (wp * NI + i) * 16 + (lane >> 4) * 4;
                if (q >= a.t.nq || p >= a.t.np) continue;
                *reinterpret_cast<i32x4*>(o + (int64_t)q * a.t.pitch + p) = acc[i][j];
                if (PAIR) *reinterpret_cast<i32x4*>(o + plane + (int64_t)q * a.t.pitch + p) = acc[i + NI][j];
            }
        }
        __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));           // no load into LDS outlives the workgroup
        return;
    }
    if (threadIdx.x < L::BQ) scale_q[threadIdx.x] = my_q;
    if (threadIdx.x < kP) {
        scale_p[0][threadIdx.x] = my_p;
        if (PAIR) scale_p[PAIR ? 1 : 0][threadIdx.x] = my_p2;
    }
    // behind each_row's barrier every scale is there
    each_row<L>(acc, p0, q0, a.t.np, a.t.nq, wave, lane, pb0, pb1, qb0, qb1, [&](int q, int p, int (&v)[8], int (&u)[8]) {
        float w0[8], w1[8];
        __builtin_memcpy(w0, __builtin_assume_aligned(scale_p[0] + (p - p0), 16), 32);
        if (PAIR) __builtin_memcpy(w1, __builtin_assume_aligned(scale_p[PAIR ? 1 : 0] + (p - p0), 16), 32);
        finish<T, PAIR>(a.t.epi, w0, w1, scale_q[q - q0], q, p, a.t.np, v, u);
    });
}

// Adds the parts [splits][matrices][T][pitch]; eight features a thread.
struct Parts {
    const int* part;
    int splits, M, T, pitch;
    Epilogue epi;
    Scales s;
};

template <class T, bool PAIR>
__global__ __launch_bounds__(256) void k_i8_finish(const Parts a)
{
    const int64_t per = a.pitch / 8, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= per * a.T) return;
    const int64_t t = e / per, plane = (int64_t)a.T * a.pitch;
    const int m = (int)(e - t * per) * 8;
    const int* o = a.part + t * a.pitch + m;
    int v[8] = {}, u[8] = {};
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {
        const int* oz = o + (int64_t)z * (PAIR ? 2 : 1) * plane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const i32x4 w = *reinterpret_cast<const i32x4*>(oz + h * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h * 4 + i] += w[i];
            if (PAIR) {
                const i32x4 w2 = *reinterpret_cast<const i32x4*>(oz + plane + h * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) u[h * 4 + i] += w2[i];
            }
        }
    }
    float w0[8], w1[8];
    eight_scales(a.s.w[0], m, a.M, w0);
    if (PAIR) eight_scales(a.s.w[1], m, a.M, w1);
    finish<T, PAIR>(a.epi, w0, w1, a.s.x[t], t, m, a.M, v, u);
}

// The same with the scales, biases and residual of eight whole features read beforehand.
template <class T, bool PAIR>
struct Inputs {
    typedef typename T::E E;
    typedef typename T::V8 V8;
    float w[PAIR ? 2 : 1][8];
    V8 bias[PAIR ? 2 : 1], r;
    __device__ __forceinline__ void load(const Epilogue& e, const Scales& s, int64_t t, int m)
    {
#pragma unroll
        for (int k = 0; k < (PAIR ? 2 : 1); ++k) {
            __builtin_memcpy(w[k], s.w[k] + m, 32);
            if (e.bias[k]) __builtin_memcpy(&bias[k], static_cast<const E*>(e.bias[k]) + m, 16);
        }
        if (!PAIR && e.R) __builtin_memcpy(&r, static_cast<const E*>(e.R) + t * e.ldr + m, 16);
    }
    __device__ __forceinline__ void finish(const Epilogue& e, float sx, int64_t t, int m, int M, const int (&v)[8], const int (&u)[8]) const
    {
        float z[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] = (float)v[i] * sx * w[0][i];
            if (e.bias[0]) z[i] += (float)bias[0][i];
            if (PAIR) {
                y[i] = (float)u[i] * sx * w[PAIR ? 1 : 0][i];
                if (e.bias[1]) y[i] += (float)bias[PAIR ? 1 : 0][i];
            }
        }
        activate(e.act, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (PAIR) z[i] *= y[i];
            else if (e.R) z[i] += (float)r[i];
        }
        store8<T>(e.Y, e.ldy, t, m, M, z);
    }
};

// ---- few tokens -------------------------------------------------------------------
// A workgroup owns 16 rows of Q (of both matrices of a pair); its waves take equal runs of
// columns, a lane's 16 bytes of a row being its operand, with H chunks of 64 columns in
// flight.  OWN > 0: each workgroup makes the codes of up to OWN tokens itself, in LDS, while its
// first chunks of Q are on their way: the launch in front (4 to 6 us) is not needed.  A thread
// holds all that it reads of the tokens in registers, NX chunks of eight a token.  OWN < 0: the
// same for short rows, a wave a token, up to -OWN tokens each.
struct FewI8 {
    const int8_t* Q[2];
    int64_t ldq;
    const int8_t* x;             // codes [T][ldx]
    int64_t ldx;
    Rows rows;                   // OWN: the tokens, at least eight columns; scale: written where part is
    int M, T, chunks;            // of 64 columns
    int splits, pitch;
    int* part;                   // [splits][matrices][T][pitch], or null
    Scales s;
    Epilogue epi;
};

constexpr int kOwnBytes = 60 << 10;      // LDS for codes and the waves' sums
constexpr int kOwnPad = 16;              // between the codes' rows: other banks

template <class T, int NT, bool PAIR, int H, int OWN, int NX>
__global__ __launch_bounds__(1024) void k_i8_few(const FewI8 a)
{
    typedef typename T::E E;
    constexpr int NM = PAIR ? 2 : 1;
    extern __shared__ __align__(16) int red[];                // [waves][NM][NT][64] of four features; OWN: codes [T][ldx + pad]
    __shared__ uint32_t tops[OWN > 0 ? OWN : 1][16];
    __shared__ float own_scale[OWN > 0 ? OWN : OWN < 0 ? 32 : 1];
    const int nwaves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int m0 = blockIdx.x * 16;
    const int64_t row = m0 + r < a.M ? m0 + r : a.M - 1;      // rows and tokens past the last repeat it
    int8_t* const codes = reinterpret_cast<int8_t*>(red + nwaves * NM * NT * 256);
    const int ldc = (int)a.ldx + kOwnPad;
    const int8_t* w[NM];
    const int8_t* x[NT];
#pragma unroll
    for (int m = 0; m < NM; ++m) w[m] = a.Q[m] + row * a.ldq + g * 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = n * 16 + r < a.T ? n * 16 + r : a.T - 1;
        x[n] = (OWN ? codes + t * ldc : a.x + (int64_t)t * a.ldx) + g * 16;
    }
    i32x4 acc[NM][NT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = i32x4{0, 0, 0, 0};
    // the wave's chunks of its split
    const int c0 = (int)((int64_t)a.chunks * blockIdx.y / a.splits), c1 = (int)((int64_t)a.chunks * (blockIdx.y + 1) / a.splits);
    const int wb = c0 + (c1 - c0) * wave / nwaves, n = c0 + (c1 - c0) * (wave + 1) / nwaves - wb;
    i32x4 wv[NM][H], xv[OWN ? 1 : NT][OWN ? 1 : H];
    const auto load_w = [&](int k, int j) {
        const int64_t c = (int64_t)(wb + k) * 64;
#pragma unroll
        for (int m = 0; m < NM; ++m) wv[m][j] = *reinterpret_cast<const i32x4*>(w[m] + c);
    };
    const auto load_x = [&](int k, int j) {
        const int64_t c = (int64_t)(wb + k) * 64;
#pragma unroll
        for (int t = 0; t < NT; ++t) xv[t][j] = *reinterpret_cast<const i32x4*>(x[t] + c);
    };
    const auto multiply = [&](int k, int j) {
        const int64_t c = (int64_t)(wb + k) * 64;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            i32x4 v;
            if constexpr (OWN != 0) v = *reinterpret_cast<const i32x4*>(x[t] + c);
            else v = xv[t][j];
#pragma unroll
            for (int m = 0; m < NM; ++m) acc[m][t] = I8::mfma(wv[m][j], v, acc[m][t]);
        }
    };
    // thread -> token t, features m .. m + 7 of the result; what its epilogue reads is requested now, not behind the sums
    const int t_out = threadIdx.x >> 1, m_out = m0 + (threadIdx.x & 1) * 8;
    const bool early = t_out < a.T && m_out + 8 <= a.M && !a.part;
    Inputs<T, PAIR> in;
    if (early) in.load(a.epi, a.s, t_out, m_out);
    const auto prefetch = [&] {
#pragma unroll
        for (int j = 0; j < H; ++j)
            if (j < n) {
                if constexpr (OWN == 0) load_x(j, j);
                load_w(j, j);
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    if constexpr (OWN > 0) {
        const E* const X = static_cast<const E*>(a.rows.X);
        const int cols = a.rows.cols, stride = blockDim.x * 8;
        Eight<E> v[OWN][NX];
        // chunks past the end repeat the row's last eight elements
#pragma unroll
        for (int t = 0; t < OWN; ++t)
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int c = (int)threadIdx.x * 8 + i * stride;
                __builtin_memcpy(&v[t][i].v, X + (t < a.T ? t : a.T - 1) * a.rows.ldx + (c < cols - 8 ? c : cols - 8), 16);
            }
        __builtin_amdgcn_sched_barrier(0);
        prefetch();
#pragma unroll
        for (int t = 0; t < OWN; ++t) {
            Top<E> most;
#pragma unroll
            for (int i = 0; i < NX; ++i) most.add(v[t][i]);
            const uint32_t top = wave_max(most.bits());
            if (lane == 0) tops[t][wave] = top;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < OWN; ++t) {
            if (t >= a.T) break;
            const uint32_t top = wave_max(lane < nwaves ? tops[t][lane & 15] : 0u);
            const Coder<E> coder(top);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                // the codes from c on, of a chunk read `late` elements too early; zeros behind the row
                const int c = (int)threadIdx.x * 8 + i * stride, late = c - (c < cols - 8 ? c : cols - 8);
                uint64_t k = __builtin_bit_cast(uint64_t, coder.codes(v[t][i]));
                k = late < 8 ? k >> (8 * late) : 0;
                if (c < (int)a.ldx) *reinterpret_cast<uint64_t*>(codes + t * ldc + c) = k;
            }
            if (threadIdx.x == 0) {
                own_scale[t] = Coder<E>::scale(top);
                if (a.part && blockIdx.x == 0 && blockIdx.y == 0) a.rows.scale[t] = own_scale[t];
            }
        }
        __syncthreads();
    } else if constexpr (OWN < 0) {
        const E* const X = static_cast<const E*>(a.rows.X);
        const int cols = a.rows.cols;
        Eight<E> v[-OWN][NX];
#pragma unroll
        for (int k = 0; k < -OWN; ++k)
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int c = lane * 8 + i * 512, t = wave + k * nwaves;
                __builtin_memcpy(&v[k][i].v, X + (t < a.T ? t : a.T - 1) * a.rows.ldx + (c < cols - 8 ? c : cols - 8), 16);
            }
        __builtin_amdgcn_sched_barrier(0);
        prefetch();
#pragma unroll
        for (int k = 0; k < -OWN; ++k) {
            const int t = wave + k * nwaves;
            if (t >= a.T) break;
            Top<E> most;
#pragma unroll
            for (int i = 0; i < NX; ++i) most.add(v[k][i]);
            const uint32_t top = wave_max(most.bits());
            const Coder<E> coder(top);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int c = lane * 8 + i * 512, late = c - (c < cols - 8 ? c : cols - 8);
                uint64_t q = __builtin_bit_cast(uint64_t, coder.codes(v[k][i]));
                q = late < 8 ? q >> (8 * late) : 0;
                if (c < (int)a.ldx) *reinterpret_cast<uint64_t*>(codes + t * ldc + c) = q;
            }
            if (lane == 0) {
                own_scale[t] = Coder<E>::scale(top);
                if (a.part && blockIdx.x == 0 && blockIdx.y == 0) a.rows.scale[t] = own_scale[t];
            }
        }
        __syncthreads();
    } else {
        prefetch();
    }
    // a chunk's registers are refilled as soon as they are used
#pragma unroll 1
    for (int b = 0; b < n; b += H) {
#pragma unroll
        for (int j = 0; j < H; ++j) {
            if (b + j >= n) break;
            multiply(b + j, j);
            __builtin_amdgcn_sched_barrier(0);
            if (b + j + H < n) {
                if constexpr (OWN == 0) load_x(b + j + H, j);
                load_w(b + j + H, j);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<i32x4*>(red + (((wave * NM + m) * NT + n) * 64 + lane) * 4) = acc[m][n];
    __syncthreads();
    const int t = t_out, f = threadIdx.x & 1;
    if (t >= a.T || m_out >= a.M) return;
    int z[2][8] = {};
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 v = {0, 0, 0, 0};
            for (int k = 0; k < nwaves; ++k)
                v += *reinterpret_cast<const i32x4*>(red + (((k * NM + m) * NT + (t >> 4)) * 64 + (f * 2 + h) * 16 + (t & 15)) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][h * 4 + i] = v[i];
        }
    if (a.part) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            int* o = a.part + (((int64_t)blockIdx.y * NM + m) * a.T + t) * a.pitch + m_out;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = z[m][i];
        }
        return;
    }
    float sx;
    if constexpr (OWN != 0) sx = own_scale[t];
    else sx = a.s.x[t];
    if (early) return in.finish(a.epi, sx, t, m_out, a.M, z[0], z[1]);
    float w0[8], w1[8];
    eight_scales(a.s.w[0], m_out, a.M, w0);
    if (PAIR) eight_scales(a.s.w[1], m_out, a.M, w1);
    finish<T, PAIR>(a.epi, w0, w1, sx, t, m_out, a.M, z[0], z[1]);
}

// ---- plan -----------------------------------------------------------------------
struct Plan {
    int few, waves;              // few tokens
    int small, ntp, ntq, steps;  // tiles
    int splits, pitch;
    size_t part_bytes;
};

// Whether tokens are few: while the codes' products stay below 1.2e9 (one or two, which need no launch
// in front, always).  Matrices from memory, few and tiles: 8192 x 8192 by 8 tokens 20.5 and 23.6 us,
// by 17 26.2 and 24.4, by 32 32.7 and 25.6; pairs of it by 3 32.4 and 34.9, by 16 39.2 and 35.7;
// 28672 x 8192 by 3 48.2 and 56.3, by 8 56.0 and 56.4, by 32 97 and 59; 8192 x 4096 by 32 21.9 and 21.0.
// The rule is wrong for pairs of 11008 x 4096 by 16 (32.0, 37.9) and 2048 x 16384 by 16 (25.7, 20.7).
bool few_tokens(int64_t T, int64_t M, int64_t N, int nm)
{
    return T <= 2 || (T <= 32 && (double)T * (double)M * (double)N * nm < 1.2e9);
}

// The tiled products' model of microseconds with steps of 128 columns.
Plan make_plan(int64_t T, int64_t M, int64_t N, int nm)
{
    Plan p{};
    p.pitch = (int)((M + 7) / 8 * 8);
    p.splits = 1;
    if (few_tokens(T, M, N, nm)) {
        // Waves a workgroup of 16 rows, one token, matrices from memory.  At 512 groups of rows one matrix
        // takes four and a pair eight: 8192 x 2048, 4096, 8192 and 28672 8.2, 11.2, 16.5 and 51.2 us with four,
        // 8.5, 10.5, 16.4 and 53.5 with eight; pairs of 8192 x 2048, 4096 and 8192 12.2, 17.6 and 28.3 with four,
        // 11.4, 17.3 and 28.5 with eight.  Above, both take four (28672 x 8192 44.7 and 47.0; pairs of 9216 x 4096
        // 20.9 and 23.7); below, eight (7168 x 8192 15.3 and 15.6, pairs of it 26.5 and 26.3; 4096 x 11008 14.4
        // with eight and 15.3 with sixteen) or, for few groups of long rows, sixteen (2048 x 8192 11.0 with eight
        // and 10.1).  The columns are split over workgroups where even sixteen waves a workgroup leave half of the
        // CUs idle: 1024 x 16384 11.0 over four, 13.1 over two.
        const int64_t groups = (M + 15) / 16, blocks = round64(N) / 512;
        p.few = 1;
        p.waves = groups >= (nm > 1 ? 513 : 512) ? 4 : groups >= 128 && groups < 256 && blocks >= 16 ? 16 : 8;
        while (p.splits < 16 && groups * p.splits < 128 && blocks >= (int64_t)p.waves * p.splits * 2) p.splits *= 2;
        if (p.splits > 1 && groups * p.splits < 256 && blocks >= (int64_t)p.waves * p.splits * 2) p.splits *= 2;
    } else {
        double least = 1e300;
        for (int small = 0; small < 2; ++small) {
            const int bp = (small ? 128 : 256) / nm, bq = small ? 128 : 256;
            const int ntp = (int)((M + bp - 1) / bp), ntq = (int)((T + bq - 1) / bq);
            const int steps = (int)((round64(N) + 127) / 128), pairs = (steps + 1) / 2;
            if (small && (int64_t)ntp * ntq >= 1 << 22) continue;     // a launch takes fewer than 2^32 threads
            for (int sp = 1; sp <= 16 && sp <= pairs; ++sp) {
                const int64_t tiles = (int64_t)ntp * ntq * sp;
                const double st = 2.0 * ((pairs + sp - 1) / sp);
                double cost;
                if (!small) {
                    cost = (double)((tiles + 255) / 256) * (st * 1.45 + 10.0);
                } else {
                    const int64_t rest = tiles % 512;
                    cost = (double)(tiles / 512) * (st * 1.15 + 4.0) + (rest ? st * (rest <= 256 ? 0.8 : 1.15) + 4.0 : 0.0);
                }
                if (sp > 1) cost += 9.5 + 0.8e-6 * (double)M * T * nm * (sp + 1);
                if (cost < least) {
                    least = cost;
                    p.small = small; p.ntp = ntp; p.ntq = ntq; p.steps = steps; p.splits = sp;
                }
            }
        }
    }
    p.part_bytes = p.splits > 1 ? (size_t)p.splits * nm * T * p.pitch * sizeof(int) : 0;
    return p;
}

struct Call {
    int64_t T;
    int dtype, nm;
    const vq_i8matrix* W[2];
    const void* X; int64_t ldx;
    Epilogue epi;
};

// Whether a few-token product makes its own codes: one or two tokens that its threads' registers
// and LDS hold.  Matrices from memory, one token by 4096 x 11008: 14.4 us, 16.9 with the launch in
// front; 8192 x 2048, 7.6 and 9.4; two by 2048 x 8192, 11.7 and 12.1.  Four are the same either way.
bool own_codes(int64_t T, int64_t N, int waves, int nm)
{
    const int64_t chunks = (round64(N) / 8 + waves * 64 - 1) / (waves * 64);
    return N >= 8 && T <= 2 && chunks <= 4 && T * (round64(N) + kOwnPad) + waves * nm * 1024 <= kOwnBytes;
}

// Chunks of eight a lane and token where waves make the codes of a few short rows, four in all;
// 0 where they do not (8 by a pair of 8192 x 2048: 11.5 us, 14.6 with the launch in front).
int wave_codes(int64_t T, int64_t N, int waves, int nm)
{
    if (N < 8 || T * (round64(N) + kOwnPad) + (int64_t)waves * nm * (T > 16 ? 2 : 1) * 1024 > kOwnBytes) return 0;
    for (int nx : {1, 2, 4})
        if (N <= 512 * nx && T <= waves * (4 / nx)) return nx;
    return 0;
}

template <class T, int NT, bool PAIR>
void few_launch(const FewI8& f, int waves, bool own, int nx, hipStream_t st)
{
    const dim3 grid((unsigned)((f.M + 15) / 16), (unsigned)f.splits);
    const size_t lds = (size_t)waves * (PAIR ? 2 : 1) * NT * 256 * sizeof(int);
    if constexpr (NT == 1) {
        if (own) {
            const size_t all = lds + f.T * (f.ldx + kOwnPad);
            if (f.T == 1) hipLaunchKernelGGL((k_i8_few<T, 1, PAIR, 4, 1, 4>), grid, dim3(waves * 64), all, st, f);
            else hipLaunchKernelGGL((k_i8_few<T, 1, PAIR, PAIR ? 2 : 4, 2, 4>), grid, dim3(waves * 64), all, st, f);
            return;
        }
    }
    const size_t all = lds + f.T * (f.ldx + kOwnPad);
    switch (nx) {
    case 1: hipLaunchKernelGGL((k_i8_few<T, NT, PAIR, 4, -4, 1>), grid, dim3(waves * 64), all, st, f); break;
    case 2: hipLaunchKernelGGL((k_i8_few<T, NT, PAIR, 4, -2, 2>), grid, dim3(waves * 64), all, st, f); break;
    case 4: hipLaunchKernelGGL((k_i8_few<T, NT, PAIR, 4, -1, 4>), grid, dim3(waves * 64), all, st, f); break;
    default: hipLaunchKernelGGL((k_i8_few<T, NT, PAIR, 4, 0, 1>), grid, dim3(waves * 64), lds, st, f);
    }
}

template <class T, bool PAIR>
vq_status launch(const Call& c, const Plan& p, const Rows& rows, int* part, hipStream_t st)
{
    const int8_t* const x = rows.q;
    const float* const sx = rows.scale;
    const bool own = p.few && own_codes(c.T, rows.cols, p.waves, c.nm);
    const int nx = p.few && !own ? wave_codes(c.T, rows.cols, p.waves, c.nm) : 0;
    if (!own && nx == 0) VQ_TRY(rows_codes(rows, c.dtype, st));
    const vq_i8matrix& w = *c.W[0];
    const Scales s{sx, {w.scale, PAIR ? c.W[1]->scale : nullptr}};
    const int64_t ldx = round64(w.N);
    if (p.few) {
        const FewI8 f{{w.q, PAIR ? c.W[1]->q : nullptr}, w.ldq, x, ldx, rows, (int)w.M, (int)c.T, (int)(ldx / 64), p.splits, p.pitch, part, s, c.epi};
        if (c.T > 16) few_launch<T, 2, PAIR>(f, p.waves, false, nx, st);
        else few_launch<T, 1, PAIR>(f, p.waves, own, nx, st);
        VQ_LAUNCHED("k_i8_few");
    } else {
        I8Tile a{};
        a.t.P[0] = reinterpret_cast<const char*>(w.q);
        a.t.P[1] = PAIR ? reinterpret_cast<const char*>(c.W[1]->q) : a.t.P[0];
        a.t.Q[0] = a.t.Q[1] = reinterpret_cast<const char*>(x);
        a.t.ldp = (int)(w.ldq / 2); a.t.ldq = (int)(ldx / 2);
        a.t.kP = a.t.kQ = (int)(ldx / 2);
        a.t.np = (int)w.M; a.t.nq = (int)c.T;
        a.t.ntp = p.ntp; a.t.ntq = p.ntq;
        a.t.steps = a.t.seg_steps = p.steps;
        a.t.splits = p.splits; a.t.pitch = p.pitch;
        a.t.part = reinterpret_cast<float*>(part);
        a.t.epi = c.epi;
        a.s = s;
        // 64 tokens by 28672 x 8192, from memory, 70.7 us and 58.6 in turns, by 57344 x 8192 115 and 98, by a pair
        // of 32768 x 4096 65 and 56; two rounds of tiles, a pair of 57344 x 8192, 177 and 191
        a.turn = p.small && in_turn(a.t);
        const dim3 grid((unsigned)(p.ntp * p.ntq), (unsigned)p.splits);
        if (p.small) hipLaunchKernelGGL((k_i8_gemm<T, 4, 2, PAIR>), grid, dim3(kThreads), 0, st, a);
        else hipLaunchKernelGGL((k_i8_gemm<T, 8, 4, PAIR>), grid, dim3(kThreads), 0, st, a);
        VQ_LAUNCHED("k_i8_gemm");
    }
    if (p.splits > 1) {
        const Parts f{part, p.splits, (int)w.M, (int)c.T, p.pitch, c.epi, s};
        hipLaunchKernelGGL((k_i8_finish<T, PAIR>), dim3(grid_for(c.T * (p.pitch / 8), 256)), dim3(256), 0, st, f);
        VQ_LAUNCHED("k_i8_finish");
    }
    return VQ_OK;
}

size_t workspace(int64_t T, int64_t M, int64_t N, int nm)
{
    return align_up(T * round64(N)) + align_up(T * sizeof(float)) + align_up(make_plan(T, M, N, nm).part_bytes);
}

vq_status product(const Call& c, void* ws, hipStream_t st)
{
    const int64_t N = c.W[0]->N, ldx = round64(N);
    const Plan p = make_plan(c.T, c.W[0]->M, N, c.nm);
    char* at = static_cast<char*>(ws);
    int8_t* x = reinterpret_cast<int8_t*>(at);
    float* sx = reinterpret_cast<float*>(at += align_up(c.T * ldx));
    int* part = p.part_bytes ? reinterpret_cast<int*>(at += align_up(c.T * sizeof(float))) : nullptr;
    const Rows rows{c.X, c.T, c.ldx, (int)N, x, ldx, sx, odd_rows(c.X, c.ldx)};
    if (c.dtype == VQ_BF16) return c.nm > 1 ? launch<Bf16, true>(c, p, rows, part, st) : launch<Bf16, false>(c, p, rows, part, st);
    return c.nm > 1 ? launch<F16, true>(c, p, rows, part, st) : launch<F16, false>(c, p, rows, part, st);
}

// ---- argument checks ------------------------------------------------------------
vq_status check_sizes(const std::string& call, int64_t T, int64_t M, int64_t N)
{
    VQ_CHECK(T >= 0 && T <= kMaxI8Tokens, call + ": T must be in [0, 2^28]");
    VQ_CHECK(M >= 1 && M <= kMaxSize, call + ": M must be in [1, 2^20]");
    VQ_CHECK(N >= 1 && N <= kMaxColumns, call + ": N must be in [1, 2^17]");
    VQ_CHECK(T * std::max(M, N) <= ((int64_t)1 << 38), call + ": T * max(M, N) must be at most 2^38");
    return VQ_OK;
}

vq_status check_codes(const std::string& call, const char* what, const vq_i8matrix* w)
{
    VQ_CHECK(w, call + ": " + what + " is null");
    VQ_CHECK(w->q && w->scale, call + ": " + what + " has a null pointer");
    VQ_CHECK(aligned16(w->q), call + ": codes of " + what + " are not 16-byte aligned");
    VQ_CHECK(w->ldq % kRowBytes == 0 && w->ldq >= w->N && w->ldq <= 2 * kMaxLd,
             call + ": ldq of " + what + " must be a multiple of 64, at least N and at most 2^22");
    VQ_CHECK(reinterpret_cast<uintptr_t>(w->scale) % 4 == 0, call + ": scale of " + what + " is not aligned to its elements");
    return VQ_OK;
}

vq_status check_types(const std::string& call, int dtype, int act)
{
    VQ_CHECK(dtype == VQ_BF16 || dtype == VQ_F16, call + ": dtype must be VQ_BF16 or VQ_F16");
    VQ_CHECK(act >= VQ_ACT_NONE && act <= VQ_ACT_SIGMOID, call + ": unknown activation");
    return VQ_OK;
}

}  // namespace
}  // namespace vq

using namespace vq;

extern "C" {

vq_status vq_quantize_rows(int64_t rows, int64_t cols, int dtype, const void* X, int64_t ldx, int8_t* q, int64_t ldq,
                           float* scale, void* stream)
{
    const std::string call = "vq_quantize_rows";
    VQ_CHECK(rows >= 0 && rows <= kMaxI8Tokens, call + ": rows must be in [0, 2^28]");
    VQ_CHECK(cols >= 1 && cols <= kMaxSize, call + ": cols must be in [1, 2^20]");
    VQ_CHECK(dtype == VQ_BF16 || dtype == VQ_F16 || dtype == VQ_F32, call + ": unknown dtype");
    if (rows == 0) return VQ_OK;
    VQ_CHECK(X && q && scale, call + ": null pointer");
    VQ_TRY(check_ld(call, "X", X, ldx, cols));
    VQ_CHECK(dtype != VQ_F32 || reinterpret_cast<uintptr_t>(X) % 4 == 0, call + ": X is not aligned to its elements");
    VQ_CHECK(reinterpret_cast<uintptr_t>(scale) % 4 == 0, call + ": scale is not aligned to its elements");
    VQ_CHECK(aligned16(q) && ldq % kRowBytes == 0 && ldq >= cols && ldq <= ((int64_t)1 << 40),
             call + ": q must be 16-byte aligned and ldq a multiple of 64, at least cols");
    VQ_TRY(check_apart(call, {q, scale}, {X}));
    VQ_TRY(check_device());
    VQ_MATRIX(X, rows, cols, ldx, call.c_str(), "X");
    TimedRegion tr("quantize_rows", 0, as_stream(stream));
    return rows_codes({X, rows, ldx, (int)cols, q, ldq, scale, dtype != VQ_F32 && odd_rows(X, ldx)}, dtype, as_stream(stream));
}

size_t vq_linear_i8_workspace_bytes(int64_t M, int64_t N, int64_t T)
{
    if (check_sizes("vq_linear_i8", T, M, N) != VQ_OK || T == 0) return 0;
    return workspace(T, M, N, 1);
}

vq_status vq_linear_i8(const vq_i8matrix* W, int64_t T, int dtype, int act, const void* X, int64_t ldx, const void* bias,
                       const void* R, int64_t ldr, void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_linear_i8";
    VQ_TRY(check_types(call, dtype, act));
    VQ_TRY(check_codes(call, "W", W));
    const int64_t M = W->M, N = W->N;
    VQ_TRY(check_sizes(call, T, M, N));
    if (T == 0) return VQ_OK;
    VQ_CHECK(X && Y, "vq_linear_i8: null pointer");
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "bias", bias, M, M));
    VQ_TRY(check_ld(call, "R", R, ldr, M));
    VQ_TRY(check_ld(call, "Y", Y, ldy, M));
    VQ_TRY(check_apart(call, {Y}, {X, W->q, W->scale, bias}));
    VQ_CHECK(Y != R || ldy == ldr, "vq_linear_i8: Y in place of R needs R's leading dimension");
    VQ_TRY(check_workspace(call, ws, ws_bytes, workspace(T, M, N, 1)));
    VQ_TRY(check_device());
    VQ_MATRIX(X, T, N, ldx, call, "X");
    VQ_VALUES(W->scale, M, false, call, "scale of W");
    VQ_MATRIX(bias, 1, M, M, call, "bias");
    VQ_MATRIX(R, T, M, ldr, call, "R");
    TimedRegion tr("linear_i8", 0, as_stream(stream));
    return product({T, dtype, 1, {W, nullptr}, X, ldx, {act, {bias, nullptr}, R, Y, {nullptr, nullptr}, ldr, ldy, 0}}, ws, as_stream(stream));
}

size_t vq_gated_i8_workspace_bytes(int64_t M, int64_t N, int64_t T)
{
    if (check_sizes("vq_gated_i8", T, M, N) != VQ_OK || T == 0) return 0;
    return workspace(T, M, N, 2);
}

vq_status vq_gated_i8(const vq_i8matrix* Wg, const vq_i8matrix* Wu, int64_t T, int dtype, int act, const void* X, int64_t ldx,
                      const void* bg, const void* bu, void* H, int64_t ldh, void* ws, size_t ws_bytes, void* stream)
{
    const char* call = "vq_gated_i8";
    VQ_TRY(check_types(call, dtype, act));
    VQ_TRY(check_codes(call, "Wg", Wg));
    VQ_TRY(check_codes(call, "Wu", Wu));
    VQ_CHECK(Wg->M == Wu->M && Wg->N == Wu->N && Wg->ldq == Wu->ldq, "vq_gated_i8: Wg and Wu must have the same M, N and ldq");
    const int64_t M = Wg->M, N = Wg->N;
    VQ_TRY(check_sizes(call, T, M, N));
    if (T == 0) return VQ_OK;
    VQ_CHECK(X && H, "vq_gated_i8: null pointer");
    VQ_TRY(check_ld(call, "X", X, ldx, N));
    VQ_TRY(check_ld(call, "bg", bg, M, M));
    VQ_TRY(check_ld(call, "bu", bu, M, M));
    VQ_TRY(check_ld(call, "H", H, ldh, M));
    VQ_TRY(check_apart(call, {H}, {X, Wg->q, Wg->scale, Wu->q, Wu->scale, bg, bu}));
    VQ_TRY(check_workspace(call, ws, ws_bytes, workspace(T, M, N, 2)));
    VQ_TRY(check_device());
    VQ_MATRIX(X, T, N, ldx, call, "X");
    VQ_VALUES(Wg->scale, M, false, call, "scale of Wg");
    VQ_VALUES(Wu->scale, M, false, call, "scale of Wu");
    VQ_MATRIX(bg, 1, M, M, call, "bg");
    VQ_MATRIX(bu, 1, M, M, call, "bu");
    TimedRegion tr("gated_i8", 0, as_stream(stream));
    return product({T, dtype, 2, {Wg, Wu}, X, ldx, {act, {bg, bu}, nullptr, H, {nullptr, nullptr}, 0, ldh, 0}}, ws, as_stream(stream));
}

}  // extern "C"
