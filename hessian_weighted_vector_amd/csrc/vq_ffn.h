// Shared by the feed-forward kernels (dense products, few-token products,
// products from the compressed form): 16-bit element types, activations and
// the epilogue that every forward product ends in.  Not part of the ABI.
#pragma once

#include "vq_internal.h"

#include <initializer_list>

namespace vq {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// A call's workspace: large enough, and where one is needed on a 16-byte boundary, since
// its parts and copies are written and read 16 bytes at a time.
inline vq_status check_workspace(const char* call, const void* ws, size_t ws_bytes, size_t need)
{
    if (need == 0) return VQ_OK;
    VQ_WS(ws && ws_bytes >= need, std::string(call) + ": workspace too small");
    VQ_CHECK(aligned16(ws), std::string(call) + ": workspace is not 16-byte aligned");
    return VQ_OK;
}

constexpr int64_t kMaxSize = 1 << 20;    // of a matrix's rows and columns

inline vq_status check_ld(const std::string& call, const char* what, const void* p, int64_t ld, int64_t cols)
{
    VQ_CHECK(p == nullptr || ld >= cols, call + ": leading dimension of " + what + " is below its row length");
    VQ_CHECK(p == nullptr || ld <= ((int64_t)1 << 40), call + ": leading dimension of " + what + " is too large");
    VQ_CHECK((reinterpret_cast<uintptr_t>(p) & 1u) == 0, call + ": " + what + " is not aligned to its elements");
    return VQ_OK;
}

// No output (null ones aside) begins where an input or another output does.
inline vq_status check_apart(const std::string& call, std::initializer_list<const void*> outputs, std::initializer_list<const void*> inputs)
{
    for (auto o = outputs.begin(); o != outputs.end(); ++o) {
        if (!*o) continue;
        for (const void* i : inputs) VQ_CHECK(*o != i, call + ": outputs may not alias inputs");
        for (auto p = outputs.begin(); p != o; ++p) VQ_CHECK(*o != *p, call + ": outputs may not alias each other");
    }
    return VQ_OK;
}

#define VQ_MATRIX(a, rows, cols, ld, call, what) \
    VQ_TRY(check_matrix((a), (rows), (cols), (ld), dtype, (call), (what), as_stream(stream)))

// 16-bit element types: storage E, vectors of four and eight, and the
// 16 x 16 x 32 matrix instruction with float32 accumulation.  Stores round to
// nearest even once, from float32.
struct Bf16 {
    static constexpr int kDtype = VQ_BF16;
    typedef f32x4 Acc;                          // four sums
    typedef __bf16 E;
    typedef __bf16 V4 __attribute__((ext_vector_type(4)));
    typedef __bf16 V8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mfma(V8 a, V8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ V4 lds_tr(__attribute__((address_space(3))) V4* p) { return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(p); }
};
struct F16 {
    static constexpr int kDtype = VQ_F16;
    typedef f32x4 Acc;
    typedef _Float16 E;
    typedef _Float16 V4 __attribute__((ext_vector_type(4)));
    typedef _Float16 V8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mfma(V8 a, V8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ V4 lds_tr(__attribute__((address_space(3))) V4* p)
    {
        typedef short S4 __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(V4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) S4*)p));
    }
};

// ---- activations --------------------------------------------------------
// Dense products: the result is rounded to 16 bits, so the exponential and the
// reciprocal are the hardware's (a few float32 ulp; results below about 1e-36 may be
// 0).  The tanh form of GELU is z * logistic(2 v), which needs no tanh and loses
// nothing for negative z.
__device__ inline float logistic_fast(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluC = 0.79788456080286536f;       // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// erfc(z / -sqrt 2) / 2 = the normal distribution function, without the
// cancellation of 1 + erf in the lower tail.
__device__ inline float normal_cdf(float z) { return 0.5f * erfcf(-kSqrtHalf * z); }

// act of eight values; the choice is made once for all.  z * logistic tends to 0
// where the logistic is 0; NaN stays NaN.
__device__ inline void activate(int act, float (&z)[8])
{
#define VQ_EACH(EXPR)                                 \
    _Pragma("unroll") for (int i = 0; i < 8; ++i)     \
    {                                                 \
        const float v = z[i];                         \
        z[i] = (EXPR);                                \
    }
    switch (act) {
    case VQ_ACT_RELU: VQ_EACH(v > 0.0f ? v : (v <= 0.0f ? 0.0f : v)) break;
    case VQ_ACT_SILU: VQ_EACH(v * logistic_fast(v)) break;
    case VQ_ACT_GELU: VQ_EACH(v * normal_cdf(v)) break;
    case VQ_ACT_GELU_TANH: VQ_EACH(v * logistic_fast(2.0f * kGeluC * (v + kGeluA * v * v * v))) break;
    case VQ_ACT_SIGMOID: VQ_EACH(logistic_fast(v)) break;
    default: break;
    }
#undef VQ_EACH
}

// z times the logistic function of v, to float32's smallest values: the exponential is
// never of a positive argument, so where it is tiny the result is too, and not 0.
__device__ inline float times_logistic(float z, float v)
{
    const float e = expf(-fabsf(v));
    return (v < 0.0f ? z * e : z) / (1.0f + e);
}

// The activations in full float32 accuracy (float32 results).  An error of the exponential's
// argument is the result's relative error, so the tanh form's argument takes three
// roundings (z^2, multiply-add, product) and two rounded constants: 4 * 2^-24 of it.
__device__ inline float act_full(int act, float z)
{
    switch (act) {
    case VQ_ACT_RELU: return z > 0.0f ? z : (z <= 0.0f ? 0.0f : z);
    case VQ_ACT_SILU: return times_logistic(z, z);
    case VQ_ACT_GELU: return z * normal_cdf(z);
    case VQ_ACT_GELU_TANH: return times_logistic(z, z * fmaf(2.0f * kGeluC * kGeluA, z * z, 2.0f * kGeluC));
    case VQ_ACT_SIGMOID: return times_logistic(1.0f, z);
    default: return z;
    }
}

// z -> act'(z) and, where wanted, a = act(z), of eight values.  ReLU's derivative at
// 0 is 0; NaN stays NaN in both.
template <bool VALUE>
__device__ inline void act_grad(int act, float (&z)[8], float (&a)[8])
{
#define VQ_EACH(BODY)                                 \
    _Pragma("unroll") for (int i = 0; i < 8; ++i)     \
    {                                                 \
        const float v = z[i];                         \
        float val, der;                               \
        BODY;                                         \
        z[i] = der;                                   \
        if (VALUE) a[i] = val;                        \
    }
    switch (act) {
    case VQ_ACT_RELU: VQ_EACH(val = v > 0.0f ? v : (v <= 0.0f ? 0.0f : v); der = v > 0.0f ? 1.0f : val) break;
    case VQ_ACT_SILU: VQ_EACH(const float s = logistic_fast(v); val = v * s; der = s * (1.0f + v * (1.0f - s))) break;
    case VQ_ACT_GELU: VQ_EACH(const float c = normal_cdf(v); val = v * c; der = c + v * kInvSqrt2Pi * __expf(-0.5f * v * v)) break;
    case VQ_ACT_GELU_TANH:
        // (1 - s) is 0 long before v^2 reaches the bound, which keeps 0 * inf away
        VQ_EACH(const float q = v * v; const float s = logistic_fast(2.0f * kGeluC * v * (1.0f + kGeluA * q)); val = v * s;
                der = s + val * (1.0f - s) * (2.0f * kGeluC) * (1.0f + 3.0f * kGeluA * fminf(q, 1e6f)))
        break;
    case VQ_ACT_SIGMOID:
        // the derivative is even, and from e = exp(-|v|) nothing cancels: e / (1 + e)^2
        VQ_EACH(const float e = __expf(-fabsf(v)); const float s = __builtin_amdgcn_rcpf(1.0f + e); val = v < 0.0f ? e * s : s;
                der = e * s * s)
        break;
    default: VQ_EACH(val = v; der = 1.0f)
    }
#undef VQ_EACH
}

// ---- epilogue -----------------------------------------------------------
// Output element (token t, feature m) from float32 sums:
//   one product:  Z = s + bias, Y = act(Z) + R
//   gated pair:   G = s0 + bias0, U = s1 + bias1, Y = act(G) * U
// Z (or G and U) are also stored where the caller keeps them.  Each stored
// value is rounded once, from float32; the activation reads the unrounded sums.
struct Epilogue {
    int act;
    const void* bias[2];     // nullable
    const void* R;           // nullable
    void* Y;
    void* Z[2];              // nullable
    int64_t ldr, ldy, ldz;
};

// Eight 16-bit elements at any element's address.  A 16-byte load runs at full rate
// from any multiple of four bytes and at less than half from others, so it starts at
// the word that holds the first element, and the last element comes by itself.
struct Words {
    uint32_t q[4];
    uint16_t last;
    __device__ __forceinline__ void load(const void* p)
    {
        // by pointer arithmetic: an address made from a number would be loaded as of any memory, not the GPU's alone
        const char* const at = static_cast<const char*>(p);
        __builtin_memcpy(q, __builtin_assume_aligned(at - (reinterpret_cast<uintptr_t>(p) & 2), 4), 16);
        last = *reinterpret_cast<const uint16_t*>(at + 14);
    }
    // The elements; p as loaded from, or less by whole words.
    __device__ __forceinline__ uint4 get(const void* p) const
    {
        const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(p) & 2;
        return {__builtin_amdgcn_alignbyte(q[1], q[0], s), __builtin_amdgcn_alignbyte(q[2], q[1], s),
                __builtin_amdgcn_alignbyte(q[3], q[2], s), __builtin_amdgcn_alignbyte(last, q[3], s)};
    }
};

// Whether some of a matrix's rows begin at an odd element.
inline bool odd_rows(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 2) || (ld & 1); }

// Reads or writes features m .. m+7 of row t (those below M): one 16-byte access
// where all eight exist, at any element-aligned address (the hardware takes
// unaligned vector accesses; aligned rows run at full speed).
template <class T>
__device__ inline void store8(void* base, int64_t ld, int64_t t, int m, int M, const float (&v)[8])
{
    typename T::E* o = static_cast<typename T::E*>(base) + t * ld + m;
    typename T::V8 w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (typename T::E)v[i];
    if (m + 8 <= M) {
        __builtin_memcpy(o, &w, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (m + i < M) o[i] = w[i];
    }
}

template <class T, bool ODD = false>
__device__ inline void load8(const void* base, int64_t ld, int64_t t, int m, int M, float (&v)[8])
{
    const typename T::E* p = static_cast<const typename T::E*>(base) + t * ld + m;
    if (m + 8 <= M) {
        typename T::V8 w;
        if (ODD) {
            Words a;
            a.load(p);
            const uint4 u = a.get(p);
            __builtin_memcpy(&w, &u, 16);
        } else {
            __builtin_memcpy(&w, p, 16);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = m + i < M ? (float)p[i] : 0.0f;
    }
}

// Features m .. m+7 of token t (those below M).
template <class T>
__device__ inline void epilogue_one(const Epilogue& e, int64_t t, int m, int M, float (&z)[8])
{
    if (e.bias[0]) {
        float b[8];
        load8<T>(e.bias[0], 0, 0, m, M, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += b[i];
    }
    if (e.Z[0]) store8<T>(e.Z[0], e.ldz, t, m, M, z);
    activate(e.act, z);
    if (e.R) {
        float r[8];
        load8<T>(e.R, e.ldr, t, m, M, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += r[i];
    }
    store8<T>(e.Y, e.ldy, t, m, M, z);
}

template <class T>
__device__ inline void epilogue_pair(const Epilogue& e, int64_t t, int m, int M, float (&g)[8], float (&u)[8])
{
    float b[8];
    if (e.bias[0]) {
        load8<T>(e.bias[0], 0, 0, m, M, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += b[i];
    }
    if (e.bias[1]) {
        load8<T>(e.bias[1], 0, 0, m, M, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += b[i];
    }
    if (e.Z[0]) {
        store8<T>(e.Z[0], e.ldz, t, m, M, g);
        store8<T>(e.Z[1], e.ldz, t, m, M, u);
    }
    activate(e.act, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] *= u[i];
    store8<T>(e.Y, e.ldy, t, m, M, g);
}

// ---- operands -------------------------------------------------------------
constexpr int64_t kMaxLd = 1 << 21;      // tile offsets stay below 2^31 bytes

// Hands out workspace slices; with no base it only counts.  Every call counts
// first and compares with the caller's bytes.
struct Arena {
    char* base;
    size_t used = 0;
    void* take(size_t bytes)
    {
        char* p = base + used;
        used += align_up(bytes);
        return base ? p : nullptr;
    }
};

inline int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

struct Mat {
    const void* p;
    int64_t rows, cols, ld;
};

// Whether the tiled product's 16-byte loads can read the matrix as it is.
inline bool loads_ok(const Mat& m) { return aligned16(m.p) && m.ld % 8 == 0 && m.cols % 8 == 0 && m.ld <= kMaxLd; }

struct Pack {
    const uint16_t* s;
    uint16_t* o;
    int64_t rows, ld, ldp;
    int cols;
    int odd;                   // some rows begin at an odd element
};
struct Packs {
    Pack m[3];
    int count = 0;
    int blocks = 0;            // a matrix's
};

// Block `block` of `blocks` of the copy of m.
__device__ __forceinline__ void pack_rows(const Pack& m, int block, int blocks)
{
    const int64_t per = m.ldp / 8;
    const int64_t n = m.rows * per;
    for (int64_t e = (int64_t)block * 256 + threadIdx.x; e < n; e += (int64_t)blocks * 256) {
        const int64_t r = e / per;
        const int c = (int)(e - r * per) * 8;
        const uint16_t* p = m.s + r * m.ld + c;
        alignas(16) uint16_t v[8];
        if (c + 8 <= m.cols) {
            if (m.odd) {
                Words w;
                w.load(p);
                const uint4 u = w.get(p);
                __builtin_memcpy(v, &u, 16);
            } else {
                __builtin_memcpy(v, p, 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < m.cols ? p[i] : (uint16_t)0;
        }
        *reinterpret_cast<uint4*>(m.o + r * m.ldp + c) = *reinterpret_cast<const uint4*>(v);
    }
}

// The copies in one launch; blocks of a matrix whose copy has n chunks of eight.
vq_status pack_launch(const Packs& list, hipStream_t st);
inline int pack_blocks(int64_t n) { return (int)((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384); }

// ---- the tiled product --------------------------------------------------
// out[q, p] = sum over segments and k of P[p, k] Q[q, k] (p contiguous in the
// output).  An operand is k-contiguous (element (r, k) at r * ld + k) or
// k-strided (element (r, k) at k * ld + r).  Operands that reach the kernel
// have 16-byte aligned rows (base, ld) and a multiple of eight elements along
// their contiguous axis.
enum GemmKind {
    GEMM_LINEAR,    // both k-contiguous; linear epilogue
    GEMM_GATED,     // both k-contiguous; P is a pair, gated epilogue
    GEMM_DX,        // P k-strided, Q k-contiguous; two segments where gated
    GEMM_DW         // both k-strided; two outputs (Q[0], Q[1]) where gated
};

struct GemmArgs {
    GemmKind kind;
    int dtype;
    int np, nq;                 // features (of each matrix of a pair), output rows
    int nseg, nbatch;           // segments summed; outputs in one launch
    int64_t kP, kQ;             // valid k of each operand (kP = kQ up to zero padding)
    const void* P[2];
    const void* Q[2];
    int64_t ldp, ldq;
    int wp, wq;                 // valid elements along a k-strided operand's rows
    Epilogue epi;
    void* Y2;                   // second output (nbatch = 2)
};

size_t gemm_workspace(GemmKind kind, int64_t np, int64_t nq, int64_t K, int nseg, int nbatch);
vq_status gemm_launch(const GemmArgs& a, void* ws, size_t ws_bytes, hipStream_t st);

// A product's sizes: K is the smaller of its operands' valid k.
struct GemmSize {
    GemmKind kind;
    int64_t np, nq, K;
    int nseg, nbatch;
};

// Bias gradients: db = the sum of n partial rows of M, for up to two outputs.
struct BiasSum {
    const float* part[2];
    void* db[2];
    int64_t n;
    int M, outputs;
};
vq_status bias_sum_launch(int dtype, const BiasSum& b, hipStream_t st);

// A GEMM_DX and a GEMM_DW product and the bias gradients (outputs may be 0), in one
// launch where that is faster.
size_t gemm_two_workspace(const GemmSize& x, const GemmSize& w);
vq_status gemm_two_launch(const GemmArgs& x, const GemmArgs& w, const BiasSum& b, void* ws, size_t ws_bytes, hipStream_t st);

// Adds float32 parts [splits][matrices][nq][pitch] in order and applies the epilogue.
vq_status finish_parts(int dtype, bool pair, const float* part, int splits, int np, int nq, int pitch, const Epilogue& e,
                       hipStream_t st);

// ---- few tokens -----------------------------------------------------------
// The forward products for up to 32 tokens, any strides and alignment; whether that is the faster way.
struct FewArgs {
    int64_t T, M, K;
    int dtype, nm;
    const void* X; int64_t ldx;
    const void* W[2]; int64_t ldw;
    Epilogue epi;
};
bool few_tokens(int64_t T, int64_t M, int64_t K, int nm);
size_t few_workspace(int64_t T, int64_t M, int64_t K, int nm);
vq_status few_product(const FewArgs& f, void* ws, hipStream_t st);

}  // namespace vq
