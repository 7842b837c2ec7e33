// AdamW over many tensors in one launch (vq_adamw_plan, vq_adamw).
//
//   g = scale * grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in float32, p rounded once where it is kept in 16 bits.  Each element is read and
// written once and nothing is shared, so bytes bound it: 28 a parameter with a float32
// master, 16-bit copy and gradient, and 32-bit moments; 16 with 8-bit moments.
//
// The plan is a table on the GPU: one entry a tensor and one a chunk of 4096
// elements, so a workgroup finds its work in two dependent loads, however many
// tensors there are, and no tensor's end leaves more than a part of one chunk idle.
// Three tensors of 45.1 M elements (bf16, masters): 700 us (5.4 TB/s; a large read reaches 6.2, a copy 4.9),
// 411 us with 8-bit moments (5.3 TB/s); 256 of up to 8192 elements 5.8 to 6.2 us.
//
// 8-bit moments.  256 consecutive elements of a tensor share a float32 scale: m is kept
// as e4m3 codes of m / s with s = max|m| / 448, and v as codes of sqrt(v) / s with s =
// max sqrt(v) / 448, since the root has half of v's exponents and is what the step
// divides by.  A code is off by at most 2^-4 of its value (2^-10 s below 2^-6 s).  A
// root that is not zero is stored as at least the smallest code: a later step would
// divide by it.  The step itself uses the moments before they are rounded.  A wave's
// four elements a lane are one block, so its largest value comes from lane exchanges.
#include "vq_internal.h"

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <type_traits>
#include <vector>

namespace vq {
namespace {

constexpr int kBlock = 256;              // elements that share a scale; a wave's at a time
constexpr int kChunk = 4096;             // elements of a workgroup
constexpr int kPerWave = kChunk / kBlock / 4;
constexpr float kTop = 448.0f;           // the largest e4m3 value
constexpr float kLeast = 0x1p-9f;        // the smallest positive one

struct Chunk {
    uint32_t tensor, index;
};

struct Coefficients {
    float b1, c1, b2, c2;                // c = 1 - b, rounded from double
    float decay, rate, root, eps;        // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};

struct Args {
    const vq_adamw_tensor* tensors;
    const Chunk* chunks;
    const Coefficients* from_device;     // or null: c
    const float* grad_scale;             // or null
    Coefficients c;
};

template <class E>
__device__ __forceinline__ void load4(const void* p, int64_t i, int n, float (&v)[4])
{
    const E* e = static_cast<const E*>(p) + i;
    typedef E V __attribute__((ext_vector_type(4)));
    V w = {};
    if (n >= 4) {
        __builtin_memcpy(&w, e, sizeof(w));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) w[k] = e[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (float)w[k];
}

template <class E>
__device__ __forceinline__ void store4(void* p, int64_t i, int n, const float (&v)[4])
{
    E* e = static_cast<E*>(p) + i;
    typedef E V __attribute__((ext_vector_type(4)));
    V w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (E)v[k];
    if (n >= 4) {
        __builtin_memcpy(e, &w, sizeof(w));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) e[k] = w[k];
    }
}

__device__ __forceinline__ uint32_t load_codes(const void* p, int64_t i, int n)
{
    const uint8_t* e = static_cast<const uint8_t*>(p) + i;
    uint32_t w = 0;
    if (n >= 4) {
        __builtin_memcpy(&w, e, 4);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) w |= (uint32_t)e[k] << (8 * k);
    }
    return w;
}

__device__ __forceinline__ void store_codes(void* p, int64_t i, int n, uint32_t w)
{
    uint8_t* e = static_cast<uint8_t*>(p) + i;
    if (n >= 4) {
        __builtin_memcpy(e, &w, 4);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) e[k] = (uint8_t)(w >> (8 * k));
    }
}

__device__ __forceinline__ void decode(uint32_t w, float (&v)[4])
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
}

// Codes of the quotients by scale, as float32 divides.  ROOT: of the elements' roots.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode_divided(const float (&x)[4], float scale)
{
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float v = ROOT ? sqrtf(x[k]) : x[k];
        y[k] = scale > 0.0f ? v / scale : v;
        y[k] = y[k] > kTop ? kTop : y[k] < -kTop ? -kTop : y[k];     // the quotient's rounding
        if (ROOT && x[k] > 0.0f && y[k] < kLeast) y[k] = kLeast;
    }
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
}

// The wave's block in codes, and its scale; with ROOT of the roots of x.  NaN stays NaN (the
// maximum passes over it).
//
// Four divisions and four exact roots a lane would take as long as the memory.  The hardware's
// reciprocal and root give the quotients within 2^-22; both ends of an interval of 2^-21 around
// each are coded, and where they agree the quotient's code is theirs.  The others, a few in a
// million, and blocks whose largest is so small that a reciprocal or a root could be
// subnormal, are divided.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(const float (&x)[4], float& scale)
{
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    scale = (ROOT ? sqrtf(top) : top) * (1.0f / kTop);
    if (!(top >= 0x1p-90f && top < INFINITY)) return encode_divided<ROOT>(x, scale);
    const float r = __builtin_amdgcn_rcpf(scale);
    float lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float y = (ROOT ? __builtin_amdgcn_sqrtf(x[k]) : x[k]) * r;
        const float least = ROOT && x[k] > 0.0f ? kLeast : -INFINITY;
        lo[k] = y * (1.0f - 0x1p-21f);
        hi[k] = __builtin_amdgcn_fmed3f(y * (1.0f + 0x1p-21f), -kTop, kTop);      // a number for NaN: the ends differ
        if (ROOT) {
            lo[k] = lo[k] < least ? least : lo[k];
            hi[k] = hi[k] < least ? least : hi[k];
        }
    }
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(lo[0], lo[1], 0, false), b = __builtin_amdgcn_cvt_pk_fp8_f32(hi[0], hi[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(lo[2], lo[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(hi[2], hi[3], b, true);
    return a == b ? (uint32_t)a : encode_divided<ROOT>(x, scale);
}

// P: the parameter's type (the master is float32); G: the gradient's.
template <class P, class G, bool MASTER, int BITS>
__global__ __launch_bounds__(256) void k_adamw(const Args a)
{
    const Chunk ch = a.chunks[blockIdx.x];
    const vq_adamw_tensor t = a.tensors[ch.tensor];
    const Coefficients c = a.from_device ? *a.from_device : a.c;
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t begin = (int64_t)ch.index * kChunk + wave * kBlock;
    float g[kPerWave][4], p[kPerWave][4], m[kPerWave][4], v[kPerWave][4], sm[kPerWave], sv[kPerWave];
    uint32_t cm[kPerWave], cv[kPerWave];
    // every load before the first use
#pragma unroll
    for (int b = 0; b < kPerWave; ++b) {
        const int64_t i = begin + b * 4 * kBlock + lane * 4;
        const int n = i < t.n ? (t.n - i < 4 ? (int)(t.n - i) : 4) : 0;
        load4<G>(t.grad, i, n, g[b]);
        if (MASTER) load4<float>(t.master, i, n, p[b]);
        else load4<P>(t.param, i, n, p[b]);
        if (BITS == 32) {
            load4<float>(t.m, i, n, m[b]);
            load4<float>(t.v, i, n, v[b]);
        } else {
            cm[b] = load_codes(t.m, i, n);
            cv[b] = load_codes(t.v, i, n);
            const int64_t s = i / kBlock;
            sm[b] = i - lane * 4 < t.n ? t.m_scale[s] : 0.0f;
            sv[b] = i - lane * 4 < t.n ? t.v_scale[s] : 0.0f;
        }
    }
#pragma unroll
    for (int b = 0; b < kPerWave; ++b) {
        const int64_t first = begin + b * 4 * kBlock, i = first + lane * 4;
        if (first >= t.n) break;                              // the wave's own blocks, all lanes
        const int n = i < t.n ? (t.n - i < 4 ? (int)(t.n - i) : 4) : 0;
        if (BITS == 8) {
            decode(cm[b], m[b]);
            decode(cv[b], v[b]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[b][k] *= sm[b];
                const float r = v[b][k] * sv[b];
                v[b][k] = r * r;
            }
        }
        // the step's root and reciprocal are the hardware's, off by a unit in the last place each; the moments are not
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float gk = g[b][k] * gs;
            m[b][k] = c.b1 * m[b][k] + c.c1 * gk;
            v[b][k] = c.b2 * v[b][k] + c.c2 * (gk * gk);
            const float root = __builtin_amdgcn_sqrtf(v[b][k]);
            p[b][k] = p[b][k] * c.decay - c.rate * (m[b][k] * __builtin_amdgcn_rcpf(root * c.root + c.eps));
        }
        if (MASTER) store4<float>(t.master, i, n, p[b]);
        store4<P>(t.param, i, n, p[b]);
        if (BITS == 32) {
            store4<float>(t.m, i, n, m[b]);
            store4<float>(t.v, i, n, v[b]);
        } else {
            if (n < 4) {                                      // elements past the tensor's end have no part in the scale
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k >= n) m[b][k] = v[b][k] = 0.0f;
            }
            float s0, s1;
            const uint32_t w0 = encode<false>(m[b], s0), w1 = encode<true>(v[b], s1);
            store_codes(t.m, i, n, w0);
            store_codes(t.v, i, n, w1);
            if (lane == 0) {
                t.m_scale[first / kBlock] = s0;
                t.v_scale[first / kBlock] = s1;
            }
        }
    }
}

// New gradients of tensors first .. first + count, taken from the kernel's own arguments, so
// that nothing on the host has to outlive the call.
constexpr int kPointers = 448;
struct GradPointers {
    const void* grad[kPointers];
    int64_t first;
    int count;
};

__global__ __launch_bounds__(512) void k_adamw_grads(const GradPointers a, vq_adamw_tensor* tensors)
{
    if ((int)threadIdx.x < a.count) tensors[a.first + threadIdx.x].grad = a.grad[threadIdx.x];
}

Coefficients coefficients(double lr, double b1, double b2, double eps, double wd, double power1, double power2)
{
    Coefficients c;
    c.b1 = (float)b1; c.c1 = (float)(1 - b1);
    c.b2 = (float)b2; c.c2 = (float)(1 - b2);
    c.decay = (float)(1 - lr * wd);
    c.rate = (float)(lr / (1 - power1));
    c.root = (float)(1 / std::sqrt(1 - power2));
    c.eps = (float)eps;
    return c;
}

// The step's number on the GPU, for captured graphs: counts it and makes the coefficients.
__global__ void k_adamw_tick(int64_t* step, const float* lr_from, double lr, double b1, double b2, double eps, double wd,
                             Coefficients* out)
{
    if (threadIdx.x) return;
    const int64_t t = *step + 1;
    *step = t;
    if (lr_from) lr = (double)*lr_from;
    Coefficients c;
    c.b1 = (float)b1; c.c1 = (float)(1 - b1);
    c.b2 = (float)b2; c.c2 = (float)(1 - b2);
    c.decay = (float)(1 - lr * wd);
    c.rate = (float)(lr / (1 - pow(b1, (double)t)));
    c.root = (float)(1 / sqrt(1 - pow(b2, (double)t)));
    c.eps = (float)eps;
    *out = c;
}

size_t tensors_bytes(int64_t count) { return align_up((size_t)count * sizeof(vq_adamw_tensor)); }

template <class P, class G, bool MASTER>
void launch_bits(const Args& a, int64_t chunks, int bits, hipStream_t st)
{
    const dim3 grid((unsigned)chunks);
    if (bits == 32) hipLaunchKernelGGL((k_adamw<P, G, MASTER, 32>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_adamw<P, G, MASTER, 8>), grid, dim3(256), 0, st, a);
}

template <class P, class G>
void launch_master(const Args& a, const vq_adamw_plan_t& p, hipStream_t st)
{
    if constexpr (!std::is_same<P, float>::value) {
        if (p.has_master) return launch_bits<P, G, true>(a, p.chunks, p.state_bits, st);
    }
    launch_bits<P, G, false>(a, p.chunks, p.state_bits, st);
}

template <class P>
void launch_grad(const Args& a, const vq_adamw_plan_t& p, hipStream_t st)
{
    if (p.grad_dtype == VQ_BF16) launch_master<P, __bf16>(a, p, st);
    else if (p.grad_dtype == VQ_F16) launch_master<P, _Float16>(a, p, st);
    else launch_master<P, float>(a, p, st);
}

bool known(int dtype) { return dtype == VQ_BF16 || dtype == VQ_F16 || dtype == VQ_F32; }
size_t size_of(int dtype) { return dtype == VQ_F32 ? 4 : 2; }
bool off(const void* p, size_t align) { return reinterpret_cast<uintptr_t>(p) % align != 0; }

int64_t chunks_of(const vq_adamw_tensor& t) { return (t.n + kChunk - 1) / kChunk; }

// Half-open address ranges, to find two that meet.
struct Range {
    uintptr_t a, b;
    bool written;
};

// What new gradients are checked against: the tensors' sizes, and what a step writes, in order and apart.
struct Known {
    std::vector<int64_t> n;
    std::vector<Range> written;
    // Whether a step writes between a and b.  `at` is the first range that ends behind a: where the last one
    // asked for lay near, it is still that (searched for each of 1000 gradients, a step's call took 15 us more).
    bool writes(uintptr_t a, uintptr_t b, size_t& at) const
    {
        if ((at > 0 && written[at - 1].b > a) || (at < written.size() && written[at].b <= a))
            at = std::upper_bound(written.begin(), written.end(), a, [](uintptr_t x, const Range& w) { return x < w.b; }) - written.begin();
        return at < written.size() && written[at].a < b;
    }
};

// VQ_CHECK=1: the values of n elements, in rows for the counting kernel.
vq_status check_elements(const void* p, int64_t n, int dtype, const char* what, hipStream_t st)
{
    constexpr int64_t kRow = 4096;
    VQ_TRY(check_matrix(p, n / kRow, kRow, kRow, dtype, "vq_adamw", what, st));
    return check_matrix(static_cast<const char*>(p) + n / kRow * kRow * size_of(dtype), 1, n % kRow, kRow, dtype, "vq_adamw", what, st);
}

vq_status check_inputs(const vq_adamw_plan_t& p, const void* tensors, hipStream_t st)
{
    std::vector<vq_adamw_tensor> t(p.count);
    VQ_HIP(hipMemcpyAsync(t.data(), tensors, t.size() * sizeof(vq_adamw_tensor), hipMemcpyDeviceToHost, st));
    VQ_HIP(hipStreamSynchronize(st));
    for (const vq_adamw_tensor& x : t) {
        VQ_TRY(check_elements(x.grad, x.n, p.grad_dtype, "a gradient", st));
        VQ_TRY(check_elements(p.has_master ? x.master : x.param, x.n, p.has_master ? VQ_F32 : p.param_dtype, "a parameter", st));
        if (p.state_bits == 32) {
            VQ_TRY(check_elements(x.m, x.n, VQ_F32, "m", st));
            VQ_TRY(check_elements(x.v, x.n, VQ_F32, "v", st));
        } else {
            VQ_TRY(check_elements(x.m_scale, (x.n + kBlock - 1) / kBlock, VQ_F32, "m_scale", st));
            VQ_TRY(check_elements(x.v_scale, (x.n + kBlock - 1) / kBlock, VQ_F32, "v_scale", st));
        }
    }
    return VQ_OK;
}

}  // namespace
}  // namespace vq

using namespace vq;

extern "C" {

size_t vq_adamw_plan_bytes(const vq_adamw_tensor* tensors, int64_t count)
{
    if (count < 0 || (count > 0 && !tensors)) return 0;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (tensors[i].n < 0 || tensors[i].n > ((int64_t)1 << 40)) return 0;
        chunks += chunks_of(tensors[i]);
    }
    return align_up(sizeof(Coefficients)) + tensors_bytes(count) + align_up((size_t)chunks * sizeof(Chunk));
}

static vq_status make_plan(const vq_adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype, int has_master,
                           int state_bits, void* table, size_t table_bytes, vq_adamw_plan_t* plan, void* stream)
{
    const std::string call = "vq_adamw_plan";
    VQ_CHECK(plan, call + ": plan is null");
    VQ_CHECK(count >= 0 && count <= (1 << 24), call + ": count must be in [0, 2^24]");
    VQ_CHECK(count == 0 || tensors, call + ": tensors is null");
    VQ_CHECK(known(param_dtype) && known(grad_dtype), call + ": unknown dtype");
    VQ_CHECK(state_bits == 32 || state_bits == 8, call + ": state_bits must be 32 or 8");
    VQ_CHECK(!has_master || param_dtype != VQ_F32, call + ": float32 parameters have no master");
    int64_t chunks = 0;
    std::vector<Range> ranges;
    for (int64_t i = 0; i < count; ++i) {
        const vq_adamw_tensor& t = tensors[i];
        const std::string at = call + ": tensor " + std::to_string(i);
        VQ_CHECK(t.n >= 0 && t.n <= ((int64_t)1 << 40), at + ": n must be in [0, 2^40]");
        if (t.n == 0) continue;
        VQ_CHECK(t.param && t.grad && t.m && t.v, at + ": null pointer");
        VQ_CHECK(!has_master || t.master, at + ": master is null");
        VQ_CHECK(state_bits == 32 || (t.m_scale && t.v_scale), at + ": 8-bit states need m_scale and v_scale");
        VQ_CHECK(!off(t.param, size_of(param_dtype)) && !off(t.grad, size_of(grad_dtype)) && (!has_master || !off(t.master, 4)) &&
                     (state_bits == 8 || (!off(t.m, 4) && !off(t.v, 4))) &&
                     (state_bits == 32 || (!off(t.m_scale, 4) && !off(t.v_scale, 4))),
                 at + ": a pointer is not aligned to its elements");
        chunks += chunks_of(t);
        const auto add = [&](const void* p, size_t bytes, bool written) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(p);
            ranges.push_back({a, a + bytes, written});
        };
        const size_t n = (size_t)t.n, blocks = (n + kBlock - 1) / kBlock;
        add(t.param, n * size_of(param_dtype), true);
        add(t.grad, n * size_of(grad_dtype), false);
        if (has_master) add(t.master, n * 4, true);
        add(t.m, n * (state_bits / 8), true);
        add(t.v, n * (state_bits / 8), true);
        if (state_bits == 8) {
            add(t.m_scale, blocks * 4, true);
            add(t.v_scale, blocks * 4, true);
        }
    }
    VQ_CHECK(chunks < ((int64_t)1 << 24), call + ": more than 2^24 chunks of 4096 elements");      // 2^32 threads
    // a tensor given twice, or two that overlap, would be stepped twice at once
    std::sort(ranges.begin(), ranges.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
    uintptr_t any = 0, written = 0;                           // ends of the ranges so far
    for (const Range& r : ranges) {
        VQ_CHECK(r.a >= (r.written ? any : written), call + ": tensors overlap");
        any = std::max(any, r.b);
        if (r.written) written = std::max(written, r.b);
    }
    *plan = vq_adamw_plan_t{nullptr, count, 0, param_dtype, grad_dtype, has_master ? 1 : 0, state_bits, nullptr};
    if (chunks == 0) return VQ_OK;
    const size_t need = vq_adamw_plan_bytes(tensors, count);
    VQ_WS(table && table_bytes >= need, call + ": table too small");
    VQ_CHECK(aligned16(table), call + ": table is not 16-byte aligned");
    VQ_TRY(check_device());
    const size_t at_tensors = align_up(sizeof(Coefficients)), at_chunks = at_tensors + tensors_bytes(count);
    std::unique_ptr<Known> known(new Known);
    for (int64_t i = 0; i < count; ++i) known->n.push_back(tensors[i].n);
    for (const Range& r : ranges)
        if (r.written) known->written.push_back(r);
    std::vector<char> host(need);
    std::copy(tensors, tensors + count, reinterpret_cast<vq_adamw_tensor*>(host.data() + at_tensors));
    Chunk* c = reinterpret_cast<Chunk*>(host.data() + at_chunks);
    for (int64_t i = 0; i < count; ++i)
        for (int64_t k = 0; k < chunks_of(tensors[i]); ++k) *c++ = {(uint32_t)i, (uint32_t)k};
    VQ_HIP(hipMemcpyAsync(table, host.data(), need, hipMemcpyHostToDevice, as_stream(stream)));
    VQ_HIP(hipStreamSynchronize(as_stream(stream)));
    plan->table = table;
    plan->chunks = chunks;
    plan->known = known.release();
    return VQ_OK;
}

vq_status vq_adamw_plan(const vq_adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype, int has_master,
                        int state_bits, void* table, size_t table_bytes, vq_adamw_plan_t* plan, void* stream)
{
    try {
        return make_plan(tensors, count, param_dtype, grad_dtype, has_master, state_bits, table, table_bytes, plan, stream);
    } catch (const std::bad_alloc&) {
        return fail(VQ_ERR_INVALID, "vq_adamw_plan: out of host memory");
    }
}

void vq_adamw_plan_free(vq_adamw_plan_t* plan)
{
    if (!plan) return;
    delete static_cast<Known*>(plan->known);
    plan->known = nullptr;
}

vq_status vq_adamw_grads(const vq_adamw_plan_t* plan, const void* const* grads, int64_t count, void* stream)
{
    const std::string call = "vq_adamw_grads";
    VQ_CHECK(plan, call + ": plan is null");
    VQ_CHECK(count == plan->count, call + ": count must be the plan's");
    VQ_CHECK(known(plan->grad_dtype) && plan->chunks >= 0 && (plan->chunks == 0 || plan->table), call + ": the plan is not made");
    if (plan->chunks == 0) return VQ_OK;
    VQ_CHECK(grads, call + ": grads is null");
    const size_t size = size_of(plan->grad_dtype);
    for (int64_t i = 0; i < count; ++i)
        VQ_CHECK(!off(grads[i], size), call + ": gradient " + std::to_string(i) + " is not aligned to its elements");
    const Known* const known = static_cast<const Known*>(plan->known);
    VQ_CHECK(known, call + ": the plan is not made, or was freed");
    size_t at = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (known->n[i] == 0) continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
        VQ_CHECK(g, call + ": gradient " + std::to_string(i) + " is null");
        VQ_CHECK(!known->writes(g, g + known->n[i] * size, at), call + ": gradient " + std::to_string(i) + " overlaps what a step writes");
    }
    VQ_TRY(check_device());
    vq_adamw_tensor* const tensors =
        reinterpret_cast<vq_adamw_tensor*>(static_cast<char*>(plan->table) + align_up(sizeof(Coefficients)));
    for (int64_t first = 0; first < count; first += kPointers) {
        GradPointers a{};
        a.first = first;
        a.count = (int)std::min<int64_t>(count - first, kPointers);
        std::copy(grads + first, grads + first + a.count, a.grad);
        hipLaunchKernelGGL(k_adamw_grads, dim3(1), dim3(512), 0, as_stream(stream), a, tensors);
        VQ_LAUNCHED("k_adamw_grads");
    }
    return VQ_OK;
}

vq_status vq_adamw(const vq_adamw_plan_t* plan, double lr, double beta1, double beta2, double eps, double weight_decay,
                   int64_t step, int64_t* step_from, const float* lr_from, const float* grad_scale, void* stream)
{
    const std::string call = "vq_adamw";
    VQ_CHECK(plan, call + ": plan is null");
    VQ_CHECK(lr_from || std::isfinite(lr), call + ": lr must be finite");
    VQ_CHECK(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1, call + ": betas must be in [0, 1)");
    VQ_CHECK(eps >= 0 && std::isfinite(eps) && std::isfinite(weight_decay), call + ": eps must be finite and not negative, weight_decay finite");
    VQ_CHECK(step_from || step >= 1, call + ": step counts from 1");
    VQ_CHECK(!lr_from || step_from, call + ": lr_from needs step_from");
    if (plan->chunks == 0 && !step_from) return VQ_OK;
    VQ_CHECK(plan->chunks >= 0 && plan->count >= 0 && (plan->chunks == 0 || plan->table), call + ": the plan is not made");
    VQ_CHECK(known(plan->param_dtype) && known(plan->grad_dtype) && (plan->state_bits == 32 || plan->state_bits == 8),
             call + ": the plan is not made");
    VQ_CHECK(!off(step_from, 8) && !off(lr_from, 4) && !off(grad_scale, 4), call + ": a pointer is not aligned to its elements");
    VQ_CHECK(!step_from || plan->table, call + ": a step count on the GPU needs a plan with elements");
    VQ_TRY(check_device());
    TimedRegion tr("adamw", 0, as_stream(stream));
    char* const base = static_cast<char*>(plan->table);
    Args a{};
    a.tensors = reinterpret_cast<const vq_adamw_tensor*>(base + align_up(sizeof(Coefficients)));
    a.chunks = reinterpret_cast<const Chunk*>(base + align_up(sizeof(Coefficients)) + tensors_bytes(plan->count));
    a.grad_scale = grad_scale;
    if (values_check_on() && plan->chunks > 0) {
        try {
            VQ_TRY(check_inputs(*plan, a.tensors, as_stream(stream)));
        } catch (const std::bad_alloc&) {
            return fail(VQ_ERR_INVALID, call + ": out of host memory");
        }
    }
    if (step_from) {
        a.from_device = reinterpret_cast<const Coefficients*>(base);
        hipLaunchKernelGGL(k_adamw_tick, dim3(1), dim3(64), 0, as_stream(stream), step_from, lr_from, lr, beta1, beta2, eps,
                           weight_decay, reinterpret_cast<Coefficients*>(base));
        VQ_LAUNCHED("k_adamw_tick");
    } else {
        a.c = coefficients(lr, beta1, beta2, eps, weight_decay, std::pow(beta1, (double)step), std::pow(beta2, (double)step));
    }
    if (plan->param_dtype == VQ_BF16) launch_grad<__bf16>(a, *plan, as_stream(stream));
    else if (plan->param_dtype == VQ_F16) launch_grad<_Float16>(a, *plan, as_stream(stream));
    else launch_grad<float>(a, *plan, as_stream(stream));
    VQ_LAUNCHED("k_adamw");
    return VQ_OK;
}

}  // extern "C"
