// Dense products for few tokens (decoding): the weights are read once, straight
// from memory into matrix-core operands, and nothing else is large.
//
//   out[t, m] = sum_k W[m, k] X[t, k] for t < 16 NT, with the shared epilogue.
//
// A workgroup owns 16 rows of W (of both matrices of a gated pair); its waves
// take blocks of 32 H columns in turn.  A lane's operand of one matrix
// instruction is eight consecutive columns of one row, so 16 bytes a lane load
// it without LDS, and a block's H loads cover 64 H contiguous bytes of a row.
// The next block's weights are requested before the present one is used.  The
// waves' sums are added in wave order through LDS; where the rows give too few
// workgroups to keep the memory busy, the columns are split over workgroups and
// the tiled product's second kernel adds the parts.
//
// Bound by the weights' bytes.  Loads are at any element-aligned address.  One
// token: 4096 x 11008 bf16 in 17.5 us (5.2 TB/s; a large read reaches 6.2), a pair
// of 8192 x 2048 fp16 in 12.8 us (5.2 TB/s).
#include "vq_few.h"

namespace vq {
namespace {

constexpr int kRows = 16;

struct Few {
    const char* W[2];
    const char* X;
    int64_t ldw, ldx, K;
    int M, T;
    int splits, pitch;
    float* part;                 // [splits][matrices][T][pitch], or null
    Epilogue epi;
};

template <class T, int NT, bool PAIR, int H, bool ODD>
__global__ __launch_bounds__(1024) void k_few(const Few a)
{
    typedef typename T::E E;
    typedef typename T::V8 V8;
    constexpr int NM = PAIR ? 2 : 1;
    constexpr int B = 32 * H;
    extern __shared__ __align__(16) float red[];                 // [waves][NM][NT][64] of four features
    const int nwaves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int m0 = blockIdx.x * kRows;
    const int64_t row = m0 + r < a.M ? m0 + r : a.M - 1;         // rows and tokens past the last repeat it;
    const E* w[NM];                                              // their sums are not stored
    const E* x[NT];
#pragma unroll
    for (int m = 0; m < NM; ++m) w[m] = reinterpret_cast<const E*>(a.W[m]) + row * a.ldw;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        x[n] = reinterpret_cast<const E*>(a.X) + (int64_t)(n * 16 + r < a.T ? n * 16 + r : a.T - 1) * a.ldx;

    f32x4 acc[NM][NT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int nfull = (int)(a.K / B);                            // blocks of whole chunks
    const int f0 = (int)((int64_t)nfull * blockIdx.y / a.splits), f1 = (int)((int64_t)nfull * (blockIdx.y + 1) / a.splits);
    Ahead<T, ODD> wv[NM][H], xv[NT][H];
    const auto load = [&](int kb, int j) {
        const int64_t c = (int64_t)kb * B + j * 32 + g * 8;
#pragma unroll
        for (int n = 0; n < NT; ++n) xv[n][j].load(x[n], c);
#pragma unroll
        for (int m = 0; m < NM; ++m) wv[m][j].load(w[m], c);
    };
    const auto multiply = [&](int j) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n] = T::mfma(wv[m][j].get(w[m]), xv[n][j].get(x[n]), acc[m][n]);
    };
    // the loads keep their order, so that a chunk is awaited alone
    int kb = f0 + wave;
    if (kb < f1) {
#pragma unroll
        for (int j = 0; j < H; ++j) {
            load(kb, j);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll 1
        for (; kb + nwaves < f1; kb += nwaves) {
            // a chunk's registers are refilled for the next block as soon as they are used
#pragma unroll
            for (int j = 0; j < H; ++j) {
                multiply(j);
                __builtin_amdgcn_sched_barrier(0);
                load(kb + nwaves, j);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < H; ++j) multiply(j);
    }
    // columns past the last whole block: steps of 32, dealt to the waves of the last split
    if (blockIdx.y == a.splits - 1) {
        const int steps = (int)((a.K - (int64_t)nfull * B + 31) / 32);
        for (int s = wave; s < steps; s += nwaves) {
            const int64_t c = (int64_t)nfull * B + s * 32 + g * 8;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const V8 v = chunk_tail<T>(w[m], c, a.K);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[m][n] = T::mfma(v, chunk_tail<T>(x[n], c, a.K), acc[m][n]);
            }
        }
    }

#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<f32x4*>(red + (((wave * NM + m) * NT + n) * 64 + lane) * 4) = acc[m][n];
    __syncthreads();
    // thread -> token t, features m0 + 8 f .. + 7 (lanes t%16 + 16 (2 f) and the next group)
    const int t = threadIdx.x >> 1, f = threadIdx.x & 1;
    if (t >= a.T || m0 + f * 8 >= a.M) return;
    float z[NM][8];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < nwaves; ++k)
                v += *reinterpret_cast<const f32x4*>(
                    red + (((k * NM + m) * NT + (t >> 4)) * 64 + (f * 2 + h) * 16 + (t & 15)) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][h * 4 + i] = v[i];
        }
    if (a.part) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            float* o = a.part + (((int64_t)blockIdx.y * NM + m) * a.T + t) * a.pitch + m0 + f * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = z[m][i];
        }
    } else if (PAIR) {
        epilogue_pair<T>(a.epi, t, m0 + f * 8, a.M, z[0], z[NM - 1]);
    } else {
        epilogue_one<T>(a.epi, t, m0 + f * 8, a.M, z[0]);
    }
}

// Sixteen waves a workgroup where the rows give less than two workgroups of
// eight a CU: pair of 4096 x 8192, 27 us with sixteen and 33 with eight; 2048 x
// 8192, 16 tokens, 13.5 and 17; the other way round 4096 x 8192, one token, 19 and
// 15.  With more rows eight: 8192 x 8192, 25 and 34 us.  The columns are split
// over workgroups where the rows give less than one of sixteen and every wave of
// every split keeps a block: 1024 x 16384, 13-16 us over four, 20 over one; 1024
// x 4096, one: 8.9 us, and 12.7 over two with their second launch.
struct FewPlan { int waves, splits; };
FewPlan few_plan(int64_t M, int64_t K)
{
    const int64_t groups = (M + kRows - 1) / kRows, blocks = K / 256;
    FewPlan p{groups < 512 && blocks >= 16 ? 16 : 8, 1};
    while (p.splits < 16 && groups * p.splits < 256 && blocks >= (int64_t)p.waves * p.splits * 2) p.splits *= 2;
    return p;
}

template <class T, int NT, bool PAIR, int H>
vq_status few_kernel(const Few& a, int waves, hipStream_t st)
{
    const bool odd = odd_rows(a.W[0], a.ldw) || odd_rows(a.X, a.ldx) || (PAIR && odd_rows(a.W[1], a.ldw));
    const dim3 grid((unsigned)((a.M + kRows - 1) / kRows), (unsigned)a.splits);
    const size_t lds = (size_t)waves * (PAIR ? 2 : 1) * NT * 256 * sizeof(float);
    if (odd) hipLaunchKernelGGL((k_few<T, NT, PAIR, H, true>), grid, dim3(waves * 64), lds, st, a);
    else hipLaunchKernelGGL((k_few<T, NT, PAIR, H, false>), grid, dim3(waves * 64), lds, st, a);
    VQ_LAUNCHED("k_few");
    return VQ_OK;
}

template <class T, int NT>
vq_status few_launch(const Few& a, int waves, bool pair, hipStream_t st)
{
    if (pair) VQ_TRY((few_kernel<T, NT, true, 4>(a, waves, st)));
    else VQ_TRY((few_kernel<T, NT, false, NT == 1 ? 8 : 4>(a, waves, st)));
    if (a.splits > 1) VQ_TRY(finish_parts(T::kDtype, pair, a.part, a.splits, a.M, a.T, a.pitch, a.epi, st));
    return VQ_OK;
}

}  // namespace

// Up to 32 tokens, while the weights' elements times the tokens stay below 6e8: past
// that the tiled product, which reads the tokens once a tile, is mostly faster.  One
// token by 8192 x 8192: 25 us here and 26 us tiled, 32 45 and 28; 4096 x 4096, 32 tokens:
// 14 and 16; pair of 8192 x 8192, one 40 and 43.  The product of sizes does not separate
// the two everywhere; below the threshold this way is the slower for one token by 8192 x
// 28672 (107 us here, 91 tiled), by 16384 x 4096 (27, 25) and by pairs of 28672 x 8192 (168,
// 161) and 16384 x 4096 (48, 43), and for eight by 8192 x 8192 (29, 26) and 11008 x 4096 (22, 21).
bool few_tokens(int64_t T, int64_t M, int64_t K, int nm) { return T <= 32 && (double)T * (double)M * (double)K * nm < 6e8; }

size_t few_workspace(int64_t T, int64_t M, int64_t K, int nm)
{
    const int s = few_plan(M, K).splits;
    return s > 1 ? align_up((size_t)s * nm * T * ((M + 7) / 8 * 8) * sizeof(float)) : 0;
}

vq_status few_product(const FewArgs& f, void* ws, hipStream_t st)
{
    Few a{};
    for (int i = 0; i < f.nm; ++i) a.W[i] = static_cast<const char*>(f.W[i]);
    a.X = static_cast<const char*>(f.X);
    a.ldw = f.ldw; a.ldx = f.ldx; a.K = f.K;
    a.M = (int)f.M; a.T = (int)f.T;
    const FewPlan p = few_plan(f.M, f.K);
    a.splits = p.splits;
    a.pitch = (int)((f.M + 7) / 8 * 8);
    a.part = a.splits > 1 ? static_cast<float*>(ws) : nullptr;
    a.epi = f.epi;
    const bool pair = f.nm > 1;
    if (f.dtype == VQ_BF16) return f.T > 16 ? few_launch<Bf16, 2>(a, p.waves, pair, st) : few_launch<Bf16, 1>(a, p.waves, pair, st);
    return f.T > 16 ? few_launch<F16, 2>(a, p.waves, pair, st) : few_launch<F16, 1>(a, p.waves, pair, st);
}

}  // namespace vq
