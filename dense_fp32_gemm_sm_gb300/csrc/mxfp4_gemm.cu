// mxfp4_gemm.cu -- the product of two quantised matrices: which kernel runs it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fgemm_internal.h"
#include "mxfp4_device.cuh"
#include "mxfp4_launch.h"

namespace fgemm {
namespace mx {

template <class T>
fgemm_status launch_tc_type(const GemmArgs &g, GemmPlan plan, cudaStream_t stream);
extern template fgemm_status launch_tc_type<float>(const GemmArgs &, GemmPlan, cudaStream_t);
extern template fgemm_status launch_tc_type<__nv_bfloat16>(const GemmArgs &, GemmPlan, cudaStream_t);
extern template fgemm_status launch_tc_type<__half>(const GemmArgs &, GemmPlan, cudaStream_t);

template <class T>
fgemm_status launch_fused_type(const GemmArgs &g, const void *x, long long ldx, int ranks, cudaStream_t stream);
extern template fgemm_status launch_fused_type<float>(const GemmArgs &, const void *, long long, int, cudaStream_t);
extern template fgemm_status launch_fused_type<__nv_bfloat16>(const GemmArgs &, const void *, long long, int, cudaStream_t);
extern template fgemm_status launch_fused_type<__half>(const GemmArgs &, const void *, long long, int, cudaStream_t);

namespace {

// Stages of a CTA whose quantised tokens (16 rows of codes, two atoms) fit in FUSED_SMEM.
constexpr long long FUSED_STAGES = FUSED_SMEM / (16 * 128 + 2 * ATOM_BYTES);

// C = act(beta * C + bias): alpha or K is 0.
template <class T>
__global__ void __launch_bounds__(256) no_products_kernel(const GemmArgs g)
{
    after_previous_kernel();
    const long long total = (long long)g.M * g.N;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long r = i / g.N, c = i - r * g.N;
        T *const out = static_cast<T *>(g.c) + r * g.ldc + c;
        float o = 0.0f;
        if (g.beta != 0.0f) o = g.beta * to_float(*out);
        if (g.bias) o += g.bias[c];
        if (g.relu) o = relu(o);
        *out = from_float<T>(o);
    }
}

template <class T>
fgemm_status run_gemm(const GemmArgs &g, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    if (g.K == 0) {
        const long long total = (long long)g.M * g.N;
        const dim3 grid((unsigned)std::min<long long>((total + 255) / 256, 8ll * sms));
        return launch(no_products_kernel<T>, grid, 256, 0, stream, 1, g) == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
    }
    return launch_tc_type<T>(g, plan_gemm(g.M, g.N, g.K, (int)sizeof(T), sms), stream);
}

}  // namespace

// Estimated microseconds of the ways a product can run, fitted to measurements on one GB300 (30
// shapes from 96 x 300 x 2000 to 8192 x 11008 x 4096, FP32 and BF16: the way with the least
// estimate took 0.3 % longer than the fastest on average, 10 % at most).  Tiles over CTAs (or
// pairs) come in rounds, each of so many stages and a boundary; C is written beside them.
// For fewer rows than 96, where only the number of ranks is chosen, the same estimate serves
// unfitted, and it weighs 2, 4 and 8 ranks with one CTA an SM although the kernel takes any
// number to 8 and two CTAs an SM.
static double rounds(long long M, long long tile_m, long long N, long long tile_n, long long units)
{
    const long long tiles = ((M + tile_m - 1) / tile_m) * ((N + tile_n - 1) / tile_n);
    return (double)((tiles + units - 1) / units);
}

// Of a split over `ranks` CTAs: the stages of a CTA one after the other, or B at the memory's
// rate, then the joining of the sums.
static double split_time(long long tiles, double stages, double b_time, int ranks, int sms)
{
    const double join = ranks == 1 ? 0.0 : ranks == 2 ? 1.6 : ranks == 4 ? 1.7 : 3.3;
    const double waves = (double)((tiles * ranks + sms - 1) / sms), steps = (double)(((long long)stages + ranks - 1) / ranks);
    return 4.0 + std::max(0.25 * steps * waves + 0.9 * (waves - 1.0), b_time) + join;
}

GemmPlan plan_gemm(long long M, long long N, long long K, int element_size, int sms)
{
    const double stages = (double)((blocks_of(K) + 7) / 8);
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    const long long tiles = ((M + nt - 1) / nt) * ((N + 127) / 128);
    const double b_time = (double)N * (double)blocks_of(K) * 17.0 / 6.5e6, c_time = (double)M * (double)N * element_size / 6.5e6;
    GemmPlan best{nt, 1};
    double least = split_time(tiles, stages, b_time, 1, sms);
    auto consider = [&](GemmPlan plan, double time) {
        if (time < least) {
            best = plan;
            least = time;
        }
    };
    for (int r = 2; r <= 8 && r <= stages && tiles * r <= sms; r *= 2)
        consider(GemmPlan{nt, r}, split_time(tiles, stages, b_time, r, sms));
    if (nt < 64) return best;
    consider(GemmPlan{128, 0}, 3.5 + rounds(M, 128, N, 128, sms) * (0.7 + 0.26 * stages) + 0.25 * c_time);
    consider(GemmPlan{PAIRS_192, 0}, 4.8 + rounds(M, 192, N, 256, sms / 2) * (1.6 + 0.215 * stages) + 0.30 * c_time);
    consider(GemmPlan{PAIRS_256, 0}, 4.6 + rounds(M, 256, N, 256, sms / 2) * (1.8 + 0.295 * stages) + 0.40 * c_time);
    return best;
}

fgemm_status launch_gemm(fgemm_dtype type, const GemmArgs &g, cudaStream_t stream)
{
    switch (type) {
    case FGEMM_F32: return run_gemm<float>(g, stream);
    case FGEMM_BF16: return run_gemm<__nv_bfloat16>(g, stream);
    default: return run_gemm<__half>(g, stream);
    }
}

bool linear_fused(long long M, long long K)
{
    return M <= LINEAR_ROWS && (blocks_of(K) + 7) / 8 <= 8 * FUSED_STAGES;
}

int linear_ranks(long long N, long long K, int sms)
{
    // Up to four ranks as two CTAs an SM allow: they divide the quantising too (one token through
    // 4096 x 11008 took 8.5, 7.8, 7.5 and 10.7 us with 1, 2, 3 and 4).  A cluster of eight costs
    // more than it saves, and is for a K whose tokens need its shared memory.
    const long long stages = (blocks_of(K) + 7) / 8, tiles = (N + 127) / 128;
    int ranks = 1;
    while (ranks < 4 && ranks < stages && (ranks + 1) * tiles <= 2 * sms) ++ranks;
    while (ranks < 8 && stages > ranks * FUSED_STAGES) ++ranks;
    return ranks;
}

fgemm_status launch_linear(fgemm_dtype type, const void *x, long long ldx, const GemmArgs &g, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    const int ranks = linear_ranks(g.N, g.K, sms);
    switch (type) {
    case FGEMM_F32: return launch_fused_type<float>(g, x, ldx, ranks, stream);
    case FGEMM_BF16: return launch_fused_type<__nv_bfloat16>(g, x, ldx, ranks, stream);
    default: return launch_fused_type<__half>(g, x, ldx, ranks, stream);
    }
}

}  // namespace mx
}  // namespace fgemm
