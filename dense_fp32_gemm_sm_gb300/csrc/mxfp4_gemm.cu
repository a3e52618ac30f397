// mxfp4_gemm.cu -- the product of two quantised matrices: which kernel runs it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fgemm_internal.h"
#include "mxfp4_device.cuh"

namespace fgemm {
namespace mx {

template <class T>
fgemm_status launch_tc_type(const GemmArgs &g, int nt, int ranks, cudaStream_t stream);
extern template fgemm_status launch_tc_type<float>(const GemmArgs &, int, int, cudaStream_t);
extern template fgemm_status launch_tc_type<__nv_bfloat16>(const GemmArgs &, int, int, cudaStream_t);
extern template fgemm_status launch_tc_type<__half>(const GemmArgs &, int, int, cudaStream_t);

template <class T>
fgemm_status launch_fused_type(const GemmArgs &g, const void *x, long long ldx, int nt, int ranks, cudaStream_t stream);
extern template fgemm_status launch_fused_type<float>(const GemmArgs &, const void *, long long, int, int, cudaStream_t);
extern template fgemm_status launch_fused_type<__nv_bfloat16>(const GemmArgs &, const void *, long long, int, int,
                                                              cudaStream_t);
extern template fgemm_status launch_fused_type<__half>(const GemmArgs &, const void *, long long, int, int, cudaStream_t);

namespace {

// Stages of a CTA whose quantised tokens (16 rows of codes, two atoms) fit in FUSED_SMEM.
constexpr long long FUSED_STAGES = FUSED_SMEM / (16 * 128 + 2 * ATOM_BYTES);

// C = act(beta * C + bias): alpha or K is 0.
template <class T>
__global__ void __launch_bounds__(256) no_products_kernel(const GemmArgs g)
{
    const long long total = (long long)g.M * g.N;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long r = i / g.N, c = i - r * g.N;
        T *const out = static_cast<T *>(g.c) + r * g.ldc + c;
        float o = 0.0f;
        if (g.beta != 0.0f) o = g.beta * to_float(*out);
        if (g.bias) o += g.bias[c];
        if (g.relu) o = fmaxf(o, 0.0f);
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
        no_products_kernel<T><<<(unsigned)std::min<long long>((total + 255) / 256, 8ll * sms), 256, 0, stream>>>(g);
        return cudaGetLastError() == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
    }
    const GemmPlan plan = plan_gemm(g.M, g.N, g.K, sms);
    return launch_tc_type<T>(g, plan.nt, plan.ranks, stream);
}

}  // namespace

// Microseconds of a tile's stages over `ranks` CTAs, up to a constant: the stages of a CTA one
// after the other (two CTAs on an SM share it), or B's bytes at the memory's rate; then what
// joining the ranks' sums takes.
static double split_time(long long N, long long K, long long tiles, long long stages, int ranks, int sms)
{
    const double join[4] = {0.0, 1.0, 1.1, 2.7};
    const long long ctas = tiles * ranks, waves = (ctas + sms - 1) / sms;
    const double steps = 0.21 * (double)((stages + ranks - 1) / ranks) * (double)waves;
    return std::max(steps, (double)N * (double)blocks_of(K) * 17.0 / 6.5e6) +
           join[ranks == 1 ? 0 : ranks == 2 ? 1 : ranks == 4 ? 2 : 3];
}

static int best_ranks(long long N, long long K, long long tiles, long long stages, int sms)
{
    int best = 1;
    for (int r = 2; r <= 8 && r <= stages; r *= 2)
        if (split_time(N, K, tiles, stages, r, sms) < split_time(N, K, tiles, stages, best, sms)) best = r;
    return best;
}

GemmPlan plan_gemm(long long M, long long N, long long K, int sms)
{
    const long long stages = (blocks_of(K) + 7) / 8, tiles_w = (N + 127) / 128;
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    const long long tiles = tiles_w * ((M + nt - 1) / nt);
    if (nt == 64 && tiles_w * ((M + 255) / 256) >= sms) return GemmPlan{512, 0};
    if (nt == 64 && tiles >= 2 * sms) return GemmPlan{128, 0};
    return GemmPlan{nt, best_ranks(N, K, tiles, stages, sms)};
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

GemmPlan plan_linear(long long N, long long K, int sms)
{
    // As many ranks as two CTAs an SM allow: they divide the quantising too.  (A cluster of
    // eight costs more than it saves, and is for a K whose tokens need their shared memory.)
    const long long stages = (blocks_of(K) + 7) / 8, tiles = (N + 127) / 128;
    int ranks = 1;
    while (ranks < 8 && 2 * ranks <= stages && (stages > ranks * FUSED_STAGES || (ranks < 4 && 2 * ranks * tiles <= 2 * sms)))
        ranks *= 2;
    return GemmPlan{16, ranks};
}

fgemm_status launch_linear(fgemm_dtype type, const void *x, long long ldx, const GemmArgs &g, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    const GemmPlan plan = plan_linear(g.N, g.K, sms);
    switch (type) {
    case FGEMM_F32: return launch_fused_type<float>(g, x, ldx, plan.nt, plan.ranks, stream);
    case FGEMM_BF16: return launch_fused_type<__nv_bfloat16>(g, x, ldx, plan.nt, plan.ranks, stream);
    default: return launch_fused_type<__half>(g, x, ldx, plan.nt, plan.ranks, stream);
    }
}

}  // namespace mx
}  // namespace fgemm
