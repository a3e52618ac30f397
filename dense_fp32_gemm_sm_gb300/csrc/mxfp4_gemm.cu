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

namespace {

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

GemmPlan plan_gemm(long long M, long long N, long long K, int sms)
{
    const long long stages = (blocks_of(K) + 7) / 8, tiles_w = (N + 127) / 128;
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const long long tiles = tiles_w * ((M + nt - 1) / nt);
    if (nt == 128 && tiles_w * ((M + 255) / 256) >= sms) return GemmPlan{256, 0};
    if (nt == 128 && tiles >= sms) return GemmPlan{128, 0};
    int ranks = 1;
    while (ranks < 8 && 2 * ranks * tiles <= 2 * sms && 2 * ranks <= stages) ranks *= 2;
    return GemmPlan{nt, ranks};
}

fgemm_status launch_gemm(fgemm_dtype type, const GemmArgs &g, cudaStream_t stream)
{
    switch (type) {
    case FGEMM_F32: return run_gemm<float>(g, stream);
    case FGEMM_BF16: return run_gemm<__nv_bfloat16>(g, stream);
    default: return run_gemm<__half>(g, stream);
    }
}

}  // namespace mx
}  // namespace fgemm
