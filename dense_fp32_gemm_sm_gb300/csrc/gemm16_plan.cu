// gemm16_plan.cu -- how a 16-bit product runs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fgemm_internal.h"
#include "gemm16.h"

namespace fgemm {
namespace h16 {

Plan plan_product(long long M, long long N, long long K, int ragged, long long groups, bool sums, bool fine, int sms)
{
    Plan plan{1, 256, 1, 1, 0};
    plan.in_turns = fine && K > 512;
    return plan;
}

fgemm_status launch_product(const Product &q, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) return FGEMM_ERR_LAUNCH;
    const Plan plan = plan_product(q.M, q.N, q.K, q.ragged, q.groups, q.partial != nullptr,
                                   q.partial != nullptr || q.out_type == FGEMM_F32, sms);
    return q.type == FGEMM_BF16 ? launch_product_type<__nv_bfloat16>(q, plan, stream)
                                : launch_product_type<__half>(q, plan, stream);
}

}  // namespace h16
}  // namespace fgemm
