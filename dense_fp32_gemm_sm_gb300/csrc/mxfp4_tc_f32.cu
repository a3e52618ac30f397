// mxfp4_tc_f32.cu -- the MXFP4 product's instances with C (and unquantised A) of type f32.
#include "mxfp4_tc_launch.cuh"

namespace fgemm {
namespace mx {

template fgemm_status launch_tc_type<float>(const GemmArgs &g, GemmPlan plan, cudaStream_t stream);
template fgemm_status launch_fused_type<float>(const GemmArgs &g, const void *x, long long ldx, int ranks, cudaStream_t stream);

}  // namespace mx
}  // namespace fgemm
