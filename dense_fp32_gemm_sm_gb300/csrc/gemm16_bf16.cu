// gemm16_bf16.cu -- kernel instances of the products of BF16 matrices.
#include "gemm16_launch.cuh"

namespace fgemm {
namespace h16 {

template fgemm_status launch_product_type<__nv_bfloat16, __nv_bfloat16>(const Product &q, const Plan &plan, cudaStream_t stream);

}  // namespace h16
}  // namespace fgemm
