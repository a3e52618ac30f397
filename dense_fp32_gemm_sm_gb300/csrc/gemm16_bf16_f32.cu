// gemm16_bf16_f32.cu -- kernel instances of the products of BF16 matrices into FP32.
#include "gemm16_launch.cuh"

namespace fgemm {
namespace h16 {

template fgemm_status launch_product_type<__nv_bfloat16, float>(const Product &q, const Plan &plan, cudaStream_t stream);

}  // namespace h16
}  // namespace fgemm
