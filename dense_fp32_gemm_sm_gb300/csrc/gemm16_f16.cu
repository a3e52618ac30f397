// gemm16_f16.cu -- kernel instances of the products of F16 matrices.
#include "gemm16_launch.cuh"

namespace fgemm {
namespace h16 {

template fgemm_status launch_product_type<__half, __half>(const Product &q, const Plan &plan, cudaStream_t stream);

}  // namespace h16
}  // namespace fgemm
