// mxfp4_api.cu -- the C entries of the MXFP4 operators: argument checks (host integer code,
// before any CUDA call) and dispatch.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_internal.h"
#include "mxfp4.h"

namespace fgemm {
namespace mx {
namespace {

bool valid_type(fgemm_dtype t) { return t == FGEMM_F32 || t == FGEMM_BF16 || t == FGEMM_F16; }
size_t type_size(fgemm_dtype t) { return t == FGEMM_F32 ? 4 : 2; }
bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// An unquantised matrix whose rows hold `cols` elements.
bool valid_matrix(const void *p, fgemm_dtype t, long long cols, long long ld)
{
    return p != nullptr && aligned(p, type_size(t)) && ld >= (cols > 1 ? cols : 1);
}

// The leading dimension of the codes of a quantised matrix with `cols` columns.
bool valid_codes_ld(long long cols, long long ld)
{
    const long long need = 16 * blocks_of(cols);
    return ld % 16 == 0 && ld >= (need > 16 ? need : 16);
}

bool valid_quantised(const void *codes, const void *scales, long long cols, long long ld)
{
    return codes != nullptr && scales != nullptr && aligned(codes, 16) && aligned(scales, 16) &&
           valid_codes_ld(cols, ld);
}

size_t codes_bytes(long long rows, long long cols)
{
    return sat_mul((size_t)rows, (size_t)(16 * blocks_of(cols)));
}

size_t scales_bytes(long long rows, long long cols)
{
    return sat_mul((size_t)((rows + ATOM_ROWS - 1) / ATOM_ROWS), (size_t)(atoms_of(blocks_of(cols)) * ATOM_BYTES));
}

size_t round256(size_t n) { return sat_add(n, 255) / 256 * 256; }

// The layer's quantised tokens: rows of whole blocks, and where there are many, rows that start on
// 64 bytes, as the product reads them faster (4096 x 4096 x 4000 with both operands' rows on
// 16: 36 us, on 64: 27; 32 x 4096 x 11000: 7.2 both ways).
long long tokens_ld(long long M, long long K) { return M > 64 ? 64 * ((K + 127) / 128) : 16 * blocks_of(K); }

struct Direction {
    void *codes;
    int ld;
    void *scales;
};

// The checks that both quantising entries share.
bool valid_directions(const Direction &rows, const Direction &cols, long long M, long long N)
{
    const bool r = rows.codes || rows.scales, c = cols.codes || cols.scales;
    if (!r && !c) return false;
    if (r && !valid_quantised(rows.codes, rows.scales, N, rows.ld)) return false;
    return !c || valid_quantised(cols.codes, cols.scales, M, cols.ld);
}

QuantParams quant_params(int M, int N, const void *x, int ldx, const Direction &rows, const Direction &cols)
{
    QuantParams p{};
    p.x = x;
    p.ldx = ldx;
    p.M = M;
    p.N = N;
    p.row_codes = static_cast<uint8_t *>(rows.codes);
    p.row_scales = static_cast<uint8_t *>(rows.scales);
    p.ld_row = rows.ld;
    p.col_codes = static_cast<uint8_t *>(cols.codes);
    p.col_scales = static_cast<uint8_t *>(cols.scales);
    p.ld_col = cols.ld;
    return p;
}

}  // namespace
}  // namespace mx
}  // namespace fgemm

using namespace fgemm;
using namespace fgemm::mx;

extern "C" {

size_t fgemm_mxfp4_codes_size(int rows, int cols)
{
    return rows > 0 && cols > 0 ? codes_bytes(rows, cols) : 0;
}

size_t fgemm_mxfp4_scales_size(int rows, int cols)
{
    return rows > 0 && cols > 0 ? scales_bytes(rows, cols) : 0;
}

fgemm_status fgemm_mxfp4_quantize(fgemm_dtype type, int M, int N, const void *X, int ldx,
                                  void *row_codes, int ld_row_codes, void *row_scales,
                                  void *col_codes, int ld_col_codes, void *col_scales,
                                  cudaStream_t stream)
{
    const Direction rows{row_codes, ld_row_codes, row_scales}, cols{col_codes, ld_col_codes, col_scales};
    if (!valid_type(type) || M < 0 || N < 0) return FGEMM_ERR_INVALID_VALUE;
    if (ldx < (N > 1 ? N : 1)) return FGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return FGEMM_OK;
    if (!valid_matrix(X, type, N, ldx) || !valid_directions(rows, cols, M, N)) return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(M, N, 0)) return FGEMM_ERR_NOT_SUPPORTED;
    return launch_quantize(type, quant_params(M, N, X, ldx, rows, cols), stream);
}

size_t fgemm_mxfp4_quantize_grad_workspace_size(int M, int N)
{
    if (M < 1 || N < 1) return 0;
    return sat_mul((size_t)((M + (long long)ATOM_ROWS - 1) / ATOM_ROWS), (size_t)N * sizeof(float));
}

fgemm_status fgemm_mxfp4_quantize_grad(fgemm_dtype type, int M, int N, const void *G, int ldg,
                                       const void *Y, int ldy, void *row_codes, int ld_row_codes,
                                       void *row_scales, void *col_codes, int ld_col_codes,
                                       void *col_scales, float *bias_grad, void *workspace,
                                       size_t workspace_bytes, cudaStream_t stream)
{
    const Direction rows{row_codes, ld_row_codes, row_scales}, cols{col_codes, ld_col_codes, col_scales};
    if (!valid_type(type) || M < 0 || N < 0) return FGEMM_ERR_INVALID_VALUE;
    if (ldg < (N > 1 ? N : 1) || (Y && ldy < (N > 1 ? N : 1))) return FGEMM_ERR_INVALID_VALUE;
    if (bias_grad && !aligned(bias_grad, 4)) return FGEMM_ERR_INVALID_VALUE;
    if (N == 0) return FGEMM_OK;
    if (M == 0) {  // a sum of no rows
        if (!bias_grad) return FGEMM_OK;
        return cudaMemsetAsync(bias_grad, 0, (size_t)N * sizeof(float), stream) == cudaSuccess ? FGEMM_OK
                                                                                                : FGEMM_ERR_LAUNCH;
    }
    if (!valid_matrix(G, type, N, ldg) || (Y && !aligned(Y, type_size(type))) || !valid_directions(rows, cols, M, N))
        return FGEMM_ERR_INVALID_VALUE;
    if (bias_grad && (!workspace || !aligned(workspace, 16) ||
                      workspace_bytes < fgemm_mxfp4_quantize_grad_workspace_size(M, N)))
        return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(M, N, 0)) return FGEMM_ERR_NOT_SUPPORTED;
    QuantParams p = quant_params(M, N, G, ldg, rows, cols);
    p.gate = Y;
    p.ldgate = ldy;
    p.bias_grad = bias_grad;
    p.partial = static_cast<float *>(workspace);
    return launch_quantize(type, p, stream);
}

fgemm_status fgemm_mxfp4_dequantize(fgemm_dtype type, int M, int N, const void *codes, int ld_codes,
                                    const void *scales, void *X, int ldx, cudaStream_t stream)
{
    if (!valid_type(type) || M < 0 || N < 0) return FGEMM_ERR_INVALID_VALUE;
    if (ldx < (N > 1 ? N : 1) || !valid_codes_ld(N, ld_codes)) return FGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return FGEMM_OK;
    if (!valid_matrix(X, type, N, ldx) || !valid_quantised(codes, scales, N, ld_codes)) return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(M, N, 0)) return FGEMM_ERR_NOT_SUPPORTED;
    DequantParams p{};
    p.codes = static_cast<const uint8_t *>(codes);
    p.scales = static_cast<const uint8_t *>(scales);
    p.ld = ld_codes;
    p.x = X;
    p.ldx = ldx;
    p.M = M;
    p.N = N;
    return launch_dequantize(type, p, stream);
}

fgemm_status fgemm_mxfp4_gemm(fgemm_dtype type, int M, int N, int K, float alpha,
                              const void *A_codes, int ld_A_codes, const void *A_scales,
                              const void *B_codes, int ld_B_codes, const void *B_scales,
                              float beta, void *C, int ldc, const float *bias, int apply_relu,
                              cudaStream_t stream)
{
    if (!valid_type(type) || M < 0 || N < 0 || K < 0) return FGEMM_ERR_INVALID_VALUE;
    if (!valid_codes_ld(K, ld_A_codes) || !valid_codes_ld(K, ld_B_codes)) return FGEMM_ERR_INVALID_VALUE;
    if (ldc < (N > 1 ? N : 1) || (bias && !aligned(bias, 4))) return FGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return FGEMM_OK;
    if (!valid_matrix(C, type, N, ldc)) return FGEMM_ERR_INVALID_VALUE;
    const bool products = K > 0 && alpha != 0.0f;
    if (products && (!valid_quantised(A_codes, A_scales, K, ld_A_codes) ||
                     !valid_quantised(B_codes, B_scales, K, ld_B_codes)))
        return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(M, N, K)) return FGEMM_ERR_NOT_SUPPORTED;
    GemmArgs g{};
    g.M = M;
    g.N = N;
    g.K = products ? K : 0;
    g.alpha = products ? alpha : 0.0f;
    g.beta = beta;
    g.a = static_cast<const uint8_t *>(A_codes);
    g.a_scales = static_cast<const uint8_t *>(A_scales);
    g.lda = ld_A_codes;
    g.b = static_cast<const uint8_t *>(B_codes);
    g.b_scales = static_cast<const uint8_t *>(B_scales);
    g.ldb = ld_B_codes;
    g.c = C;
    g.ldc = ldc;
    g.bias = bias;
    g.relu = apply_relu ? 1 : 0;
    return launch_gemm(type, g, stream);
}

int fgemm_mxfp4_plan(fgemm_dtype type, int M, int N, int K, int num_sms)
{
    if (!valid_type(type) || M < 1 || N < 1 || K < 1 || num_sms < 2 || !dims_supported(M, N, K)) return -1;
    const GemmPlan plan = plan_gemm(M, N, K, (int)type_size(type), num_sms);
    return 16 * plan.nt + plan.ranks;
}

size_t fgemm_mxfp4_linear_workspace_size(int M, int N, int K)
{
    if (M < 1 || N < 1 || K < 1 || linear_fused(M, K)) return 0;
    return sat_add(round256(sat_mul((size_t)M, (size_t)tokens_ld(M, K))), scales_bytes(M, K));
}

fgemm_status fgemm_mxfp4_linear(fgemm_dtype type, int M, int N, int K, const void *X, int ldx,
                                const void *W_codes, int ld_W_codes, const void *W_scales,
                                const float *bias, int apply_relu, void *Y, int ldy,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (!valid_type(type) || M < 0 || N < 0 || K < 0) return FGEMM_ERR_INVALID_VALUE;
    if (ldx < (K > 1 ? K : 1) || !valid_codes_ld(K, ld_W_codes)) return FGEMM_ERR_INVALID_VALUE;
    if (ldy < (N > 1 ? N : 1) || (bias && !aligned(bias, 4))) return FGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return FGEMM_OK;
    if (!valid_matrix(Y, type, N, ldy)) return FGEMM_ERR_INVALID_VALUE;
    if (K > 0 && (!valid_matrix(X, type, K, ldx) || !valid_quantised(W_codes, W_scales, K, ld_W_codes)))
        return FGEMM_ERR_INVALID_VALUE;
    const size_t need = fgemm_mxfp4_linear_workspace_size(M, N, K);
    if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(M, N, K)) return FGEMM_ERR_NOT_SUPPORTED;
    GemmArgs g{};
    g.M = M;
    g.N = N;
    g.K = K;
    g.alpha = 1.0f;
    g.b = static_cast<const uint8_t *>(W_codes);
    g.b_scales = static_cast<const uint8_t *>(W_scales);
    g.ldb = ld_W_codes;
    g.c = Y;
    g.ldc = ldy;
    g.bias = bias;
    g.relu = apply_relu ? 1 : 0;
    if (K == 0) return launch_gemm(type, g, stream);
    if (linear_fused(M, K)) return launch_linear(type, X, ldx, g, stream);
    uint8_t *const codes = static_cast<uint8_t *>(workspace);
    const int ld = (int)tokens_ld(M, K);
    uint8_t *const scales = codes + round256((size_t)M * (size_t)ld);
    const fgemm_status st = launch_quantize(
        type, quant_params(M, K, X, ldx, Direction{codes, ld, scales}, Direction{nullptr, 0, nullptr}), stream);
    if (st != FGEMM_OK) return st;
    g.a = codes;
    g.a_scales = scales;
    g.lda = ld;
    g.dependent = 1;
    return launch_gemm(type, g, stream);
}

}  // extern "C"
