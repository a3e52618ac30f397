// gemm16_api.cu -- the C entries of the 16-bit layers: argument checks (host integer code, before
// any CUDA call), copies of operands that the products cannot read as they are, and dispatch.
#include <cuda_runtime.h>

#include <cstdint>

#include "fgemm_internal.h"
#include "gemm16.h"

namespace fgemm {
namespace h16 {
namespace {

bool valid_type(fgemm_dtype t) { return t == FGEMM_BF16 || t == FGEMM_F16; }
bool valid_types(fgemm_dtype t, fgemm_dtype out) { return valid_type(t) && (out == t || out == FGEMM_F32); }
bool valid_act(fgemm_activation a) { return a >= FGEMM_ACT_NONE && a <= FGEMM_ACT_SILU; }
bool valid_op(fgemm_op op) { return op == FGEMM_OP_N || op == FGEMM_OP_T; }
size_t type_size(fgemm_dtype t) { return t == FGEMM_F32 ? 4 : 2; }
bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool valid_ld(long long cols, long long ld) { return ld >= (cols > 1 ? cols : 1); }
bool valid_matrix(const void *p, fgemm_dtype t) { return p != nullptr && aligned(p, type_size(t)); }

size_t round256(size_t n) { return sat_add(n, 255) / 256 * 256; }
long long even_ld(long long cols) { return (cols + 7) / 8 * 8; }

// Bytes of a copy with rows on 16 bytes.
size_t copy_bytes(long long rows, long long cols, long long batch)
{
    return sat_mul(sat_mul((size_t)rows, (size_t)batch), (size_t)even_ld(cols) * 2);
}

// Whether TMA reads a matrix as it is.
bool readable(const void *p, long long rows, long long ld, long long batch, long long stride)
{
    return aligned(p, 16) && (rows <= 1 || ld % 8 == 0) && (batch <= 1 || stride % 8 == 0) && ld < (1ll << 38) &&
           stride < (1ll << 38);
}

// Pieces of a caller's workspace, one after the other, each from a multiple of 256 bytes.
struct Space {
    uint8_t *at;
    size_t left;
    bool ok;
    void *take(size_t bytes)
    {
        void *const p = at;
        if (!at || bytes > left) {
            ok = false;
            return nullptr;
        }
        const size_t step = round256(bytes) < left ? round256(bytes) : left;
        at += step;
        left -= step;
        return p;
    }
};

size_t partial_bytes(long long groups, long long M, long long N)
{
    return sat_mul((size_t)partial_rows(groups, M), sat_mul((size_t)N, sizeof(float)));
}

size_t sums_bytes(long long groups, long long M, long long N)
{
    return sat_add(round256(partial_bytes(groups, M, N)), sizeof(int) * (size_t)(groups + 1));
}

// What the product entries share once their arguments are checked: room for partial sums, copies of operands
// that are not on 16 bytes, the product, the sums.
fgemm_status run(Product &q, float *col_sums, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const bool products = q.K > 0 && q.alpha != 0.0f;
    const long long batch = q.ragged == RAGGED_ROWS ? q.groups : 1;
    const long long a_rows = q.ta ? q.K : q.M, a_cols = q.ta ? q.M : q.K, b_rows = q.tb ? q.N : q.K, b_cols = q.tb ? q.K : q.N;
    Space space{static_cast<uint8_t *>(workspace), workspace_bytes, true};
    if (col_sums) {
        q.partials = partial_rows(q.groups, q.M);
        q.partial = static_cast<float *>(space.take(partial_bytes(q.groups, q.M, q.N)));
        q.partial_start = static_cast<int *>(space.take(sizeof(int) * (size_t)(q.groups + 1)));
    }
    const bool copy_a = products && !readable(q.a, a_rows, q.lda, 1, 0);
    const bool copy_b = products && !readable(q.b, b_rows, q.ldb, batch, q.stride_b);
    void *const a = copy_a ? space.take(copy_bytes(a_rows, a_cols, 1)) : nullptr;
    void *const b = copy_b ? space.take(copy_bytes(b_rows, b_cols, batch)) : nullptr;
    if (!space.ok || ((col_sums || copy_a || copy_b) && !aligned(workspace, 16))) return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(q.M, q.N, q.K)) return FGEMM_ERR_NOT_SUPPORTED;
    if (copy_a || copy_b) {
        const Realign none{}, ca = copy_a ? realign(q.a, q.lda, 0, a_rows, (int)a_cols, 1, a) : none;
        const Realign cb = copy_b ? realign(q.b, q.ldb, q.stride_b, b_rows, (int)b_cols, batch, b) : none;
        const fgemm_status st = launch_realign(ca, cb, stream);
        if (st != FGEMM_OK) return st;
    }
    if (copy_a) {
        q.a = a;
        q.lda = even_ld(a_cols);
    }
    if (copy_b) {
        q.b = b;
        q.ldb = even_ld(b_cols);
        q.stride_b = b_rows * q.ldb;
    }
    const fgemm_status st = launch_product(q, stream);
    if (st != FGEMM_OK || !col_sums) return st;
    return launch_sums(q.partial, q.partials, q.partial_start, nullptr, q.groups, q.N, col_sums, stream);
}

fgemm_status zero(float *x, size_t n, cudaStream_t stream)
{
    if (!x || n == 0) return FGEMM_OK;
    return cudaMemsetAsync(x, 0, n * sizeof(float), stream) == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
}

// Operands of one product, or of products by groups of rows (groups < 1: refused; offsets null: one product).
fgemm_status product(fgemm_dtype type, fgemm_dtype out_type, fgemm_op transa, fgemm_op transb, int groups, int M, int N, int K,
                     const int *offsets, bool grouped, float alpha, const void *A, int lda, const void *B, int ldb,
                     long long strideB, Product &q, bool &empty)
{
    empty = false;
    if (!valid_types(type, out_type) || !valid_op(transa) || !valid_op(transb) || M < 0 || N < 0 || K < 0)
        return FGEMM_ERR_INVALID_VALUE;
    if (!valid_ld(transa == FGEMM_OP_T ? M : K, lda) || !valid_ld(transb == FGEMM_OP_T ? K : N, ldb))
        return FGEMM_ERR_INVALID_VALUE;
    if (groups < 1 || strideB < 0) return FGEMM_ERR_INVALID_VALUE;
    q = Product{};
    q.type = type;
    q.out_type = out_type;
    q.M = M;
    q.N = N;
    q.K = K;
    q.ta = transa == FGEMM_OP_T;
    q.tb = transb == FGEMM_OP_T;
    q.alpha = alpha;
    q.a = A;
    q.b = B;
    q.lda = lda;
    q.ldb = ldb;
    q.stride_b = strideB;
    q.ragged = grouped ? RAGGED_ROWS : RAGGED_NONE;
    q.groups = groups;
    q.offsets = offsets;
    empty = M == 0 || N == 0;
    if (empty) return FGEMM_OK;
    if (K > 0 && alpha != 0.0f && (!valid_matrix(A, type) || !valid_matrix(B, type))) return FGEMM_ERR_INVALID_VALUE;
    if (grouped && (!offsets || !aligned(offsets, 4))) return FGEMM_ERR_INVALID_VALUE;
    return groups > FGEMM_MAX_GROUPS ? FGEMM_ERR_NOT_SUPPORTED : FGEMM_OK;
}

// The forward epilogue.
bool forward(Product &q, const float *bias, fgemm_activation act, void *Z, int ldz, float beta, const void *R, int ldr, void *Y,
             int ldy)
{
    if (!valid_act(act) || (bias && !aligned(bias, 4)) || !valid_ld(q.N, ldy)) return false;
    if (Z && (!valid_ld(q.N, ldz) || !aligned(Z, 2))) return false;
    if (beta != 0.0f && !valid_ld(q.N, ldr)) return false;
    if (q.M > 0 && q.N > 0 && (!valid_matrix(Y, q.out_type) || (beta != 0.0f && !valid_matrix(R, q.out_type)))) return false;
    q.bias = bias;
    q.act = act;
    q.z = Z;
    q.ldz = ldz;
    q.beta = beta;
    q.r = R;
    q.ldr = ldr;
    q.y = Y;
    q.ldy = ldy;
    return true;
}

// The epilogue of the gradient.
bool backward(Product &q, fgemm_activation act, const void *Z, int ldz, void *Y, int ldy, const float *col_sums)
{
    if (!valid_act(act) || !valid_ld(q.N, ldy) || (col_sums && !aligned(col_sums, 4))) return false;
    if (act != FGEMM_ACT_NONE && !valid_ld(q.N, ldz)) return false;
    if (q.M > 0 && q.N > 0 && (!valid_matrix(Y, q.out_type) || (act != FGEMM_ACT_NONE && !valid_matrix(Z, q.type)))) return false;
    q.slope = 1;
    q.act = act;
    q.z = const_cast<void *>(Z);
    q.ldz = ldz;
    q.y = Y;
    q.ldy = ldy;
    return true;
}

}  // namespace
}  // namespace h16
}  // namespace fgemm

using namespace fgemm;
using namespace fgemm::h16;

extern "C" {

size_t fgemm_gemm16_copy_workspace_size(fgemm_op transa, fgemm_op transb, int groups, int M, int N, int K)
{
    if (!valid_op(transa) || !valid_op(transb) || groups < 1 || M < 1 || N < 1 || K < 1) return 0;
    const bool ta = transa == FGEMM_OP_T, tb = transb == FGEMM_OP_T;
    return sat_add(round256(copy_bytes(ta ? K : M, ta ? M : K, 1)), copy_bytes(tb ? N : K, tb ? K : N, groups));
}

size_t fgemm_gemm16_sums_workspace_size(int groups, int M, int N)
{
    return groups < 1 || M < 1 || N < 1 ? 0 : round256(sums_bytes(groups, M, N));
}

fgemm_status fgemm_gemm16(fgemm_dtype type, fgemm_dtype out_type, fgemm_op transa, fgemm_op transb, int M, int N, int K,
                          float alpha, const void *A, int lda, const void *B, int ldb, const float *bias,
                          fgemm_activation act, void *Z, int ldz, float beta, const void *R, int ldr, void *Y, int ldy,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    Product q;
    bool empty;
    const fgemm_status st = product(type, out_type, transa, transb, 1, M, N, K, nullptr, false, alpha, A, lda, B, ldb, 0, q, empty);
    if (st != FGEMM_OK) return st;
    if (!forward(q, bias, act, Z, ldz, beta, R, ldr, Y, ldy)) return FGEMM_ERR_INVALID_VALUE;
    return empty ? FGEMM_OK : run(q, nullptr, workspace, workspace_bytes, stream);
}

fgemm_status fgemm_gemm16_grad(fgemm_dtype type, fgemm_dtype out_type, fgemm_op transa, fgemm_op transb, int M, int N, int K,
                               float alpha, const void *A, int lda, const void *B, int ldb, fgemm_activation act,
                               const void *Z, int ldz, void *Y, int ldy, float *col_sums, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream)
{
    Product q;
    bool empty;
    const fgemm_status st = product(type, out_type, transa, transb, 1, M, N, K, nullptr, false, alpha, A, lda, B, ldb, 0, q, empty);
    if (st != FGEMM_OK) return st;
    if (!backward(q, act, Z, ldz, Y, ldy, col_sums)) return FGEMM_ERR_INVALID_VALUE;
    if (empty) return zero(col_sums, (size_t)N, stream);
    return run(q, col_sums, workspace, workspace_bytes, stream);
}

fgemm_status fgemm_gemm16_grouped(fgemm_dtype type, fgemm_dtype out_type, fgemm_op transb, int groups, int M, int N, int K,
                                  const int *offsets, float alpha, const void *A, int lda, const void *B, int ldb,
                                  long long strideB, const float *bias, fgemm_activation act, void *Z, int ldz, float beta,
                                  const void *R, int ldr, void *Y, int ldy, void *workspace, size_t workspace_bytes,
                                  cudaStream_t stream)
{
    Product q;
    bool empty;
    const fgemm_status st =
        product(type, out_type, FGEMM_OP_N, transb, groups, M, N, K, offsets, true, alpha, A, lda, B, ldb, strideB, q, empty);
    if (st != FGEMM_OK) return st;
    if (!forward(q, bias, act, Z, ldz, beta, R, ldr, Y, ldy)) return FGEMM_ERR_INVALID_VALUE;
    return empty ? FGEMM_OK : run(q, nullptr, workspace, workspace_bytes, stream);
}

fgemm_status fgemm_gemm16_grouped_grad(fgemm_dtype type, fgemm_dtype out_type, fgemm_op transb, int groups, int M, int N, int K,
                                       const int *offsets, float alpha, const void *A, int lda, const void *B, int ldb,
                                       long long strideB, fgemm_activation act, const void *Z, int ldz, void *Y, int ldy,
                                       float *col_sums, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    Product q;
    bool empty;
    const fgemm_status st =
        product(type, out_type, FGEMM_OP_N, transb, groups, M, N, K, offsets, true, alpha, A, lda, B, ldb, strideB, q, empty);
    if (st != FGEMM_OK) return st;
    if (!backward(q, act, Z, ldz, Y, ldy, col_sums)) return FGEMM_ERR_INVALID_VALUE;
    if (empty) return zero(col_sums, (size_t)N * (size_t)groups, stream);
    return run(q, col_sums, workspace, workspace_bytes, stream);
}

fgemm_status fgemm_gemm16_weight_grad(fgemm_dtype type, fgemm_dtype out_type, int groups, int M, int N, int K,
                                      const int *offsets, float alpha, const void *A, int lda, const void *G, int ldg,
                                      float beta, void *C, int ldc, long long strideC, void *workspace,
                                      size_t workspace_bytes, cudaStream_t stream)
{
    if (!valid_types(type, out_type) || groups < 1 || M < 0 || N < 0 || K < 0) return FGEMM_ERR_INVALID_VALUE;
    if (!valid_ld(K, lda) || !valid_ld(N, ldg) || !valid_ld(N, ldc) || strideC < 0) return FGEMM_ERR_INVALID_VALUE;
    if (N == 0 || K == 0) return FGEMM_OK;
    // Outputs of different groups must not share elements.
    if (groups > 1 && strideC < (long long)(K - 1) * ldc + N) return FGEMM_ERR_INVALID_VALUE;
    if (!valid_matrix(C, out_type) || !offsets || !aligned(offsets, 4)) return FGEMM_ERR_INVALID_VALUE;
    if (M > 0 && alpha != 0.0f && (!valid_matrix(A, type) || !valid_matrix(G, type))) return FGEMM_ERR_INVALID_VALUE;
    if (groups > FGEMM_MAX_GROUPS) return FGEMM_ERR_NOT_SUPPORTED;
    Product q{};
    q.type = type;
    q.out_type = out_type;
    q.M = K;
    q.N = N;
    q.K = M;
    q.ta = 1;
    q.alpha = alpha;
    q.a = A;
    q.b = G;
    q.lda = lda;
    q.ldb = ldg;
    q.ragged = RAGGED_DEPTH;
    q.groups = groups;
    q.offsets = offsets;
    q.beta = beta;
    q.r = C;
    q.ldr = ldc;
    q.y = C;
    q.ldy = ldc;
    q.stride_y = strideC;
    return run(q, nullptr, workspace, workspace_bytes, stream);
}

fgemm_status fgemm_act16_grad(fgemm_dtype type, int groups, int M, int N, const int *offsets, fgemm_activation act, const void *G,
                              int ldg, const void *Z, int ldz, void *D, int ldd, float *col_sums, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream)
{
    if (!valid_type(type) || !valid_act(act) || groups < 1 || M < 0 || N < 0) return FGEMM_ERR_INVALID_VALUE;
    if (groups > 1 && !offsets) return FGEMM_ERR_INVALID_VALUE;
    if (!valid_ld(N, ldg) || (act != FGEMM_ACT_NONE && !valid_ld(N, ldz)) || (D && !valid_ld(N, ldd)))
        return FGEMM_ERR_INVALID_VALUE;
    if (!D && !col_sums) return FGEMM_ERR_INVALID_VALUE;
    if (!aligned(offsets, 4) || !aligned(col_sums, 4)) return FGEMM_ERR_INVALID_VALUE;
    if (groups > FGEMM_MAX_GROUPS) return FGEMM_ERR_NOT_SUPPORTED;
    if (N == 0) return FGEMM_OK;
    if (M == 0) return zero(col_sums, (size_t)N * (size_t)groups, stream);
    if (!valid_matrix(G, type) || (act != FGEMM_ACT_NONE && !valid_matrix(Z, type)) || (D && !valid_matrix(D, type)))
        return FGEMM_ERR_INVALID_VALUE;
    if (col_sums && (!workspace || !aligned(workspace, 16) || workspace_bytes < partial_bytes(groups, M, N)))
        return FGEMM_ERR_INVALID_VALUE;
    if (!dims_supported(M, N, 0)) return FGEMM_ERR_NOT_SUPPORTED;
    ActGrad p{};
    p.type = type;
    p.act = act;
    p.groups = groups;
    p.M = M;
    p.N = N;
    p.offsets = offsets;
    p.g = G;
    p.z = act != FGEMM_ACT_NONE ? Z : nullptr;
    p.d = D;
    p.ldg = ldg;
    p.ldz = ldz;
    p.ldd = ldd;
    p.partial = col_sums ? static_cast<float *>(workspace) : nullptr;
    return launch_act_grad(p, col_sums, stream);
}

int fgemm_gemm16_plan(fgemm_dtype out_type, int grouped, int groups, int M, int N, int K, int sums, int num_sms)
{
    if (grouped < 0 || grouped > 2 || groups < 1 || groups > FGEMM_MAX_GROUPS || M < 1 || N < 1 || K < 1 || num_sms < 2 ||
        !dims_supported(M, N, K))
        return -1;
    const long long go = one_go(out_type, sums != 0);
    const Plan plan = grouped == 2 ? plan_product(K, N, M, RAGGED_DEPTH, groups, false, go, num_sms)
                                   : plan_product(M, N, K, grouped ? RAGGED_ROWS : RAGGED_NONE, groups, sums != 0, go, num_sms);
    return 16384 * plan.in_turns + 8192 * plan.pair + 16 * plan.nt + plan.ranks;
}

}  // extern "C"
