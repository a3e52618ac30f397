// mxfp4.h -- what the MXFP4 units share: the layout of a quantised matrix and the
// launchers behind the C entries (the layout itself is described in include/fgemm.h).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fgemm.h"

namespace fgemm {
namespace mx {

constexpr int BLOCK = 32;       // elements that share a scale
constexpr int ATOM_ROWS = 128;  // a scale atom: 128 rows x 4 blocks, 512 bytes
constexpr int ATOM_BYTES = 512;

__host__ __device__ constexpr long long blocks_of(long long cols) { return (cols + BLOCK - 1) / BLOCK; }
__host__ __device__ constexpr long long atoms_of(long long blocks) { return (blocks + 3) / 4; }

// Byte offset of the scale of row r, block b; `atoms` = atoms_of(blocks) of the matrix.
__host__ __device__ constexpr long long scale_offset(long long r, long long b, long long atoms)
{
    return ((r / ATOM_ROWS) * atoms + b / 4) * ATOM_BYTES + (r % 32) * 16 + ((r % ATOM_ROWS) / 32) * 4 +
           b % 4;
}

struct QuantParams {
    const void *x;     // M x N, leading dimension ldx
    const void *gate;  // the layer's output (its gradient's gate), or null
    long long ldx, ldgate;
    int M, N;
    uint8_t *row_codes, *row_scales;
    long long ld_row;
    uint8_t *col_codes, *col_scales;
    long long ld_col;
    float *bias_grad;  // or null
    float *partial;    // one partial column sum per 128 rows
};
fgemm_status launch_quantize(fgemm_dtype type, const QuantParams &p, cudaStream_t stream);

struct DequantParams {
    const uint8_t *codes, *scales;
    long long ld;
    void *x;
    long long ldx;
    int M, N;
};
fgemm_status launch_dequantize(fgemm_dtype type, const DequantParams &p, cudaStream_t stream);

struct GemmArgs {
    int M, N, K;
    float alpha, beta;
    const uint8_t *a, *a_scales, *b, *b_scales;
    long long lda, ldb;
    void *c;
    long long ldc;
    const float *bias;
    int relu;
    int dependent;  // A is written by the quantising kernel launched just before, B is not
};
fgemm_status launch_gemm(fgemm_dtype type, const GemmArgs &g, cudaStream_t stream);

// How a product runs.  nt 16, 32, 64: tiles of 128 rows of B by nt of A, each tile's K divided
// among the `ranks` CTAs of a cluster.  nt 128: tiles of 128 x 128 by persistent CTAs.
// PAIRS_192, PAIRS_256: tiles of 256 rows of B by 192 or 256 of A by persistent pairs of CTAs.
enum { PAIRS_192 = 384, PAIRS_256 = 512 };
struct GemmPlan {
    int nt, ranks;
};
GemmPlan plan_gemm(long long M, long long N, long long K, int element_size, int sms);

// A layer on at most LINEAR_ROWS unquantised tokens in one kernel: every CTA of a cluster of
// eight at most quantises its part of them into FUSED_SMEM bytes of shared memory.
constexpr int LINEAR_ROWS = 4;
constexpr int FUSED_SMEM = 64 * 1024;
bool linear_fused(long long M, long long K);
int linear_ranks(long long N, long long K, int sms);  // CTAs of its clusters
fgemm_status launch_linear(fgemm_dtype type, const void *x, long long ldx, const GemmArgs &g, cudaStream_t stream);

}  // namespace mx
}  // namespace fgemm
