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
    int early;         // let the next kernel of the stream start (it waits before it reads)
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
    int dependent;  // A is written by the quantising kernel launched just before, with `early`
};
fgemm_status launch_gemm(fgemm_dtype type, const GemmArgs &g, cudaStream_t stream);

// How a product runs: tiles of `nt` rows of A by 128 rows of B, each tile's K divided among
// `ranks` CTAs of a cluster (0: whole tiles, by persistent CTAs; nt is then 128, or 512 for
// pairs of CTAs with 256 rows of A, 384 for pairs with 192).
struct GemmPlan {
    int nt, ranks;
};
GemmPlan plan_gemm(long long M, long long N, long long K, int sms);

// A layer on at most LINEAR_ROWS unquantised tokens in one kernel: every CTA of a cluster of
// eight at most quantises its part of them into FUSED_SMEM bytes of shared memory.
constexpr int LINEAR_ROWS = 4;
constexpr int FUSED_SMEM = 64 * 1024;
bool linear_fused(long long M, long long K);
GemmPlan plan_linear(long long N, long long K, int sms);
fgemm_status launch_linear(fgemm_dtype type, const void *x, long long ldx, const GemmArgs &g, cudaStream_t stream);

}  // namespace mx
}  // namespace fgemm
