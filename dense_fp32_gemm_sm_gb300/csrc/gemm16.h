// gemm16.h -- what the units of the 16-bit layers share: the arguments of a product and of the
// passes around it, and the launchers behind the C entries.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fgemm.h"

namespace fgemm {
namespace h16 {

// A product, or one a group:  P = alpha op(A) op(B),  then the epilogue.
//   RAGGED_NONE   one product
//   RAGGED_ROWS   group e: rows offsets[e] .. offsets[e+1] of A and of the outputs, with B_e
//   RAGGED_DEPTH  group e: those rows are what is summed over, Y_e is an output of its own
enum Ragged { RAGGED_NONE = 0, RAGGED_ROWS = 1, RAGGED_DEPTH = 2 };

struct Product {
    fgemm_dtype type, out_type;
    int M, N, K;  // of the outputs (all groups' rows for RAGGED_ROWS), and the depth (all groups' for RAGGED_DEPTH)
    int ta, tb;   // A stored K x M, B stored N x K
    float alpha;
    const void *a, *b;
    long long lda, ldb, stride_b;
    int ragged, groups;
    const int *offsets;  // device, groups + 1
    // Epilogue.  slope == 0: Y = act(P + bias) + beta R, Z (if any) = P + bias.  slope != 0: Y = P act'(Z).
    int act, slope;
    const float *bias;  // N floats a group
    void *z;
    long long ldz;
    float beta;
    const void *r;
    long long ldr;
    void *y;
    long long ldy, stride_y;
    // Column sums of Y: partial ones, `partials` rows of N floats of room, and the first row of each group.
    float *partial;
    int *partial_start;
    long long partials;
};

// How a product runs: tiles of 128 (pair: 256) columns of the output by at most nt rows; a tile's
// depth divided among the `ranks` CTAs of a cluster (1: whole tiles by persistent CTAs or pairs);
// and whether sums over a long depth, of more than `one_go`, are added up in turns.
struct Plan {
    int pair, nt, ranks, in_turns;
};
Plan plan_product(long long M, long long N, long long K, int ragged, long long groups, bool sums, long long one_go,
                  int sms);

// Depth whose products the tensor core adds up at a time, where a longer one is added up in turns.
constexpr int LONG_DEPTH = 768;

// The depth that is added up in one go.  The tensor core cuts where FP32 addition rounds, so a sum falls short by 0.8e-9 of itself
// for each entry of depth where its addends are of one sign (F16, depth 2^16: 5.0e-5; 2^18: 2.1e-4; 2^20: 8.6e-4; in turns 4e-6
// at any of these).  Kept in FP32, or summed on, that counts from one turn on; rounded to 16 bits, from where it is
// more than a thirtieth of half a step: 1.3e-5 of F16's 4.9e-4 at 2^14, 1e-4 of BF16's 3.9e-3 at 2^17.
inline long long one_go(fgemm_dtype out_type, bool sums)
{
    if (sums || out_type == FGEMM_F32) return LONG_DEPTH;
    return out_type == FGEMM_F16 ? 1 << 14 : 1 << 17;
}

// Least rows of a tile where column sums are wanted, which bounds their partial sums.
constexpr int SUMS_ROWS = 32;
// Partial sums of columns: two of every tile of rows, or (act16_grad) one of every slice, of 16 rows at least.
inline long long partial_rows(long long groups, long long M) { return 2 * ((M + SUMS_ROWS - 1) / SUMS_ROWS + groups); }

fgemm_status launch_product(const Product &q, cudaStream_t stream);
template <class T, class O> fgemm_status launch_product_type(const Product &q, const Plan &plan, cudaStream_t stream);

// Copies of `batch` matrices of 16-bit elements, rows x cols, whose rows start on 16 bytes at y.  pieces 0: none.
struct Realign {
    const uint16_t *x;
    long long ldx, stride_x, rows, pieces;
    int cols, per_row;  // 16-byte pieces of a row
    uint4 *y;
};
Realign realign(const void *x, long long ldx, long long stride_x, long long rows, int cols, long long batch, void *y);
fgemm_status launch_realign(const Realign &a, const Realign &b, cudaStream_t stream);

struct ActGrad {
    fgemm_dtype type;
    int act, groups, M, N;
    const int *offsets;  // or null: one group of all rows
    const void *g, *z;
    void *d;
    long long ldg, ldz, ldd;
    float *partial;  // or null: no sums
};
// The gradient, and (partial not null) its column sums, N floats a group.
fgemm_status launch_act_grad(const ActGrad &p, float *sums, cudaStream_t stream);

// sums[e][j] = the partial rows of group e, of `most` there may be, of column j, in order: rows
// start[e] .. start[e+1], or (start null) those of the slices that `of` leaves.
fgemm_status launch_sums(const float *partial, long long most, const int *start, const ActGrad *of, int groups, int N, float *sums,
                         cudaStream_t stream);

}  // namespace h16
}  // namespace fgemm
