// gemm16_slices.h -- the slices that the rows of groups are cut into (the elementwise gradient's), as the kernels
// count them.  Plain C++ as well, so that the counting is tested on the CPU.
//
// Offsets come from the caller's device memory unseen by the host: each is clamped to 0 .. M, and nothing here relies
// on their order.  Out of order, the rows of all groups may come to groups / 2 times M, and their slices to more than
// an int holds (1024 groups that alternate between 0 and M, 64 rows a slice: from M = 2^28 on).
#pragma once

#ifdef __CUDACC__
#define FGEMM_SLICES_FN __host__ __device__ __forceinline__
#else
#define FGEMM_SLICES_FN inline
#endif

namespace fgemm {
namespace h16 {

FGEMM_SLICES_FN int within(int x, int most) { return x < 0 ? 0 : x > most ? most : x; }

// Rows of group e, the first at `first`.
FGEMM_SLICES_FN int rows_of(const int *offsets, int e, int M, int &first)
{
    first = within(offsets[e], M);
    const int rows = within(offsets[e + 1], M) - first;
    return rows < 0 ? 0 : rows;
}

FGEMM_SLICES_FN int slices_of(const int *offsets, int e, int M, int height)
{
    int first;
    return (rows_of(offsets, e, M, first) + height - 1) / height;
}

// Slices of the groups i, i + step, ... before e.
FGEMM_SLICES_FN long long slices_before(const int *offsets, int i, int step, int e, int M, int height)
{
    long long sum = 0;
    for (; i < e; i += step) sum += slices_of(offsets, i, M, height);
    return sum;
}

// Rows from .. to of partial sums, inside the `most` that there are.
struct PartialRows {
    long long from, to;
};

FGEMM_SLICES_FN PartialRows inside(long long from, long long to, long long most)
{
    from = from < 0 ? 0 : from > most ? most : from;
    return PartialRows{from, to > most ? most : to};
}

}  // namespace h16
}  // namespace fgemm
