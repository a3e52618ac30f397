// gemm16_rows.cu -- the passes around the 16-bit products: rows copied to 16-byte boundaries, the
// gradient through an activation with its column sums, and the adding up of partial column sums.
#include <cuda_runtime.h>

#include "fgemm_internal.h"
#include "gemm16.h"
#include "gemm16_device.cuh"
#include "mxfp4_launch.h"

namespace fgemm {
namespace h16 {
namespace {

// ---- rows on 16-byte boundaries ----------------------------------------------------------

// One or two matrices (or batches of them), the second's pieces behind the first's: a thread makes 16 bytes of a
// row.  Bounded by its reads, 2 bytes a lane and instruction, of which eight share their sectors in L1.
__global__ void __launch_bounds__(256) realign_kernel(Realign a, Realign b)
{
    after_previous_kernel();
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < a.pieces + b.pieces; i += gridDim.x * 256ll) {
        const bool second = i >= a.pieces;
        const Realign &m = second ? b : a;
        const long long piece = second ? i - a.pieces : i, row = piece / m.per_row, matrix = row / m.rows;
        const int c0 = (int)(piece - row * m.per_row) * 8;
        const uint16_t *const src = m.x + matrix * m.stride_x + (row - matrix * m.rows) * m.ldx + c0;
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c0 + j < m.cols ? src[j] : 0;
        m.y[piece] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}

// ---- the gradient through an activation --------------------------------------------------

constexpr int ACT_COLUMNS = 256;  // of a block: eight a lane
constexpr int ACT_WARPS = 8;      // rows of a block at a time

// Rows of group e, the first at `first`.
__device__ __forceinline__ int rows_of(const int *offsets, int e, int M, int &first)
{
    first = max(0, min(offsets[e], M));
    return max(max(0, min(offsets[e + 1], M)) - first, 0);
}

// D = G act'(Z) for a slice of a group's rows (`height` at most) by 256 columns, and its column sums.  The
// slices of all groups are counted through, so that a group of many rows has many blocks.
// VEC: a lane's eight columns are consecutive, 16 bytes an access; else 32 apart, for any alignment.
template <class T, bool VEC>
__global__ void __launch_bounds__(32 * ACT_WARPS, 4) act_grad_kernel(ActGrad p, int strips, int height)
{
    __shared__ float sums[ACT_WARPS][ACT_COLUMNS];
    after_previous_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strip = blockIdx.x % strips, part = blockIdx.x / strips;
    long long from = (long long)part * height, to = min(from + height, (long long)p.M);
    if (p.offsets) {
        // 32 groups at a time: the one whose slices, added up, pass this block's.
        int before = 0, e0 = 0;
        unsigned found = 0;
        for (; e0 < p.groups; e0 += 32) {
            const int e = e0 + lane;
            int first = 0;
            const int rows = e < p.groups ? rows_of(p.offsets, e, p.M, first) : 0, own = (rows + height - 1) / height;
            int sum = own;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int other = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += other;
            }
            found = __ballot_sync(0xFFFFFFFFu, before + sum > part);
            if (found) {
                const int at = __ffs(found) - 1;
                const long long start = first + (long long)(part - before - (sum - own)) * height;
                from = __shfl_sync(0xFFFFFFFFu, start, at);
                to = __shfl_sync(0xFFFFFFFFu, min(start + height, (long long)first + rows), at);
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (!found) return;  // (there is room for a short slice of every group)
    }
    const int c0 = strip * ACT_COLUMNS;
    auto column = [&](int j) { return c0 + (VEC ? 8 * lane + j : lane + 32 * j); };
    float sum[8] = {};
    const T *const G = static_cast<const T *>(p.g);
    const T *const Z = static_cast<const T *>(p.z);
    T *const D = static_cast<T *>(p.d);
    const bool gated = p.act != FGEMM_ACT_NONE;
    if (column(0) < p.N) {
        // Two rows of a warp are on their way at a time.  (Four leave two blocks an SM in place of four.)
        constexpr int BATCH = 2;
        for (long long r0 = from + warp; r0 < to; r0 += BATCH * ACT_WARPS) {
            __align__(16) T g[BATCH][8], z[BATCH][8];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const long long r = r0 + i * ACT_WARPS;
                if (r >= to) break;
                if (VEC) {
                    *reinterpret_cast<uint4 *>(g[i]) = *reinterpret_cast<const uint4 *>(G + r * p.ldg + column(0));
                    if (gated) *reinterpret_cast<uint4 *>(z[i]) = *reinterpret_cast<const uint4 *>(Z + r * p.ldz + column(0));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = column(j) < p.N;
                        g[i][j] = in ? G[r * p.ldg + column(j)] : from_float<T>(0.0f);
                        if (gated) z[i][j] = in ? Z[r * p.ldz + column(j)] : from_float<T>(0.0f);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const long long r = r0 + i * ACT_WARPS;
                if (r >= to) break;
                __align__(16) uint32_t d[4];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float v0 = to_float(g[i][j]), v1 = to_float(g[i][j + 1]);
                    if (gated) through_exactly<T>(v0, v1, to_float(z[i][j]), to_float(z[i][j + 1]), p.act);
                    sum[j] += v0;
                    sum[j + 1] += v1;
                    d[j / 2] = pack<T>(v0, v1);
                }
                if (D) {
                    if (VEC) {
                        *reinterpret_cast<uint4 *>(D + r * p.ldd + column(0)) = *reinterpret_cast<const uint4 *>(d);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (column(j) < p.N) D[r * p.ldd + column(j)] = reinterpret_cast<const T *>(d)[j];
                    }
                }
            }
        }
    }
    if (p.partial) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[warp][column(j) - c0] = sum[j];
        __syncthreads();
        const int n = c0 + (int)threadIdx.x;
        if (n < p.N) {
            float total = 0.0f;
#pragma unroll
            for (int w = 0; w < ACT_WARPS; ++w) total += sums[w][threadIdx.x];
            p.partial[(long long)part * p.N + n] = total;
        }
    }
}

// ---- partial column sums -----------------------------------------------------------------

// 32 columns of a group by 8 warps, each adding up every eighth row; then the warps' sums, in order.
// start: the groups' first partial rows; null: those of act_grad_kernel's slices.
__global__ void __launch_bounds__(256) sums_kernel(const float *partial, long long most, const int *start, const int *offsets, int M,
                                                   int height, int strips, int N, float *sums)
{
    __shared__ float part[8][32];
    after_previous_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strip = blockIdx.x % strips, e = blockIdx.x / strips, n = strip * 32 + lane;
    long long from = 0, to = most;
    if (start) {
        from = start[e];
        to = start[e + 1];
    } else if (offsets) {
        int first, before = 0;
        for (int i = lane; i < e; i += 32) before += (rows_of(offsets, i, M, first) + height - 1) / height;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
        from = before;
        to = from + (rows_of(offsets, e, M, first) + height - 1) / height;
    }
    to = min(to, most);
    float sum = 0.0f;
    if (n < N) {
#pragma unroll 4
        for (long long r = from + warp; r < to; r += 8) sum += partial[r * N + n];
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && n < N) {
#pragma unroll
        for (int w = 1; w < 8; ++w) sum += part[w][lane];
        sums[(long long)e * N + n] = sum;
    }
}

bool vectors(const void *p, long long ld) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0); }

fgemm_status status(cudaError_t e) { return e == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH; }

}  // namespace

Realign realign(const void *x, long long ldx, long long stride_x, long long rows, int cols, long long batch, void *y)
{
    const int per_row = (cols + 7) / 8;
    return Realign{static_cast<const uint16_t *>(x), ldx, stride_x, rows, rows * batch * per_row, cols, per_row, static_cast<uint4 *>(y)};
}

fgemm_status launch_realign(const Realign &a, const Realign &b, cudaStream_t stream)
{
    const long long blocks = (a.pieces + b.pieces + 255) / 256;
    const dim3 grid((unsigned)(blocks < 152 * 64 ? blocks : 152 * 64));
    return status(mx::launch(realign_kernel, grid, 256, 0, stream, 1, a, b));
}

// Rows of a slice: 64, fewer (16 at least, two a warp) where there are not blocks for all SMs: of 77 x 1237 a
// warp's eight rows, some of whose values take the definition, were 12 us.
static int slice_rows(long long M, long long N)
{
    const long long strips = (N + ACT_COLUMNS - 1) / ACT_COLUMNS, fair = (M * strips / (4 * 152) + 7) / 8 * 8;
    return (int)(fair < 16 ? 16 : fair < 64 ? fair : 64);
}

// Slices there may be: each group's last one may be short.  (partial_rows has room for them.)
static long long most_slices(const ActGrad &p)
{
    const int height = slice_rows(p.M, p.N);
    return p.offsets ? p.M / height + (p.groups < p.M ? p.groups : p.M) : (p.M + height - 1ll) / height;
}

fgemm_status launch_act_grad(const ActGrad &p, float *sums, cudaStream_t stream)
{
    const int strips = (p.N - 1) / ACT_COLUMNS + 1;
    const long long blocks = strips * most_slices(p);
    if (blocks > 0x7FFFFFFF) return FGEMM_ERR_NOT_SUPPORTED;
    const bool vec = p.N % 8 == 0 && vectors(p.g, p.ldg) && vectors(p.z, p.ldz) && vectors(p.d, p.ldd);
    const auto kernel = p.type == FGEMM_BF16 ? (vec ? act_grad_kernel<__nv_bfloat16, true> : act_grad_kernel<__nv_bfloat16, false>)
                                             : (vec ? act_grad_kernel<__half, true> : act_grad_kernel<__half, false>);
    const fgemm_status st = status(mx::launch(kernel, dim3((unsigned)blocks), 32 * ACT_WARPS, 0, stream, 1, p, strips, slice_rows(p.M, p.N)));
    if (st != FGEMM_OK || !p.partial) return st;
    return launch_sums(p.partial, most_slices(p), nullptr, &p, p.groups, p.N, sums, stream);
}

fgemm_status launch_sums(const float *partial, long long most, const int *start, const ActGrad *of, int groups, int N, float *sums,
                         cudaStream_t stream)
{
    const int strips = (N - 1) / 32 + 1;
    if ((long long)strips * groups > 0x7FFFFFFF) return FGEMM_ERR_NOT_SUPPORTED;
    return status(mx::launch(sums_kernel, dim3((unsigned)(strips * groups)), 256, 0, stream, 1, partial, most, start,
                             of ? of->offsets : nullptr, of ? of->M : 0, of ? slice_rows(of->M, of->N) : 1, strips, N, sums));
}

}  // namespace h16
}  // namespace fgemm
