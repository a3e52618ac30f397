// gemm16_rows.cu -- the passes around the 16-bit products: rows copied to 16-byte boundaries, the
// gradient through an activation with its column sums, and the adding up of partial column sums.
#include <cuda_runtime.h>

#include "fgemm_internal.h"
#include "gemm16.h"
#include "gemm16_device.cuh"
#include "gemm16_slices.h"
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

template <class T> __device__ __forceinline__ uint32_t bits_of(T x) { return reinterpret_cast<const uint16_t &>(x); }

// D = G act'(Z) for a slice of a group's rows (`height` at most) by 256 columns, and its column sums.  The
// slices of all groups are counted through, so that a group of many rows has many blocks.
// VEC: a lane's eight columns are consecutive, 16 bytes an access; else 32 apart, for any alignment.
// Memory bounds it without an activation and through ReLU (8192 x 11008: 60 and 85 us, 6.0 and 6.4 TB/s), 50
// instructions an element through GELU and SiLU (131 and 111 us), a fifth of them for the few that take the definition.
// (Those in a queue of the warp's or the block's, evaluated 32 at a time: 131 and 119 us, 133 and 125.)
// Rows that a warp has on their way at a time, and blocks an SM has registers for.  (8192 x 11008, none: 60 us with 4 and 2, 78 with
// 2 and 4; through ReLU 84 and 85; GELU and SiLU, which arithmetic bounds, 164 and 132, 153 and 112.)
__host__ __device__ constexpr int act_batch(int act) { return act == FGEMM_ACT_NONE ? 4 : 2; }
__host__ __device__ constexpr int act_blocks(int act) { return act == FGEMM_ACT_NONE ? 2 : 4; }

template <class T, bool VEC, int ACT>
__global__ void __launch_bounds__(32 * ACT_WARPS, act_blocks(ACT)) act_grad_kernel(ActGrad p, int strips, int height)
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
    constexpr bool gated = ACT != FGEMM_ACT_NONE;
    constexpr int BATCH = act_batch(ACT);
    const int rows = (int)(to - from);
    const long long ldg = p.ldg, ldz = p.ldz, ldd = p.ldd;
    // At this slice's first row and the lane's first column.
    const T *const G = static_cast<const T *>(p.g) + from * ldg + column(0);
    const T *const Z = gated ? static_cast<const T *>(p.z) + from * ldz + column(0) : nullptr;
    T *const D = p.d ? static_cast<T *>(p.d) + from * ldd + column(0) : nullptr;
    const bool in = column(0) < p.N;  // (VEC: all eight are, then)
    // Eight elements, 32 apart unless VEC, as words of two.
    auto load = [&](const T *x, uint32_t (&w)[4]) {
        if (VEC) {
            if (in) *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const uint32_t low = column(j) < p.N ? bits_of(x[32 * j]) : 0, high = column(j + 1) < p.N ? bits_of(x[32 * j + 32]) : 0;
                w[j / 2] = low | high << 16;
            }
        }
    };
#pragma unroll 1
    for (int r0 = warp; r0 < rows; r0 += BATCH * ACT_WARPS) {
        __align__(16) uint32_t g[BATCH][4], z[BATCH][4];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * ACT_WARPS;
            if (r >= rows) break;
            load(G + r * ldg, g[i]);
            if (gated) load(Z + r * ldz, z[i]);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * ACT_WARPS;
            if (r >= rows) break;
            __align__(16) uint32_t d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v0 = from_bits<T>(g[i][j]), v1 = from_bits<T>(g[i][j] >> 16);
                d[j] = through_exactly<T, ACT>(v0, v1, gated ? from_bits<T>(z[i][j]) : 0.0f, gated ? from_bits<T>(z[i][j] >> 16) : 0.0f);
                sum[2 * j] += v0;
                sum[2 * j + 1] += v1;
            }
            if (D == nullptr) continue;
            if (VEC) {
                if (in) *reinterpret_cast<uint4 *>(D + r * ldd) = *reinterpret_cast<const uint4 *>(d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (column(j) < p.N) D[r * ldd + 32 * j] = reinterpret_cast<const T *>(d)[j];
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
    PartialRows rows{0, most};
    if (start) {
        rows = inside(start[e], start[e + 1], most);
    } else if (offsets) {
        long long before = slices_before(offsets, lane, 32, e, M, height);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
        rows = inside(before, before + slices_of(offsets, e, M, height), most);
    }
    float sum = 0.0f;
    if (n < N) {
#pragma unroll 4
        for (long long r = rows.from + warp; r < rows.to; r += 8) sum += partial[r * N + n];
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

template <class T, bool VEC>
static auto act_grad_of(int act)
{
    return act == FGEMM_ACT_NONE   ? act_grad_kernel<T, VEC, FGEMM_ACT_NONE>
           : act == FGEMM_ACT_RELU ? act_grad_kernel<T, VEC, FGEMM_ACT_RELU>
           : act == FGEMM_ACT_GELU ? act_grad_kernel<T, VEC, FGEMM_ACT_GELU>
                                   : act_grad_kernel<T, VEC, FGEMM_ACT_SILU>;
}

fgemm_status launch_act_grad(const ActGrad &p, float *sums, cudaStream_t stream)
{
    const int strips = (p.N - 1) / ACT_COLUMNS + 1;
    const long long blocks = strips * most_slices(p);
    if (blocks > 0x7FFFFFFF) return FGEMM_ERR_NOT_SUPPORTED;
    const bool vec = p.N % 8 == 0 && vectors(p.g, p.ldg) && vectors(p.z, p.ldz) && vectors(p.d, p.ldd);
    const auto kernel = p.type == FGEMM_BF16 ? (vec ? act_grad_of<__nv_bfloat16, true>(p.act) : act_grad_of<__nv_bfloat16, false>(p.act))
                                             : (vec ? act_grad_of<__half, true>(p.act) : act_grad_of<__half, false>(p.act));
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
