// mxfp4_gemm.cu -- the product of two quantised matrices.
//
// C[i][j] = act(alpha * sum_b 2^(sa + sb - 254) * sum_{k in block b} a[i][k] b[j][k] + beta C + bias)
#include <algorithm>

#include "fgemm_internal.h"
#include "mxfp4_device.cuh"

namespace fgemm {
namespace mx {
namespace {

constexpr int TILE = 64;

// One 64 x 64 tile of C per CTA, 4 x 4 per thread; both operands' codes as FP32 in shared
// memory, one block of 32 at a time, whose sum then gets both scales at once (their product
// may be in range where a factor times a code is not).
template <class T>
__global__ void __launch_bounds__(256) gemm_simple_kernel(const GemmArgs g)
{
    __shared__ float as[BLOCK][TILE + 1], bs[BLOCK][TILE + 1];
    __shared__ int ea[TILE], eb[TILE];  // scale bytes, from 127; far out for NaN
    const int t = threadIdx.x, tx = t % 16, ty = t / 16;
    const long long tiles_n = (g.N + TILE - 1) / TILE, tiles = tiles_n * ((g.M + TILE - 1) / TILE);
    const long long blocks = blocks_of(g.K), atoms = atoms_of(blocks);
    for (long long w = blockIdx.x; w < tiles; w += gridDim.x) {
        const long long i0 = w / tiles_n * TILE, j0 = w % tiles_n * TILE;
        float acc[4][4] = {};
        for (long long b = 0; b < blocks; ++b) {
            if (t < 2 * TILE) {
                const bool first = t < TILE;
                const int row = t % TILE;
                const long long r = (first ? i0 : j0) + row;
                const bool in = r < (first ? g.M : g.N);
                uint4 c = make_uint4(0, 0, 0, 0);
                int s = 0;
                if (in) {
                    c = *reinterpret_cast<const uint4 *>((first ? g.a + r * g.lda : g.b + r * g.ldb) + 16 * b);
                    s = (first ? g.a_scales : g.b_scales)[scale_offset(r, b, atoms)];
                }
                (first ? ea : eb)[row] = s - 127;
                const uint32_t words[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[8];
                    decode8(words[q], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) (first ? as : bs)[8 * q + k][row] = s == 255 ? __uint_as_float(0x7FFFFFFFu) : x[k];
                }
            }
            __syncthreads();
            float dot[4][4] = {};
#pragma unroll 8
            for (int k = 0; k < BLOCK; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) dot[i][j] = fmaf(as[k][ty + 16 * i], bs[k][tx + 16 * j], dot[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += ldexpf(dot[i][j], ea[ty + 16 * i] + eb[tx + 16 * j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
                if (r >= g.M || c >= g.N) continue;
                T *const out = static_cast<T *>(g.c) + r * g.ldc + c;
                float o = g.alpha * acc[i][j];
                if (g.beta != 0.0f) o = fmaf(g.beta, to_float(*out), o);
                if (g.bias) o += g.bias[c];
                if (g.relu) o = fmaxf(o, 0.0f);
                *out = from_float<T>(o);
            }
    }
}

template <class T>
fgemm_status run_gemm(const GemmArgs &g, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    const long long tiles = ((g.N + TILE - 1) / TILE) * (long long)((g.M + TILE - 1) / TILE);
    gemm_simple_kernel<T><<<(unsigned)std::min<long long>(tiles, 8ll * sms), 256, 0, stream>>>(g);
    return cudaGetLastError() == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
}

}  // namespace

fgemm_status launch_gemm(fgemm_dtype type, const GemmArgs &g, cudaStream_t stream)
{
    switch (type) {
    case FGEMM_F32: return run_gemm<float>(g, stream);
    case FGEMM_BF16: return run_gemm<__nv_bfloat16>(g, stream);
    default: return run_gemm<__half>(g, stream);
    }
}

}  // namespace mx
}  // namespace fgemm
