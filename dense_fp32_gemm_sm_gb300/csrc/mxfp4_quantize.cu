// mxfp4_quantize.cu -- quantising a matrix to MXFP4 along its rows, its columns or both,
// with ReLU's gate and the bias's gradient on the way, and the way back.
//
// A block's scale is 2^(floor(log2 max|x|) - 2) and its codes are x / scale rounded to
// E2M1.  Both are exact but for that one rounding: the exponent comes from the bits of the
// largest magnitude and the division is a multiplication with a power of two.
#include <algorithm>
#include <atomic>

#include "ctx_id.h"
#include "fgemm_internal.h"
#include "mxfp4_device.cuh"

namespace fgemm {
namespace mx {
namespace {

constexpr int TILE = 128;  // a tile is 128 x 128: one scale atom in each direction
constexpr int THREADS = 256;
// Shared-memory tile in floats: blocks of 32 columns are 36 apart and rows 144, with 8 more
// after every 32 rows.  Then a quarter warp's 16-byte loads of four blocks in two rows
// (along rows), and a warp's loads of eight columns in four row blocks (down columns),
// fall on different banks.
constexpr int ROW_PITCH = 144, BLOCK_PITCH = 36, GROUP_PAD = 8;
constexpr int TILE_FLOATS = TILE * ROW_PITCH + (TILE / 32) * GROUP_PAD;
constexpr int SMEM_BYTES = TILE_FLOATS * 4 + 2 * ATOM_BYTES + THREADS * 4;

__device__ __forceinline__ int tile_at(int row, int col)
{
    return row * ROW_PITCH + (row >> 5) * GROUP_PAD + (col >> 5) * BLOCK_PITCH + (col & 31);
}

// One block's 32 values to its 16 bytes of codes; returns the scale byte.
__device__ __forceinline__ uint32_t encode_block(const float (&x)[32], uint4 &codes)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    const uint32_t s = scale_byte(top);
    const float f = inverse_scale(s);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[8 * j + i] * f;
        w[j] = s == 255u ? 0u : encode8(v);
    }
    codes = make_uint4(w[0], w[1], w[2], w[3]);
    return s;
}

template <class T, bool GATED>
__device__ __forceinline__ float element(const QuantParams &p, long long r, long long c)
{
    float v = to_float(static_cast<const T *>(p.x)[r * p.ldx + c]);
    if constexpr (GATED) {
        if (!(to_float(static_cast<const T *>(p.gate)[r * p.ldgate + c]) > 0.0f)) v = 0.0f;
    }
    return v;
}

template <class T, bool GATED>
__global__ void __launch_bounds__(THREADS) quantize_kernel(const QuantParams p, int vec)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *const tile = reinterpret_cast<float *>(smem);
    uint8_t *const row_atom = smem + TILE_FLOATS * 4, *const col_atom = row_atom + ATOM_BYTES;
    float *const sums = reinterpret_cast<float *>(col_atom + ATOM_BYTES);
    const int t = threadIdx.x;
    const long long tiles_n = (p.N + TILE - 1) / TILE, tiles_m = (p.M + TILE - 1) / TILE;
    const long long row_blocks = blocks_of(p.N), col_blocks = blocks_of(p.M);
    constexpr int V = 16 / (int)sizeof(T);  // elements of a 16-byte load
    if (p.early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    for (long long w = blockIdx.x; w < tiles_n * tiles_m; w += gridDim.x) {
        const long long tm = w / tiles_n, tn = w - tm * tiles_n;
        const long long r0 = tm * TILE, c0 = tn * TILE;

        // The tile, as FP32; elements beyond the matrix are 0.
        if (vec && c0 + TILE <= p.N) {
            constexpr int PER_ROW = TILE / V;
#pragma unroll 4
            for (int i = t; i < TILE * PER_ROW; i += THREADS) {
                const int row = i / PER_ROW, col = (i % PER_ROW) * V;
                const long long r = r0 + row, c = c0 + col;
                float v[V];
                if (r < p.M) {
                    T e[V];
                    *reinterpret_cast<uint4 *>(e) = __ldcs(reinterpret_cast<const uint4 *>(
                        static_cast<const T *>(p.x) + r * p.ldx + c));
#pragma unroll
                    for (int k = 0; k < V; ++k) v[k] = to_float(e[k]);
                    if constexpr (GATED) {
                        T y[V];
                        *reinterpret_cast<uint4 *>(y) = __ldcs(reinterpret_cast<const uint4 *>(
                            static_cast<const T *>(p.gate) + r * p.ldgate + c));
#pragma unroll
                        for (int k = 0; k < V; ++k) v[k] = to_float(y[k]) > 0.0f ? v[k] : 0.0f;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k) v[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < V; k += 4)
                    *reinterpret_cast<float4 *>(tile + tile_at(row, col + k)) =
                        make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
        } else {
#pragma unroll 4
            for (int i = t; i < TILE * TILE; i += THREADS) {
                const int row = i / TILE, col = i % TILE;
                tile[tile_at(row, col)] =
                    r0 + row < p.M && c0 + col < p.N ? element<T, GATED>(p, r0 + row, c0 + col) : 0.0f;
            }
        }
        __syncthreads();

        if (p.row_codes) {
#pragma unroll
            for (int i = t; i < TILE * 4; i += THREADS) {
                const int row = i >> 2, b = i & 3;
                const float4 *const src = reinterpret_cast<const float4 *>(tile + tile_at(row, 32 * b));
                float x[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) *reinterpret_cast<float4 *>(x + 4 * k) = src[k];
                uint4 codes;
                const uint32_t s = encode_block(x, codes);
                row_atom[(row % 32) * 16 + (row / 32) * 4 + b] = (uint8_t)s;
                if (r0 + row < p.M && c0 / 32 + b < row_blocks)
                    *reinterpret_cast<uint4 *>(p.row_codes + (r0 + row) * p.ld_row + (c0 / 32 + b) * 16) = codes;
            }
        }
        if (p.col_codes) {
#pragma unroll
            for (int i = t; i < TILE * 4; i += THREADS) {
                const int col = (i >> 5) * 8 + (i & 7), b = (i >> 3) & 3;
                const float *const src = tile + tile_at(32 * b, col);
                float x[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = src[k * ROW_PITCH];
                uint4 codes;
                const uint32_t s = encode_block(x, codes);
                col_atom[(col % 32) * 16 + (col / 32) * 4 + b] = (uint8_t)s;
                if (c0 + col < p.N && r0 / 32 + b < col_blocks)
                    *reinterpret_cast<uint4 *>(p.col_codes + (c0 + col) * p.ld_col + (r0 / 32 + b) * 16) = codes;
            }
        }
        if (p.bias_grad) {
            const int col = t & (TILE - 1), half = t >> 7;
            float sum = 0.0f;
#pragma unroll 8
            for (int k = 0; k < TILE / 2; ++k) sum += tile[tile_at(half * (TILE / 2) + k, col)];
            sums[t] = sum;
        }
        __syncthreads();
        if (t < 32 && p.row_codes)
            reinterpret_cast<uint4 *>(p.row_scales + (tm * atoms_of(row_blocks) + tn) * ATOM_BYTES)[t] =
                reinterpret_cast<const uint4 *>(row_atom)[t];
        if (t >= 32 && t < 64 && p.col_codes)
            reinterpret_cast<uint4 *>(p.col_scales + (tn * atoms_of(col_blocks) + tm) * ATOM_BYTES)[t - 32] =
                reinterpret_cast<const uint4 *>(col_atom)[t - 32];
        if (p.bias_grad && t >= 128 && c0 + t - 128 < p.N)
            (tiles_m == 1 ? p.bias_grad : p.partial + tm * p.N)[c0 + t - 128] = sums[t - 128] + sums[t];
        __syncthreads();
    }
}

// bias_grad[j] = the sum of the partial sums of column j, in the order of the rows.
__global__ void __launch_bounds__(256) bias_grad_kernel(const float *partial, int parts, int N, float *bias_grad)
{
    for (long long j = blockIdx.x * 256ll + threadIdx.x; j < N; j += gridDim.x * 256ll) {
        float s = 0.0f;
        for (int i = 0; i < parts; ++i) s += partial[(long long)i * N + j];
        bias_grad[j] = s;
    }
}

template <class T>
__global__ void __launch_bounds__(256) dequantize_kernel(const DequantParams p, int vec)
{
    const long long per_row = (p.N + 7) / 8, total = per_row * p.M, atoms = atoms_of(blocks_of(p.N));
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long r = i / per_row, o = i - r * per_row;  // eight elements, o-th of row r
        float x[8];
        decode8(*reinterpret_cast<const uint32_t *>(p.codes + r * p.ld + 4 * o), x);
        const float s = scale_value(p.scales[scale_offset(r, o / 4, atoms)]);
        T v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = from_float<T>(x[k] * s);
        T *const dst = static_cast<T *>(p.x) + r * p.ldx + 8 * o;
        if (vec && 8 * o + 8 <= p.N) {
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) / 2; ++k)
                reinterpret_cast<uint4 *>(dst)[k] = reinterpret_cast<const uint4 *>(v)[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (8 * o + k < p.N) dst[k] = v[k];
        }
    }
}

bool aligned16(const void *ptr, long long ld_bytes)
{
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld_bytes % 16 == 0;
}

template <class T, bool GATED>
fgemm_status run_quantize(const QuantParams &p, cudaStream_t stream)
{
    static std::atomic<unsigned long long> ready_ctx[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    std::atomic<unsigned long long> &ready = ready_ctx[dev & 63];
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ready.load(std::memory_order_acquire) != ctx) {
        if (cudaFuncSetAttribute(quantize_kernel<T, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SMEM_BYTES) != cudaSuccess) {
            (void)cudaGetLastError();
            return FGEMM_ERR_LAUNCH;
        }
        ready.store(current_context_id(), std::memory_order_release);
    }
    const long long tiles_m = (p.M + TILE - 1) / TILE, tiles = tiles_m * ((p.N + TILE - 1) / TILE);
    const int vec = aligned16(p.x, p.ldx * (long long)sizeof(T)) &&
                    (!GATED || aligned16(p.gate, p.ldgate * (long long)sizeof(T)));
    quantize_kernel<T, GATED><<<(unsigned)std::min<long long>(tiles, 3ll * sms), THREADS, SMEM_BYTES, stream>>>(p, vec);
    if (cudaGetLastError() != cudaSuccess) return FGEMM_ERR_LAUNCH;
    if (p.bias_grad && tiles_m > 1) {
        bias_grad_kernel<<<(unsigned)std::min<long long>((p.N + 255) / 256, 8ll * sms), 256, 0, stream>>>(
            p.partial, (int)tiles_m, p.N, p.bias_grad);
        if (cudaGetLastError() != cudaSuccess) return FGEMM_ERR_LAUNCH;
    }
    return FGEMM_OK;
}

template <class T>
fgemm_status run_dequantize(const DequantParams &p, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    const long long items = ((p.N + 7) / 8) * (long long)p.M;
    dequantize_kernel<T><<<(unsigned)std::min<long long>((items + 255) / 256, 16ll * sms), 256, 0, stream>>>(
        p, aligned16(p.x, p.ldx * (long long)sizeof(T)));
    return cudaGetLastError() == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
}

}  // namespace

fgemm_status launch_quantize(fgemm_dtype type, const QuantParams &p, cudaStream_t stream)
{
    switch (type) {
    case FGEMM_F32: return p.gate ? run_quantize<float, true>(p, stream) : run_quantize<float, false>(p, stream);
    case FGEMM_BF16:
        return p.gate ? run_quantize<__nv_bfloat16, true>(p, stream) : run_quantize<__nv_bfloat16, false>(p, stream);
    default: return p.gate ? run_quantize<__half, true>(p, stream) : run_quantize<__half, false>(p, stream);
    }
}

fgemm_status launch_dequantize(fgemm_dtype type, const DequantParams &p, cudaStream_t stream)
{
    switch (type) {
    case FGEMM_F32: return run_dequantize<float>(p, stream);
    case FGEMM_BF16: return run_dequantize<__nv_bfloat16>(p, stream);
    default: return run_dequantize<__half>(p, stream);
    }
}

}  // namespace mx
}  // namespace fgemm
