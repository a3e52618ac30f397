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

// The kernel's shape by element size.  A thread takes one block of a row and one of a column
// (FP32), or two blocks of rows and the same block of two neighbouring columns (16 bits).
template <int ES>
struct QuantShape {
    static constexpr int THREADS = ES == 4 ? 512 : 256;
    static constexpr int CTAS_PER_SM = ES == 4 ? 1 : 2;
    static constexpr int STAGES = 3;  // 192 KB an SM: two tiles (64 KB FP32) on their way behind one at work
    static constexpr int TILE_BYTES = TILE * TILE * ES;
    static constexpr int SMEM_BYTES = STAGES * TILE_BYTES;
    static constexpr int CHUNKS_PER_ROW = TILE * ES / 16;
    static constexpr int CHUNKS = TILE * CHUNKS_PER_ROW / THREADS;  // 16-byte pieces a thread copies
    static_assert(CHUNKS == 8, "both element sizes copy eight pieces a thread");
};

// How a tile gets to shared memory: asynchronous copies of 16 or 4 bytes, or elements through
// registers (16-bit matrices with odd leading dimensions or addresses).
enum CopyMode { COPY_16, COPY_4, COPY_ELEMENTS };

// Byte offset in the tile of the 16-byte piece c of a row: boxes of 128 bytes x 128 rows, the
// pieces of a row exchanged by its number modulo 8.  A warp's loads then fall on different
// banks both along rows (lanes: four blocks of eight rows, each starting at another piece)
// and down columns (lanes: eight neighbouring words in four row blocks, each starting at
// another row).
__device__ __forceinline__ int piece_at(int row, int c) { return (c >> 3) * (TILE * 128) + row * 128 + (((c ^ row) & 7) << 4); }
template <int ES>
__device__ __forceinline__ int element_at(int row, int col)
{
    return piece_at(row, col * ES / 16) + (col * ES) % 16;
}

__device__ __forceinline__ void copy_async_16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The larger magnitude; a NaN stays.
__device__ __forceinline__ float max_magnitude(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ __nv_bfloat162 max_magnitude(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2_nan(a, __habs2(b)); }
__device__ __forceinline__ __half2 max_magnitude(__half2 a, __half2 b) { return __hmax2_nan(a, __habs2(b)); }

template <class P> __device__ __forceinline__ P pair_of_zeros()
{
    const uint32_t z = 0;
    return reinterpret_cast<const P &>(z);
}

template <class T> struct PairOf;
template <> struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct PairOf<__half> { using type = __half2; };

__device__ __forceinline__ float2 unpack(__nv_bfloat162 x) { return __bfloat1622float2(x); }
__device__ __forceinline__ float2 unpack(__half2 x) { return __half22float2(x); }

// Words w[i ^ x] to their places.
__device__ __forceinline__ uint4 exchange(const uint32_t (&w)[4], int x)
{
    const bool one = x & 1, two = x & 2;
    const uint32_t a = one ? w[1] : w[0], b = one ? w[0] : w[1], c = one ? w[3] : w[2], d = one ? w[2] : w[3];
    return two ? make_uint4(c, d, a, b) : make_uint4(a, b, c, d);
}

// Eight values times f to eight codes; 0 in a NaN's block.
__device__ __forceinline__ uint32_t encode_scaled(const float (&x)[8], float f, uint32_t s)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i] * f;
    return s == 255u ? 0u : encode8(v);
}

// The block `blk` of tile row `row`: its codes, and its scale byte.  g: which of the lanes that
// would meet on the same banks this is (0 or 1).
template <class T>
__device__ __forceinline__ uint32_t encode_row_block(const uint8_t *tile, int row, int blk, int g, uint4 &codes)
{
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
        const int rot = blk | g << 2;  // this lane's pieces in the order j ^ rot
        float x[8][4];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            *reinterpret_cast<float4 *>(x[j]) = *reinterpret_cast<const float4 *>(tile + piece_at(row, blk * 8 + (j ^ rot)));
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max_magnitude(top, x[j][i]);
        }
        const uint32_t s = scale_byte(__float_as_uint(top));
        const float f = inverse_scale(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v[8] = {x[2 * j][0],     x[2 * j][1],     x[2 * j][2],     x[2 * j][3],
                                x[2 * j + 1][0], x[2 * j + 1][1], x[2 * j + 1][2], x[2 * j + 1][3]};
            w[j] = __byte_perm(encode_scaled(v, f, s), 0, rot & 1 ? 0x1032 : 0x3210);
        }
        codes = exchange(w, rot >> 1);
        return s;
    } else {
        using P = typename PairOf<T>::type;
        const int rot = blk >> 1 | g << 1;
        P x[4][4];
        P top2 = pair_of_zeros<P>();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<uint4 *>(x[j]) = *reinterpret_cast<const uint4 *>(tile + piece_at(row, blk * 4 + (j ^ rot)));
#pragma unroll
            for (int i = 0; i < 4; ++i) top2 = max_magnitude(top2, x[j][i]);
        }
        const float2 t2 = unpack(top2);
        const uint32_t s = scale_byte(__float_as_uint(max_magnitude(t2.x, t2.y)));
        const float f = inverse_scale(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = unpack(x[j][i]);
                v[2 * i] = u.x;
                v[2 * i + 1] = u.y;
            }
            w[j] = encode_scaled(v, f, s);
        }
        codes = exchange(w, rot);
        return s;
    }
}

// Rows 32 * blk + (i ^ 2 * blk) of a column, i = 0 .. 31, as FP32: its codes, scale byte and sum.
__device__ __forceinline__ uint32_t encode_column_block(const float (&x)[32], float top, int blk, uint4 &codes)
{
    const uint32_t s = scale_byte(__float_as_uint(top));
    const float f = inverse_scale(s);
    const uint32_t sel = blk == 0 ? 0x3210u : blk == 1 ? 0x2301u : blk == 2 ? 0x1032u : 0x0123u;  // byte p of p ^ blk
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float v[8] = {x[8 * j],     x[8 * j + 1], x[8 * j + 2], x[8 * j + 3],
                            x[8 * j + 4], x[8 * j + 5], x[8 * j + 6], x[8 * j + 7]};
        w[j] = __byte_perm(encode_scaled(v, f, s), 0, sel);
    }
    codes = make_uint4(w[0], w[1], w[2], w[3]);
    return s;
}

// Bound by memory: the matrix once in, 17/32 bytes an element and direction out.  Persistent
// CTAs; while a tile is worked on, the next two are copied.
template <class T, bool GATED>
__global__ void __launch_bounds__(QuantShape<sizeof(T)>::THREADS, QuantShape<sizeof(T)>::CTAS_PER_SM)
    quantize_kernel(const QuantParams p, int mode, int stages)
{
    using L = QuantShape<sizeof(T)>;
    constexpr int ES = (int)sizeof(T), V = 16 / ES;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const long long tiles_n = (p.N + TILE - 1) / TILE, tiles_m = (p.M + TILE - 1) / TILE, tiles = tiles_n * tiles_m;
    const long long row_blocks = blocks_of(p.N), col_blocks = blocks_of(p.M);
    const T *const X = static_cast<const T *>(p.x);
    const T *const Y = static_cast<const T *>(p.gate);
    if (p.early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Start the copies of tile w into a stage (asynchronous modes); beyond the matrix: zeros.
    auto start = [&](long long w, int stage) {
        if (w < tiles && mode != COPY_ELEMENTS) {
            const long long tm = w / tiles_n, r0 = tm * TILE, c0 = (w - tm * tiles_n) * TILE;
            const uint32_t dst = (uint32_t)__cvta_generic_to_shared(smem) + stage * L::TILE_BYTES;
            if (mode == COPY_16) {
#pragma unroll
                for (int j = 0; j < L::CHUNKS; ++j) {
                    const int q = t + j * L::THREADS, row = q / L::CHUNKS_PER_ROW, c = q % L::CHUNKS_PER_ROW;
                    const long long left = p.N - c0 - c * V;
                    const int bytes = r0 + row < p.M && left > 0 ? (int)min(left, (long long)V) * ES : 0;
                    copy_async_16(dst + piece_at(row, c), bytes ? X + (r0 + row) * p.ldx + c0 + c * V : X, bytes);
                }
            } else {
#pragma unroll 8
                for (int j = 0; j < 4 * L::CHUNKS; ++j) {
                    const int q = t + j * L::THREADS, row = q / (4 * L::CHUNKS_PER_ROW), col = q % (4 * L::CHUNKS_PER_ROW) * (4 / ES);
                    const long long left = p.N - c0 - col;
                    const int bytes = r0 + row < p.M && left > 0 ? (int)min(left, 4ll / ES) * ES : 0;
                    copy_async_4(dst + element_at<ES>(row, col), bytes ? X + (r0 + row) * p.ldx + c0 + col : X, bytes);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // The gate of this thread's own 16-byte pieces of tile w.
    uint4 gate[GATED ? L::CHUNKS : 1];
    auto fetch_gate = [&](long long w) {
        if (!GATED || w >= tiles || mode != COPY_16) return;
        const long long tm = w / tiles_n, r0 = tm * TILE, c0 = (w - tm * tiles_n) * TILE;
#pragma unroll
        for (int j = 0; j < L::CHUNKS; ++j) {
            const int q = t + j * L::THREADS, row = q / L::CHUNKS_PER_ROW, c = q % L::CHUNKS_PER_ROW;
            if (r0 + row < p.M && c0 + (c + 1) * V <= p.N) {
                gate[j] = __ldcs(reinterpret_cast<const uint4 *>(Y + (r0 + row) * p.ldgate + c0 + c * V));
            } else {
                T e[V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    e[i] = r0 + row < p.M && c0 + c * V + i < p.N ? Y[(r0 + row) * p.ldgate + c0 + c * V + i] : from_float<T>(0.0f);
                gate[j] = *reinterpret_cast<const uint4 *>(e);
            }
        }
    };

    for (int s = 0; s + 1 < stages; ++s) start(blockIdx.x + (long long)s * gridDim.x, s);
    fetch_gate(blockIdx.x);
    int stage = 0;
    for (long long w = blockIdx.x; w < tiles; w += gridDim.x) {
        const long long tm = w / tiles_n, tn = w - tm * tiles_n;
        const long long r0 = tm * TILE, c0 = tn * TILE;
        uint8_t *const tile = smem + stage * L::TILE_BYTES;
        if (mode == COPY_ELEMENTS) {
            __syncthreads();  // the previous tile has been read (one stage)
            constexpr int BATCH = 16;
            for (int j = 0; j < TILE * TILE / L::THREADS; j += BATCH) {
                T e[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int q = t + (j + i) * L::THREADS, row = q / TILE, col = q % TILE;
                    const bool in = r0 + row < p.M && c0 + col < p.N;
                    e[i] = in ? X[(r0 + row) * p.ldx + c0 + col] : from_float<T>(0.0f);
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int q = t + (j + i) * L::THREADS;
                    *reinterpret_cast<T *>(tile + element_at<ES>(q / TILE, q % TILE)) = e[i];
                }
            }
        } else {
            // This tile's copies are this thread's oldest group; at most stages - 2 follow it.
            if (stages == 3)
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        if constexpr (GATED) {
            // Each thread closes the gates of the pieces it has copied itself.
            if (mode == COPY_16) {
#pragma unroll
                for (int j = 0; j < L::CHUNKS; ++j) {
                    const int q = t + j * L::THREADS, row = q / L::CHUNKS_PER_ROW, c = q % L::CHUNKS_PER_ROW;
                    uint4 *const at = reinterpret_cast<uint4 *>(tile + piece_at(row, c));
                    T x[V], y[V];
                    *reinterpret_cast<uint4 *>(x) = *at;
                    *reinterpret_cast<uint4 *>(y) = gate[j];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (!(to_float(y[i]) > 0.0f)) x[i] = from_float<T>(0.0f);
                    *at = *reinterpret_cast<const uint4 *>(x);
                }
            } else {
                constexpr int BATCH = 16;
                __syncthreads();
                for (int j = 0; j < TILE * TILE / L::THREADS; j += BATCH) {
                    bool open[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int q = t + (j + i) * L::THREADS, row = q / TILE, col = q % TILE;
                        open[i] = r0 + row < p.M && c0 + col < p.N && to_float(Y[(r0 + row) * p.ldgate + c0 + col]) > 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int q = t + (j + i) * L::THREADS;
                        if (!open[i]) *reinterpret_cast<T *>(tile + element_at<ES>(q / TILE, q % TILE)) = from_float<T>(0.0f);
                    }
                }
            }
        }
        __syncthreads();
        if (mode != COPY_ELEMENTS) {
            // Into the stage that the previous tile has left (the barrier above: all have read it).
            if (stages == 3)
                start(w + 2ll * gridDim.x, stage == 0 ? 2 : stage - 1);
            fetch_gate(w + gridDim.x);
        }

        if (p.row_codes) {
            // Rows 2v, 2v + 1 of each quarter of the tile, four blocks: a warp's 32 scale bytes are
            // neighbours in the atom.
#pragma unroll
            for (int v = warp; v < 16; v += L::THREADS / 32) {
                const int quarter = (lane >> 2) & 3, row = 2 * v + (lane >> 4) + 32 * quarter, blk = lane & 3;
                uint4 codes;
                const uint32_t s = encode_row_block<T>(tile, row, blk, quarter & 1, codes);
                if (r0 + row < p.M && c0 / 32 + blk < row_blocks)
                    *reinterpret_cast<uint4 *>(p.row_codes + (r0 + row) * p.ld_row + (c0 / 32 + blk) * 16) = codes;
                p.row_scales[(tm * atoms_of(row_blocks) + tn) * ATOM_BYTES + 32 * v + lane] = (uint8_t)s;
            }
        }
        if (p.col_codes || p.bias_grad) {
            const int blk = lane >> 3;
            constexpr int COLS = 4 / ES;  // neighbouring columns a thread takes: a word of a row
            const int col = (8 * warp + (lane & 7)) * COLS;
            const uint8_t *const src = tile + (col * ES / 128) * (TILE * 128);
            const int piece = (col * ES / 16) & 7, within = (col * ES) % 16;
            float x[COLS][32], top[COLS], sum[COLS];
            if constexpr (ES == 4) {
                top[0] = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int row = 32 * blk + (i ^ (2 * blk));
                    x[0][i] = *reinterpret_cast<const float *>(src + row * 128 + (((piece ^ row) & 7) << 4) + within);
                    top[0] = max_magnitude(top[0], x[0][i]);
                }
            } else {
                using P = typename PairOf<T>::type;
                P top2 = pair_of_zeros<P>();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int row = 32 * blk + (i ^ (2 * blk));
                    const P u = *reinterpret_cast<const P *>(src + row * 128 + (((piece ^ row) & 7) << 4) + within);
                    top2 = max_magnitude(top2, u);
                    const float2 f = unpack(u);
                    x[0][i] = f.x;
                    x[COLS - 1][i] = f.y;
                }
                const float2 f = unpack(top2);
                top[0] = f.x;
                top[COLS - 1] = f.y;
            }
#pragma unroll
            for (int e = 0; e < COLS; ++e) {
                if (p.bias_grad) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 32; ++i) part[i & 3] += x[e][i];
                    sum[e] = (part[0] + part[1]) + (part[2] + part[3]);
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 8);
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 16);
                    if (blk == 0 && c0 + col + e < p.N)
                        (tiles_m == 1 ? p.bias_grad : p.partial + tm * p.N)[c0 + col + e] = sum[e];
                }
                if (p.col_codes) {
                    uint4 codes;
                    const uint32_t s = encode_column_block(x[e], top[e], blk, codes);
                    const int c = col + e;
                    if (c0 + c < p.N && r0 / 32 + blk < col_blocks)
                        *reinterpret_cast<uint4 *>(p.col_codes + (c0 + c) * p.ld_col + (r0 / 32 + blk) * 16) = codes;
                    p.col_scales[(tn * atoms_of(col_blocks) + tm) * ATOM_BYTES + (c % 32) * 16 + (c / 32) * 4 + blk] = (uint8_t)s;
                }
            }
        }
        if (mode != COPY_ELEMENTS) stage = stage + 1 == stages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
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

// Values from codes, 16 bytes of them a lane: a warp writes 512 consecutive bytes of a row.
// Bound by the writes.  VEC: X allows 16-byte stores; otherwise a lane's elements are 32 apart,
// so that each store of a warp still falls on consecutive addresses.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) dequantize_kernel(const DequantParams p)
{
    constexpr int V = 16 / (int)sizeof(T), SPAN = 32 * V;  // elements a lane, a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long spans = (p.N + SPAN - 1) / SPAN, groups = ((long long)p.M + 31) / 32, atoms = atoms_of(blocks_of(p.N));
    // A CTA: 32 rows of a span; a warp: rows warp, warp + 8, ...
    for (long long w = blockIdx.x; w < spans * groups; w += gridDim.x) {
        const long long g = w / spans, k0 = (w - g * spans) * SPAN;
        const long long r0 = g * 32 + warp;
        if constexpr (VEC) {
            const long long k = k0 + lane * V;
            uint32_t codes[4];
            uint32_t s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long r = r0 + 8 * i;
                if (r < p.M && k < p.N) {
                    const uint8_t *const src = p.codes + r * p.ld + k / 2;
                    codes[i] = V == 8 ? *reinterpret_cast<const uint32_t *>(src) : *reinterpret_cast<const uint16_t *>(src);
                    s[i] = p.scales[scale_offset(r, k / 32, atoms)];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long r = r0 + 8 * i;
                if (r >= p.M || k >= p.N) continue;
                float x[8];
                decode8(codes[i], x);
                const float f = scale_value(s[i]);
                T v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = from_float<T>(x[e] * f);
                T *const dst = static_cast<T *>(p.x) + r * p.ldx + k;
                if (k + V <= p.N) {
                    *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(v);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (k + e < p.N) dst[e] = v[e];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long r = r0 + 8 * i;
                if (r >= p.M) break;
                const uint8_t *const src = p.codes + r * p.ld;
                uint32_t c[V], s[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const long long k = k0 + 32 * e + lane;
                    if (k < p.N) {
                        c[e] = src[k / 2];
                        s[e] = p.scales[scale_offset(r, k / 32, atoms)];
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const long long k = k0 + 32 * e + lane;
                    if (k >= p.N) continue;
                    float x[8];
                    decode8(c[e] >> (4 * (lane & 1)), x);  // (k is odd where the lane is)
                    static_cast<T *>(p.x)[r * p.ldx + k] = from_float<T>(x[0] * scale_value(s[e]));
                }
            }
        }
    }
}

bool aligned_to(const void *ptr, long long ld_bytes, int to)
{
    return reinterpret_cast<uintptr_t>(ptr) % to == 0 && ld_bytes % to == 0;
}

template <class T, bool GATED>
fgemm_status run_quantize(const QuantParams &p, cudaStream_t stream)
{
    using L = QuantShape<sizeof(T)>;
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
                                 L::SMEM_BYTES) != cudaSuccess) {
            (void)cudaGetLastError();
            return FGEMM_ERR_LAUNCH;
        }
        ready.store(current_context_id(), std::memory_order_release);
    }
    const long long es = sizeof(T), tiles_m = (p.M + TILE - 1) / TILE, tiles = tiles_m * ((p.N + TILE - 1) / TILE);
    const int mode = aligned_to(p.x, p.ldx * es, 16) && (!GATED || aligned_to(p.gate, p.ldgate * es, 16)) ? COPY_16
                     : aligned_to(p.x, p.ldx * es, 4)                                                    ? COPY_4
                                                                                                         : COPY_ELEMENTS;
    const int stages = mode == COPY_ELEMENTS ? 1 : L::STAGES;
    quantize_kernel<T, GATED><<<(unsigned)std::min<long long>(tiles, (long long)L::CTAS_PER_SM * sms), L::THREADS,
                                stages * L::TILE_BYTES, stream>>>(p, mode, stages);
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
    constexpr int SPAN = 512 / (int)sizeof(T);
    const long long items = ((p.N + SPAN - 1) / SPAN) * (((long long)p.M + 31) / 32);
    const unsigned grid = (unsigned)std::min<long long>(items, 16ll * sms);
    if (aligned_to(p.x, p.ldx * (long long)sizeof(T), 16))
        dequantize_kernel<T, true><<<grid, 256, 0, stream>>>(p);
    else
        dequantize_kernel<T, false><<<grid, 256, 0, stream>>>(p);
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
