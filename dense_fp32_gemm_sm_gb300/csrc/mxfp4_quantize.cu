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
#include "mxfp4_launch.h"

namespace fgemm {
namespace mx {
namespace {

constexpr int TILE = 128;  // a tile is 128 x 128: one scale atom in each direction

// The kernel's shape by element size.  A thread takes one block of a row and one of a column
// (FP32), or two blocks of rows and the same block of two neighbouring columns (16 bits).
template <int ES, bool GATED>
struct QuantShape {
    static constexpr int THREADS = ES == 4 ? 512 : 256;
    static constexpr int CTAS_PER_SM = ES == 4 ? 1 : 3;
    // 192 KB an SM; gated FP32 128, as the gates' loads want room in L1 (8192 x 4096: 58 -> 56 us).
    static constexpr int STAGES = ES == 4 && !GATED ? 3 : 2;
    // FP32: the gates of a tile come while the one before is worked on, in 32 registers; 16 bits:
    // while its own copies arrive, and three CTAs an SM fit (8192 x 11008 BF16: 91 -> 88 us,
    // 2048 x 11008 31 -> 27; FP32 8192 x 4096 would go from 58 to 65).
    static constexpr bool GATES_AHEAD = ES == 4;
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

// The largest magnitude; a NaN stays.
__device__ __forceinline__ float max_magnitude(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
// Four bytes of a row: an FP32 element, or two of 16 bits.
template <class T> struct WordOf { using type = typename PairOf<T>::type; };
template <> struct WordOf<float> { using type = float; };
template <class W> __device__ __forceinline__ W zero_word() { return pair_of_zeros<W>(); }

__device__ __forceinline__ float2 unpack(__nv_bfloat162 x) { return __bfloat1622float2(x); }
__device__ __forceinline__ float2 unpack(__half2 x) { return __half22float2(x); }

// Two values times f.x and f.y, both powers of two: exact, in bf16 itself (it has f's range).
__device__ __forceinline__ float2 scaled(__nv_bfloat162 x, __nv_bfloat162 f) { return __bfloat1622float2(__hmul2(x, f)); }
__device__ __forceinline__ float2 scaled(__half2 x, float2 f)
{
    const float2 v = __half22float2(x);
    return make_float2(v.x * f.x, v.y * f.y);
}
template <class P> struct FactorOf;
template <> struct FactorOf<__nv_bfloat162> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ type make(float x, float y) { return __floats2bfloat162_rn(x, y); }
};
template <> struct FactorOf<__half2> {
    using type = float2;
    static __device__ __forceinline__ type make(float x, float y) { return make_float2(x, y); }
};

// x where y > 0, else 0, for a pair.
__device__ __forceinline__ uint32_t gated(__nv_bfloat162 y, uint32_t x) { return __hgt2_mask(y, pair_of_zeros<__nv_bfloat162>()) & x; }
__device__ __forceinline__ uint32_t gated(__half2 y, uint32_t x) { return __hgt2_mask(y, pair_of_zeros<__half2>()) & x; }

// Words w[i ^ x] to their places.
__device__ __forceinline__ uint4 exchange(const uint32_t (&w)[4], int x)
{
    const bool one = x & 1, two = x & 2;
    const uint32_t a = one ? w[1] : w[0], b = one ? w[0] : w[1], c = one ? w[3] : w[2], d = one ? w[2] : w[3];
    return two ? make_uint4(c, d, a, b) : make_uint4(a, b, c, d);
}

// Eight values times f to eight codes.
__device__ __forceinline__ uint32_t encode_scaled(const float (&x)[8], float f)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i] * f;
    return encode8(v);
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
            top = max_magnitude(top, x[j][0], x[j][1]);
            top = max_magnitude(top, x[j][2], x[j][3]);
        }
        const uint32_t s = scale_byte(__float_as_uint(top));
        const float f = inverse_scale(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v[8] = {x[2 * j][0],     x[2 * j][1],     x[2 * j][2],     x[2 * j][3],
                                x[2 * j + 1][0], x[2 * j + 1][1], x[2 * j + 1][2], x[2 * j + 1][3]};
            w[j] = __byte_perm(encode_scaled(v, f), 0, rot & 1 ? 0x1032 : 0x3210);
        }
        codes = s == 255u ? make_uint4(0, 0, 0, 0) : exchange(w, rot >> 1);
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
        const uint32_t s = scale_byte(__float_as_uint(max_magnitude(t2.x, t2.y, 0.0f)));
        const auto f = FactorOf<P>::make(inverse_scale(s), inverse_scale(s));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = scaled(x[j][i], f);
                v[2 * i] = u.x;
                v[2 * i + 1] = u.y;
            }
            w[j] = encode8(v);
        }
        codes = s == 255u ? make_uint4(0, 0, 0, 0) : exchange(w, rot);
        return s;
    }
}

// Bound by memory: the matrix once in, 17/32 bytes an element and direction out.  Persistent
// CTAs; while a tile is worked on, the next is copied, and in FP32 without a gate the one after
// it too (STAGES - 1 tiles ahead).
// ELEMENTS: mode is COPY_ELEMENTS (an instance of its own, for the registers that its loads take).
template <class T, bool GATED, bool ELEMENTS>
__global__ void __launch_bounds__(QuantShape<sizeof(T), GATED>::THREADS, ELEMENTS ? 2 : QuantShape<sizeof(T), GATED>::CTAS_PER_SM)
    quantize_kernel(const QuantParams p, int mode)
{
    using L = QuantShape<sizeof(T), GATED>;
    constexpr int ES = (int)sizeof(T), V = 16 / ES;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const long long tiles_n = (p.N + TILE - 1) / TILE, tiles_m = (p.M + TILE - 1) / TILE, tiles = tiles_n * tiles_m;
    const long long row_blocks = blocks_of(p.N), col_blocks = blocks_of(p.M);
    const T *const X = static_cast<const T *>(p.x);
    const T *const Y = static_cast<const T *>(p.gate);
    after_previous_kernel();

    // Start the copies of tile w into a stage (asynchronous modes); beyond the matrix: zeros.
    // (A thread's pieces lie in one column of pieces, a whole number of rows apart.)
    auto start = [&](long long w, int stage) {
        if (w < tiles) {
            const long long tm = w / tiles_n, r0 = tm * TILE, c0 = (w - tm * tiles_n) * TILE;
            const int rows = (int)min((long long)TILE, p.M - r0), cols = (int)min((long long)TILE, p.N - c0);
            const uint32_t dst = (uint32_t)__cvta_generic_to_shared(smem) + stage * L::TILE_BYTES;
            if (mode == COPY_16) {
                constexpr int STEP = L::THREADS / L::CHUNKS_PER_ROW;
                static_assert(STEP % 8 == 0, "the swizzle repeats");
                const int row = t / L::CHUNKS_PER_ROW, c = t % L::CHUNKS_PER_ROW;
                const int inside = max(0, min(cols - c * V, V)) * ES;
                const uint32_t at = dst + piece_at(row, c);
                const T *src = X + (r0 + row) * p.ldx + c0 + c * V;
                if (rows == TILE && inside == 16) {
#pragma unroll
                    for (int j = 0; j < L::CHUNKS; ++j, src += STEP * p.ldx) copy_async_16(at + j * STEP * 128, src, 16);
                } else {
#pragma unroll
                    for (int j = 0; j < L::CHUNKS; ++j, src += STEP * p.ldx) {
                        const int bytes = row + j * STEP < rows ? inside : 0;
                        copy_async_16(at + j * STEP * 128, bytes ? src : X, bytes);
                    }
                }
            } else {
                constexpr int WORDS = TILE * ES / 4, STEP = L::THREADS / WORDS;  // words a row
                const int row = t / WORDS, col = t % WORDS * (4 / ES);
                const int inside = max(0, min(cols - col, 4 / ES)) * ES;
                const T *src = X + (r0 + row) * p.ldx + c0 + col;
#pragma unroll 8
                for (int j = 0; j < TILE / STEP; ++j, src += STEP * p.ldx) {
                    const int bytes = row + j * STEP < rows ? inside : 0;
                    copy_async_4(dst + element_at<ES>(row + j * STEP, col), bytes ? src : X, bytes);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // This thread's elements one by one: a column's, OWN_STEP rows apart.
    constexpr int OWN = TILE * TILE / L::THREADS, OWN_STEP = L::THREADS / TILE;
    [[maybe_unused]] const int own_row = t / TILE, own_col = t % TILE;
    // The gate of this thread's own 16-byte pieces of tile w ...
    uint4 gate[GATED && !ELEMENTS ? L::CHUNKS : 1];
    auto fetch_gate = [&](long long w) {
        if (!GATED || ELEMENTS || w >= tiles) return;
        if (mode == COPY_4) {
            // ... or of its own elements, in words of one or two.
            const long long tm = w / tiles_n, r0 = tm * TILE, c0 = (w - tm * tiles_n) * TILE;
            const int rows = c0 + own_col < p.N ? (int)min((long long)TILE, p.M - r0) : 0;
            const T *src = Y + (r0 + own_row) * p.ldgate + c0 + own_col;
            T *const to = reinterpret_cast<T *>(gate);
#pragma unroll
            for (int j = 0; j < OWN; ++j, src += OWN_STEP * p.ldgate)
                to[j] = own_row + j * OWN_STEP < rows ? __ldcs(src) : from_float<T>(0.0f);
            return;
        }
        const long long tm = w / tiles_n, r0 = tm * TILE, c0 = (w - tm * tiles_n) * TILE;
        if (r0 + TILE <= p.M && c0 + TILE <= p.N) {
            const T *src = Y + (r0 + t / L::CHUNKS_PER_ROW) * p.ldgate + c0 + t % L::CHUNKS_PER_ROW * V;
#pragma unroll
            for (int j = 0; j < L::CHUNKS; ++j, src += L::THREADS / L::CHUNKS_PER_ROW * p.ldgate)
                gate[j] = __ldcs(reinterpret_cast<const uint4 *>(src));
            return;
        }
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

    // Elements through registers: a tile's are loaded while the one before is worked on.
    T ahead[ELEMENTS && !GATED ? OWN : 1];
    [[maybe_unused]] auto load_ahead = [&](long long w) {
        if (w >= tiles) return;
        const long long tm = w / tiles_n, r0 = tm * TILE, c0 = (w - tm * tiles_n) * TILE;
        const int rows = c0 + own_col < p.N ? (int)min((long long)TILE, p.M - r0) : 0;
        const T *src = X + (r0 + own_row) * p.ldx + c0 + own_col;
#pragma unroll
        for (int j = 0; j < OWN; ++j, src += OWN_STEP * p.ldx)
            ahead[j] = own_row + j * OWN_STEP < rows ? *src : from_float<T>(0.0f);
    };
    if constexpr (ELEMENTS && !GATED) load_ahead(blockIdx.x);
    if constexpr (!ELEMENTS) {
        for (int s = 0; s + 1 < L::STAGES; ++s) start(blockIdx.x + (long long)s * gridDim.x, s);
        if constexpr (L::GATES_AHEAD) fetch_gate(blockIdx.x);
    }
    int stage = 0;
    for (long long w = blockIdx.x; w < tiles; w += gridDim.x) {
        const long long tm = w / tiles_n, tn = w - tm * tiles_n;
        const long long r0 = tm * TILE, c0 = tn * TILE;
        uint8_t *const tile = smem + stage * L::TILE_BYTES;
        [[maybe_unused]] const int own_rows = c0 + own_col < p.N ? (int)min((long long)TILE, p.M - r0) : 0;
        if constexpr (!L::GATES_AHEAD) fetch_gate(w);
        if constexpr (ELEMENTS && !GATED) {
            // Two stages: what the previous round loaded is written behind the reads of the tile before.
#pragma unroll
            for (int j = 0; j < OWN; ++j) *reinterpret_cast<T *>(tile + element_at<ES>(own_row + j * OWN_STEP, own_col)) = ahead[j];
        } else if constexpr (ELEMENTS) {
            __syncthreads();  // the previous tile has been read (one stage)
            constexpr int BATCH = 16;  // loads in flight
            const T *src = X + (r0 + own_row) * p.ldx + c0 + own_col;
            const T *gsrc = GATED ? Y + (r0 + own_row) * p.ldgate + c0 + own_col : nullptr;
            for (int j = 0; j < OWN; j += BATCH) {
                T e[BATCH], y[GATED ? BATCH : 1];
#pragma unroll
                for (int i = 0; i < BATCH; ++i, src += OWN_STEP * p.ldx, gsrc += GATED ? OWN_STEP * p.ldgate : 0) {
                    const bool in = own_row + (j + i) * OWN_STEP < own_rows;
                    e[i] = in ? *src : from_float<T>(0.0f);
                    if constexpr (GATED) y[i] = in ? *gsrc : from_float<T>(0.0f);
                }
                if constexpr (GATED) {
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (!(to_float(y[i]) > 0.0f)) e[i] = from_float<T>(0.0f);
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    *reinterpret_cast<T *>(tile + element_at<ES>(own_row + (j + i) * OWN_STEP, own_col)) = e[i];
            }
        } else {
            // This tile's copies are this thread's oldest group; at most stages - 2 follow it.
            if (L::STAGES == 3)
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        if constexpr (GATED && !ELEMENTS) {
            if (mode == COPY_16) {
                // Each thread closes the gates of the pieces it has copied itself.
#pragma unroll
                for (int j = 0; j < L::CHUNKS; ++j) {
                    const int q = t + j * L::THREADS, row = q / L::CHUNKS_PER_ROW, c = q % L::CHUNKS_PER_ROW;
                    uint4 *const at = reinterpret_cast<uint4 *>(tile + piece_at(row, c));
                    uint32_t x[4];
                    const uint32_t y[4] = {gate[j].x, gate[j].y, gate[j].z, gate[j].w};
                    *reinterpret_cast<uint4 *>(x) = *at;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (ES == 4)
                            x[i] = __uint_as_float(y[i]) > 0.0f ? x[i] : 0u;
                        else
                            x[i] = gated(reinterpret_cast<const typename PairOf<T>::type &>(y[i]), x[i]);
                    }
                    *at = *reinterpret_cast<const uint4 *>(x);
                }
            } else {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < OWN; ++j)
                    if (!(to_float(reinterpret_cast<const T *>(gate)[j]) > 0.0f))
                        *reinterpret_cast<T *>(tile + element_at<ES>(own_row + j * OWN_STEP, own_col)) = from_float<T>(0.0f);
            }
        }
        __syncthreads();
        if constexpr (ELEMENTS && !GATED) load_ahead(w + gridDim.x);
        if constexpr (!ELEMENTS) {
            // Into the stage that the previous tile has left (the barrier above: all have read it).
            start(w + (L::STAGES - 1ll) * gridDim.x, stage == 0 ? L::STAGES - 1 : stage - 1);
            if constexpr (L::GATES_AHEAD) fetch_gate(w + gridDim.x);
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
            using Word = typename WordOf<T>::type;
            Word x[32];  // rows 32 blk + (i ^ 2 blk): byte p of a word of codes is then byte p ^ blk of its place
            float top[COLS] = {}, sum[COLS];
            Word top2 = zero_word<Word>();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int row = 32 * blk + (i ^ (2 * blk));
                x[i] = *reinterpret_cast<const Word *>(src + row * 128 + (((piece ^ row) & 7) << 4) + within);
                if constexpr (ES == 4) {
                    if (i & 1) top[0] = max_magnitude(top[0], x[i - 1], x[i]);
                } else {
                    top2 = max_magnitude(top2, x[i]);
                }
            }
            if constexpr (ES == 2) {
                const float2 f = unpack(top2);
                top[0] = f.x;
                top[COLS - 1] = f.y;
            }
            if (p.bias_grad) {
                float part[4][COLS] = {};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if constexpr (ES == 4) {
                        part[i & 3][0] += x[i];
                    } else {
                        const float2 f = unpack(x[i]);
                        part[i & 3][0] += f.x;
                        part[i & 3][COLS - 1] += f.y;
                    }
                }
#pragma unroll
                for (int e = 0; e < COLS; ++e) {
                    sum[e] = (part[0][e] + part[1][e]) + (part[2][e] + part[3][e]);
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 8);
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 16);
                    if (blk == 0 && c0 + col + e < p.N)
                        (tiles_m == 1 ? p.bias_grad : p.partial + tm * p.N)[c0 + col + e] = sum[e];
                }
            }
            if (p.col_codes) {
                const uint32_t sel = blk == 0 ? 0x3210u : blk == 1 ? 0x2301u : blk == 2 ? 0x1032u : 0x0123u;
                uint32_t s[COLS], codes[COLS][4];
#pragma unroll
                for (int e = 0; e < COLS; ++e) s[e] = scale_byte(__float_as_uint(top[e]) & 0x7FFFFFFFu);
                if constexpr (ES == 4) {
                    const float f = inverse_scale(s[0]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        codes[0][j] = encode_scaled(reinterpret_cast<const float (&)[8]>(x[8 * j]), f);
                } else {
                    const auto f = FactorOf<Word>::make(inverse_scale(s[0]), inverse_scale(s[COLS - 1]));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[2][8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 u = scaled(x[8 * j + i], f);
                            v[0][i] = u.x;
                            v[1][i] = u.y;
                        }
                        codes[0][j] = encode8(v[0]);
                        codes[COLS - 1][j] = encode8(v[1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < COLS; ++e) {
                    const int c = col + e;
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = s[e] == 255u ? 0u : __byte_perm(codes[e][j], 0, sel);
                    if (c0 + c < p.N && r0 / 32 + blk < col_blocks)
                        *reinterpret_cast<uint4 *>(p.col_codes + (c0 + c) * p.ld_col + (r0 / 32 + blk) * 16) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    p.col_scales[(tn * atoms_of(col_blocks) + tm) * ATOM_BYTES + (c % 32) * 16 + (c / 32) * 4 + blk] = (uint8_t)s[e];
                }
            }
        }
        if constexpr (!ELEMENTS) stage = stage + 1 == L::STAGES ? 0 : stage + 1;
        if constexpr (ELEMENTS && !GATED) stage ^= 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// bias_grad[j] = the sum of column j's partial sums, always in the same order: eight warps take
// every eighth part of 32 columns.
__global__ void __launch_bounds__(256) bias_grad_kernel(const float *partial, int parts, int N, float *bias_grad)
{
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    after_previous_kernel();
    for (long long j0 = blockIdx.x * 32ll; j0 < N; j0 += gridDim.x * 32ll) {
        const long long j = j0 + lane;
        float s = 0.0f;
        if (j < N) {
#pragma unroll 8
            for (int i = warp; i < parts; i += 8) s += partial[(long long)i * N + j];
        }
        sums[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && j < N) {
#pragma unroll
            for (int i = 1; i < 8; ++i) s += sums[i][lane];
            bias_grad[j] = s;
        }
        __syncthreads();
    }
}

// Elements of row r before X comes to a multiple of 16 bytes.
template <class T>
__device__ __forceinline__ int head_of(const DequantParams &p, long long r)
{
    return (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(static_cast<const T *>(p.x) + r * p.ldx) & 15u)) & 15u) /
           (int)sizeof(T);
}

// Values from codes, 16 bytes of them a lane: a warp writes 512 consecutive bytes of a row.
// Bound by the writes, which go past L2's other contents (__stcs: 8192 x 11008 FP32 69 -> 65 us,
// 0.93 of the measured copy rate; BF16 44 -> 39, 0.86).  VEC: all rows of X start on
// 16 bytes.
template <class T, bool VEC, int ROWS>
__global__ void __launch_bounds__(256) dequantize_kernel(const DequantParams p)
{
    constexpr int V = 16 / (int)sizeof(T), SPAN = 32 * V;  // elements a lane, a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    after_previous_kernel();
    const long long atoms = atoms_of(blocks_of(p.N)), k0 = (long long)blockIdx.x * SPAN;
    // A CTA: 8 * ROWS rows of a span; a warp: rows warp, warp + 8, ...
    for (long long r0 = (long long)blockIdx.y * (8 * ROWS) + warp; r0 < p.M; r0 += (long long)gridDim.y * (8 * ROWS)) {
        if constexpr (VEC) {
            const long long k = k0 + lane * V;
            const uint8_t *const scales = p.scales + k0 / 128 * ATOM_BYTES + (V == 8 ? lane / 16 * ATOM_BYTES + lane / 4 % 4 : lane / 8);
            uint32_t codes[ROWS], s[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + 8 * i;
                if (r < p.M && k < p.N) {
                    const uint8_t *const src = p.codes + r * p.ld + k / 2;
                    codes[i] = V == 8 ? *reinterpret_cast<const uint32_t *>(src) : *reinterpret_cast<const uint16_t *>(src);
                    s[i] = scales[scale_offset(r, 0, atoms)];
                }
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
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
                    __stcs(reinterpret_cast<uint4 *>(dst), *reinterpret_cast<const uint4 *>(v));
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (k + e < p.N) dst[e] = v[e];
                }
            }
        } else if constexpr (V == 4) {
            // FP32 rows that start anywhere: a lane's elements are 32 apart, so that each store of a
            // warp falls on consecutive addresses.  (Shifted 16-byte stores as below measured
            // 39 us at 4096 x 4096, this 24: the shifts cost more than four times the stores.)
            const uint8_t *const scales = p.scales + k0 / 128 * ATOM_BYTES;
            uint32_t c[ROWS][V], s[ROWS][V];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + 8 * i;
                if (r >= p.M) break;
                const uint8_t *const src = p.codes + r * p.ld + (k0 + lane) / 2, *const sr = scales + scale_offset(r, 0, atoms);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (k0 + 32 * e + lane < p.N) {
                        c[i][e] = src[16 * e];
                        s[i][e] = sr[e];
                    }
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + 8 * i;
                if (r >= p.M) break;
                T *const dst = static_cast<T *>(p.x) + r * p.ldx + k0 + lane;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (k0 + 32 * e + lane < p.N) {
                        const float2 x = decode2(c[i][e]);  // (the element is odd where the lane is)
                        dst[32 * e] = from_float<T>((lane & 1 ? x.y : x.x) * scale_value(s[i][e]));
                    }
            }
        } else {
            // 16-bit rows that start anywhere: a lane's 16 bytes start `head` elements further, where a
            // row of X has come to a multiple of 16 bytes, at any nibble and in up to two blocks.
            const int left = (int)min((long long)SPAN + 8, p.N - k0);  // elements of a row from k0 on
            const int words = (left + 31) / 32 * 4;                     // and words of their codes
            uint32_t lo[ROWS], hi[ROWS], s0[ROWS], s1[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + 8 * i;
                if (r >= p.M) break;
                const int k = head_of<T>(p, r) + lane * V, b0 = k / 32, b1 = (k + V - 1) / 32;
                lo[i] = hi[i] = s0[i] = s1[i] = 0;
                if (k < left) {
                    const uint32_t *const src = reinterpret_cast<const uint32_t *>(p.codes + r * p.ld + k0 / 2) + k / 8;
                    const uint8_t *const sr = p.scales + k0 / 128 * ATOM_BYTES + scale_offset(r, 0, atoms);
                    lo[i] = src[0];
                    s0[i] = sr[b0 / 4 * ATOM_BYTES + b0 % 4];
                    if (k / 8 + 1 < words) hi[i] = src[1];
                    if (32 * b1 < left) s1[i] = sr[b1 / 4 * ATOM_BYTES + b1 % 4];
                }
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + 8 * i;
                if (r >= p.M) break;
                const int head = head_of<T>(p, r), k = head + lane * V;
                T *const row = static_cast<T *>(p.x) + r * p.ldx + k0;
                if (k < left) {
                    float x[8];
                    decode8(__funnelshift_r(lo[i], hi[i], 4 * (k & 7)), x);
                    const int first = 32 - (k & 31);  // elements before the second block
                    const float f0 = scale_value(s0[i]), f1 = scale_value(s1[i]);
                    T v[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] = from_float<T>(x[e] * (e < first ? f0 : f1));
                    if (k + V <= left) {
                        __stcs(reinterpret_cast<uint4 *>(row + k), *reinterpret_cast<const uint4 *>(v));
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (k + e < left) row[k + e] = v[e];
                    }
                }
                if (k0 == 0 && lane < head && lane < p.N) {  // the elements before that
                    const float2 x = decode2((p.codes + r * p.ld)[lane / 2]);
                    row[lane] = from_float<T>((lane & 1 ? x.y : x.x) * scale_value(p.scales[scale_offset(r, 0, atoms)]));
                }
            }
        }
    }
}

bool aligned_to(const void *ptr, long long ld_bytes, int to)
{
    return reinterpret_cast<uintptr_t>(ptr) % to == 0 && ld_bytes % to == 0;
}

template <class T, bool GATED, bool ELEMENTS>
fgemm_status start_quantize(const QuantParams &p, int mode, long long tiles, int sms, cudaStream_t stream)
{
    using L = QuantShape<sizeof(T), GATED>;
    static std::atomic<unsigned long long> ready_ctx[64];
    constexpr int smem = !ELEMENTS ? L::SMEM_BYTES : GATED ? L::TILE_BYTES : 2 * L::TILE_BYTES;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    std::atomic<unsigned long long> &ready = ready_ctx[dev & 63];
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ready.load(std::memory_order_acquire) != ctx) {
        if (cudaFuncSetAttribute(quantize_kernel<T, GATED, ELEMENTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return FGEMM_ERR_LAUNCH;
        }
        ready.store(current_context_id(), std::memory_order_release);
    }
    const long long ctas = std::min<long long>(tiles, (ELEMENTS ? 2ll : (long long)L::CTAS_PER_SM) * sms);
    // (Stages that no tile of a CTA reaches are left out: the next kernel finds room beside this one.)
    const size_t used = (size_t)std::min<long long>(smem, (tiles + ctas - 1) / ctas * L::TILE_BYTES);
    return launch(quantize_kernel<T, GATED, ELEMENTS>, dim3((unsigned)ctas), L::THREADS, used, stream, 1, p, mode) == cudaSuccess
               ? FGEMM_OK
               : FGEMM_ERR_LAUNCH;
}

template <class T, bool GATED>
fgemm_status run_quantize(const QuantParams &p, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    const long long es = sizeof(T), tiles_m = (p.M + TILE - 1) / TILE, tiles = tiles_m * ((p.N + TILE - 1) / TILE);
    const int mode = aligned_to(p.x, p.ldx * es, 16) && (!GATED || aligned_to(p.gate, p.ldgate * es, 16)) ? COPY_16
                     : aligned_to(p.x, p.ldx * es, 4)                                                    ? COPY_4
                                                                                                         : COPY_ELEMENTS;
    fgemm_status st;
    if constexpr (sizeof(T) == 2) {
        st = mode == COPY_ELEMENTS ? start_quantize<T, GATED, true>(p, mode, tiles, sms, stream)
                                   : start_quantize<T, GATED, false>(p, mode, tiles, sms, stream);
    } else {
        st = start_quantize<T, GATED, false>(p, mode, tiles, sms, stream);  // (FP32 is always 4-byte aligned)
    }
    if (st != FGEMM_OK) return st;
    if (p.bias_grad && tiles_m > 1) {
        const dim3 grid((unsigned)std::min<long long>(((long long)p.N + 31) / 32, 8ll * sms));
        if (launch(bias_grad_kernel, grid, 256, 0, stream, 1, p.partial, (int)tiles_m, p.N, p.bias_grad) != cudaSuccess)
            return FGEMM_ERR_LAUNCH;
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
    constexpr int ROWS = sizeof(T) == 2 ? 8 : 4;  // a warp: 4 KB or 2 KB of X in flight
    const long long spans = ((long long)p.N + SPAN - 1) / SPAN, groups = ((long long)p.M + 8 * ROWS - 1) / (8 * ROWS);
    const bool vec = aligned_to(p.x, p.ldx * (long long)sizeof(T), 16);
    cudaError_t e;
    // Few rows of work: one a warp, over more CTAs.
    if (spans * groups < 2ll * sms) {
        const dim3 grid((unsigned)spans, (unsigned)std::min<long long>(((long long)p.M + 7) / 8, 65535));
        e = vec ? launch(dequantize_kernel<T, true, 1>, grid, 256, 0, stream, 1, p)
                : launch(dequantize_kernel<T, false, 1>, grid, 256, 0, stream, 1, p);
    } else {
        const dim3 grid((unsigned)spans, (unsigned)std::min<long long>(vec ? groups : ((long long)p.M + 31) / 32, 65535));
        e = vec ? launch(dequantize_kernel<T, true, ROWS>, grid, 256, 0, stream, 1, p)
                : launch(dequantize_kernel<T, false, 4>, grid, 256, 0, stream, 1, p);
    }
    return e == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
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
