// mxfp4_tc.cuh -- the product of two MXFP4 matrices on the tensor cores of sm_103a
// (tcgen05.mma kind::mxf4, one E8M0 scale for every 32 codes, FP32 accumulators).
//
// C[i][j] = act(alpha * sum_b 2^(sa + sb - 254) sum_{k in b} a[i][k] b[j][k] + beta C + bias[j])
//
// The MMA's 128 rows are rows of B (columns of C) and its NT columns are rows of A: an
// accumulator lane is then a column of C, a warp's 32 lanes are neighbours in a row of C,
// and the epilogue stores whole segments of rows straight from registers, for any leading
// dimension, alignment and type, with no pass through shared memory.  Few rows of A take a
// narrow NT (16 and up) without touching the 128 rows of B that the MMA wants.
//
// A stage is 256 deep: 128 bytes of codes a row, the 128-byte swizzle's row, and two atoms of
// scales (512 bytes, 128 rows x 4 blocks), which lie in memory as tcgen05.cp wants them.  One
// warp streams stages by TMA, another copies each stage's scales to tensor memory and issues
// four MMAs of depth 64; eight warps store the accumulators of the previous tile meanwhile.
//
// What bounds it (one GB300): large products by the power limit -- 8192 x 8192 x 32768 runs at
// 7.3 PFLOP/s with the SMs held at 1.54 GHz, 96 % of four 128-cycle MMAs a stage at that
// clock; with K = 4096 by the boundaries of tiles and the writing of C; few rows by reading
// B, 3.4 us after the launch and the joining of sums (16 x 11008 x 4096: 7.1 us, 3.5 at the
// memory's rate).  Both loops below are walked by whole warps, one elected lane issuing: from
// a branch on the lane number an MMA took 128 cycles to issue, whatever its width
// (8192 x 8192 x 32768: 1198 us, against 683 with the whole warps).
//
// The kernels are on the SMs while the one before them still writes (mxfp4_launch.h), so what they
// read of global memory comes by ordinary loads and copies after the wait, never by non-coherent
// ones (__ldg).  (Tokens and bias past L1, by __ldcg: one token 7.2 us in place of 6.7.)
#pragma once

#include <cooperative_groups.h>

#include "mxfp4_device.cuh"
#include "tc_gemm.cuh"

namespace fgemm {
namespace mx {

constexpr int TC_ROWS = 128;     // rows of B a tile: tensor-memory lanes
constexpr int TC_DEPTH = 256;    // codes a stage: 128 bytes a row
constexpr int TC_BLOCKS = TC_DEPTH / BLOCK;
constexpr int TC_THREADS = 320;  // producer, MMA, eight epilogue warps
constexpr int EPI_WARPS = 8;

// How a kernel divides the work: whole tiles by persistent CTAs; a tile's stages over a
// cluster; and the latter with A unquantised (SPLIT_FUSED), quantised by the epilogue's warps
// while the first stages of B are on their way.
enum TcMode { WHOLE = 0, SPLIT = 1, SPLIT_FUSED = 2 };

template <int NT, int MODE>
struct TcTile {
    static constexpr bool FUSED = MODE == SPLIT_FUSED;
    static constexpr int W_BYTES = TC_ROWS * 128;
    static constexpr int X_BYTES = NT * 128;
    static constexpr int SF_BYTES = 2 * ATOM_BYTES;  // of either operand: NT divides a group of 128 rows
    static constexpr int STAGE_BYTES = W_BYTES + SF_BYTES + (FUSED ? 0 : X_BYTES + SF_BYTES);
    // (80 to 104 KB for the tiles of 16 to 64 rows, so that two CTAs share an SM; eight stages measured
    // no faster, and three, with three CTAs an SM, 0.1 to 0.8 us slower.)
    static constexpr int STAGES = NT == 128 ? 6 : 4;
    // Fused: A's codes and scales of each of this CTA's stages follow the ring and the barriers.
    static constexpr int FUSED_BYTES = FUSED ? X_BYTES + SF_BYTES : 0;
    // Tensor memory: two accumulators of NT columns, then two buffers of scales (4 columns an atom).
    static constexpr int SF_COLS = 16;
    static constexpr int SF_BASE = 2 * NT;
    static constexpr int TMEM_USED = SF_BASE + 2 * SF_COLS;
    static constexpr int TMEM_COLS = TMEM_USED > 256 ? 512 : TMEM_USED > 128 ? 256 : TMEM_USED > 64 ? 128 : 64;
    static_assert(TMEM_USED <= 512, "tensor memory");
    static constexpr int CHUNK = NT < 32 ? NT : 32;  // accumulator columns read at a time
    static constexpr int BAR_OFFSET = STAGES * STAGE_BYTES;
    // full[S], empty[S], acc_full[2], acc_free[2], drain, x_ready, tensor-memory slot
    static constexpr int BAR_BYTES = (2 * STAGES + 6) * 8 + 8;
    static constexpr int X_OFFSET = BAR_OFFSET + 1024;
    static constexpr int SMEM_BYTES = 1024 + (FUSED ? X_OFFSET : BAR_OFFSET + BAR_BYTES);  // + alignment
    static_assert(SMEM_BYTES <= 227 * 1024 && BAR_BYTES <= 1024, "shared memory");
    static_assert(STAGES * STAGE_BYTES >= TC_ROWS * NT * 4, "a split tile's sums take the stages' place");
};

struct TcArgs {
    CUtensorMap w, x;  // codes of B and A: (bytes along K, rows), boxes of 128 bytes
    const uint8_t *w_scales, *x_scales;
    void *c;
    const void *x_plain;  // fused: A as it is, M x K
    long long ldx;
    int K, x_vec;         // x_vec: A allows 16-byte loads
    const float *bias;
    long long ldc, atoms;  // atoms: scale atoms of a 128-row group
    int M, N, blocks;      // blocks: ceil(K / 32)
    float alpha, beta;
    int relu;
    int c_pairs;  // 16-bit C: pairs of columns are 4-byte aligned
    int tiles_x, tiles_w;
    unsigned long long wait_limit_ns;
    int withhold;
    int dependent;  // the kernel before this one in the stream writes A, and only A
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// kind::mxf4: A and B E2M1, scales E8M0, both K-major, 128 x n; the pair of scales (0 or 2)
// of each 32-bit column that the MMA takes.
__host__ __device__ constexpr uint32_t mxf4_idesc(int n, int pair)
{
    return ((uint32_t)pair << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
           ((uint32_t)(TC_ROWS >> 4) << 24) | ((uint32_t)pair << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One atom of scales from shared memory to four columns of tensor memory (32 lanes of 16
// bytes, repeated in each quarter).  The descriptor: 8 rows of 16 bytes are 128 bytes apart.
__device__ __forceinline__ void copy_atom(uint32_t tmem, uint32_t smem_addr)
{
    const uint64_t desc = (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xFFFFFFFF;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(one));
    return one != 0;
}

// tc::mbar_wait by a whole warp: the same answer in all lanes, known to be uniform.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned *err, unsigned code,
                                          unsigned long long limit_ns)
{
    if (__all_sync(0xFFFFFFFFu, tc::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xFFFFFFFFu, tc::mbar_wait(bar, parity, err, code, limit_ns));
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[N])
{
    static_assert(N == 16 || N == 32, "columns");
    if constexpr (N == 32) {
        tc::tmem_ld_32cols(taddr, r);
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    }
}

// One element of C from its sum.
template <class T, bool BETA, bool RELU>
__device__ __forceinline__ float finish(const TcArgs &p, const T *out, float sum, float bias)
{
    float o = fmaf(p.alpha, sum, bias);
    if constexpr (BETA) o = fmaf(p.beta, to_float(*out), o);
    if constexpr (RELU) o = relu(o);
    return o;
}

// N sums of this lane's column of C to `rows` rows of it, the first at `out`.  The 16-bit
// types, where pairs of columns are aligned (`pairs`): lanes 2i and 2i + 1 exchange their
// values of two rows, and each stores both columns of one row, 4 bytes a lane in place of 2.
template <class T, bool BETA, bool RELU, int N>
__device__ __forceinline__ void store_rows(const TcArgs &p, T *out, const uint32_t (&r)[N], float bias, int rows, bool in,
                                           bool pairs)
{
    if constexpr (sizeof(T) == 2 && !BETA) {
        if (pairs) {
            const int odd = threadIdx.x & 1;
            T *dst = out + (odd ? p.ldc - 1 : 0);
#pragma unroll
            for (int c = 0; c < N; c += 2, dst += 2 * p.ldc) {
                const T a = from_float<T>(finish<T, BETA, RELU>(p, out, __uint_as_float(r[c]), bias));
                const T b = from_float<T>(finish<T, BETA, RELU>(p, out, __uint_as_float(r[c + 1]), bias));
                const uint32_t own = (uint32_t)reinterpret_cast<const uint16_t &>(a) |
                                     (uint32_t)reinterpret_cast<const uint16_t &>(b) << 16;
                const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
                const uint32_t both = __byte_perm(own, other, odd ? 0x3276u : 0x5410u);
                if (in && c + odd < rows) *reinterpret_cast<uint32_t *>(dst) = both;
            }
            return;
        }
    }
    if (!in) return;
    if (rows >= N) {
#pragma unroll
        for (int c = 0; c < N; ++c, out += p.ldc)
            *out = from_float<T>(finish<T, BETA, RELU>(p, out, __uint_as_float(r[c]), bias));
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c, out += p.ldc)
            if (c < rows) *out = from_float<T>(finish<T, BETA, RELU>(p, out, __uint_as_float(r[c]), bias));
    }
}

template <class T, int N>
__device__ __forceinline__ void store_chunk(const TcArgs &p, T *out, const uint32_t (&r)[N], float bias, int rows, bool in,
                                            bool pairs)
{
    if (p.beta != 0.0f) {
        if (p.relu)
            store_rows<T, true, true>(p, out, r, bias, rows, in, pairs);
        else
            store_rows<T, true, false>(p, out, r, bias, rows, in, pairs);
    } else {
        if (p.relu)
            store_rows<T, false, true>(p, out, r, bias, rows, in, pairs);
        else
            store_rows<T, false, false>(p, out, r, bias, rows, in, pairs);
    }
}

// Quantise A's p.M (at most LINEAR_ROWS) rows, from code k0 on, into `stages` stages' tiles of
// codes (NT rows, the 128-byte swizzle) and atoms of scales, by `threads` threads (t of them).
template <int NT, class T>
__device__ __forceinline__ void quantize_tokens(const TcArgs &p, uint8_t *codes, uint8_t *scales, int stages, long long k0,
                                                int t, int threads)
{
    // Four lanes a block, eight elements each, of every row: all rows' loads are in flight
    // before the first is used.  (stages * 32 items: whole warps, for the shuffles.)
    for (int o = t; o < stages * TC_BLOCKS * 4; o += threads) {
        const long long k = k0 + o * 8;
        T e[LINEAR_ROWS][8];
#pragma unroll
        for (int row = 0; row < LINEAR_ROWS; ++row) {
            if (row >= p.M) break;
            const T *const src = static_cast<const T *>(p.x_plain) + row * p.ldx + k;
            if (p.x_vec && k + 8 <= p.K) {
#pragma unroll
                for (int j = 0; j < (int)sizeof(T) / 2; ++j)
                    reinterpret_cast<uint4 *>(e[row])[j] = reinterpret_cast<const uint4 *>(src)[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) e[row][j] = k + j < p.K ? src[j] : from_float<T>(0.0f);
            }
        }
        const int stage = o / (TC_BLOCKS * 4), b = (o >> 2) % TC_BLOCKS, part = o & 3;
#pragma unroll
        for (int row = 0; row < LINEAR_ROWS; ++row) {
            if (row >= p.M) break;
            float v[8];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = to_float(e[row][j]);
                top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const uint32_t s = scale_byte(top);
            const float f = inverse_scale(s);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= f;
            const uint32_t c = s == 255u ? 0u : encode8(v);
            *reinterpret_cast<uint32_t *>(codes + stage * NT * 128 + row * 128 + ((b ^ (row & 7)) << 4) + part * 4) = c;
            if (part == 0) scales[(stage * 2 + b / 4) * ATOM_BYTES + row * 16 + b % 4] = (uint8_t)s;
        }
    }
    // Rows beyond A: codes 0 (their columns of the accumulator are not stored, whatever their scales).
    const int beyond = (NT - p.M) * 8;  // 16-byte pieces a stage
    for (int i = t; i < stages * beyond; i += threads) {
        const int stage = i / beyond, o = i - stage * beyond;
        reinterpret_cast<uint4 *>(codes + stage * NT * 128 + p.M * 128)[o] = make_uint4(0, 0, 0, 0);
    }
}

template <int NT, class T, int MODE>
__global__ void __launch_bounds__(TC_THREADS, 1) mxfp4_tc_kernel(const __grid_constant__ TcArgs p, unsigned *err)
{
    using L = TcTile<NT, MODE>;
    constexpr int S = L::STAGES;
    constexpr bool FUSED = L::FUSED;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = tc::cvta_smem(smem), bars = sbase + L::BAR_OFFSET;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full_bar = [&](int a) { return bars + 8u * (2 * S + a); };
    auto acc_free_bar = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (2 * S + 4), x_ready_bar = bars + 8u * (2 * S + 5);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + L::BAR_OFFSET + 8 * (2 * S + 6));

    // (Through a shuffle, so that branches on the warp are known to be uniform.)
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const unsigned long long lim = p.wait_limit_ns;
    const int stages_k = (p.blocks + TC_BLOCKS - 1) / TC_BLOCKS;
    int ranks = 1, rank = 0;
    if constexpr (MODE != WHOLE) {
        ranks = (int)cooperative_groups::this_cluster().num_blocks();
        rank = (int)cooperative_groups::this_cluster().block_rank();
    }
    // This CTA's stages of every tile of its own, and its tiles.
    const int k_first = (int)((long long)stages_k * rank / ranks), k_last = (int)((long long)stages_k * (rank + 1) / ranks);
    const long long tiles = (long long)p.tiles_x * p.tiles_w;
    const long long first_tile = MODE != WHOLE ? blockIdx.x / ranks : blockIdx.x;
    const long long tile_step = MODE != WHOLE ? tiles : gridDim.x;
    // Tile t: rows of A from x0, rows of B from w0.  Eight tiles along A are swept along B
    // together, so that tiles in flight share operands in L2.
    auto tile_at = [&](long long t, int &x0, int &w0) {
        const long long per_group = 8ll * p.tiles_w, group = t / per_group, in_group = t - group * per_group;
        const int height = min(p.tiles_x - (int)group * 8, 8);
        x0 = ((int)group * 8 + (int)(in_group % height)) * NT;
        w0 = (int)(in_group / height) * TC_ROWS;
    };

    if (warp == 0 && lane == 0) {
        prefetch_map(&p.w);
        if constexpr (!FUSED) prefetch_map(&p.x);
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(full_bar(s), 1);
            tc::mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(acc_full_bar(a), 1);
            tc::mbar_init(acc_free_bar(a), EPI_WARPS);
        }
        tc::mbar_init(drain_bar, 1);
        tc::mbar_init(x_ready_bar, EPI_WARPS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::cvta_smem(tmem_slot)),
                     "r"(L::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);
    // (The producer of a dependent product waits below, after it has asked for B.)
    if (!(MODE == SPLIT && p.dependent && warp == 0)) after_previous_kernel();

    if (warp == 0) {
        // ---- producer: the whole warp walks along, one lane issues ----
        // A stage: B's codes and scales, then A's codes and scales.
        auto load_w = [&](int k, int s, int w0) {
            const uint32_t at = sbase + s * L::STAGE_BYTES;
            const uint32_t sf_bytes = (p.atoms - 2ll * k > 1 ? 2 : 1) * ATOM_BYTES;  // the last may be alone
            tc::mbar_arrive_expect_tx(full_bar(s), L::W_BYTES + sf_bytes + (FUSED ? 0 : L::X_BYTES + sf_bytes));
            tma_load_2d(at, &p.w, full_bar(s), k * 128, w0);
            bulk_load(at + L::W_BYTES, p.w_scales + ((long long)(w0 / 128) * p.atoms + 2ll * k) * ATOM_BYTES, sf_bytes,
                      full_bar(s));
        };
        auto load_x = [&](int k, int s, int x0) {
            const uint32_t xc = sbase + s * L::STAGE_BYTES + L::W_BYTES + L::SF_BYTES;
            const uint32_t sf_bytes = (p.atoms - 2ll * k > 1 ? 2 : 1) * ATOM_BYTES;
            tma_load_2d(xc, &p.x, full_bar(s), k * 128, x0);
            bulk_load(xc + L::X_BYTES, p.x_scales + ((long long)(x0 / 128) * p.atoms + 2ll * k) * ATOM_BYTES, sf_bytes,
                      full_bar(s));
        };
        int g = 0;
        bool ok = true;
        for (long long t = first_tile; ok && t < tiles; t += tile_step) {
            int x0, w0, k = k_first;
            tile_at(t, x0, w0);
            if (MODE == SPLIT && p.dependent) {
                // The kernel before this one, which may still run, writes A and has itself waited for
                // all before it: B's part of the first stages, then the wait for it, then A's.
                int n = min(S, k_last - k_first);
                if (p.withhold >= 0) n = min(n, p.withhold);
                if (elect_one())
                    for (int i = 0; i < n; ++i) load_w(k_first + i, i, w0);
                __syncwarp();
                after_previous_kernel();
                if (elect_one())
                    for (int i = 0; i < n; ++i) load_x(k_first + i, i, x0);
                __syncwarp();
                k += n;
                g = n;
            }
            for (; k < k_last; ++k, ++g) {
                const int s = g % S, round = g / S;
                ok = (round == 0 || warp_wait(empty_bar(s), (round - 1) & 1, err, tc::ERR_PRODUCER, lim)) &&
                     g != p.withhold;  // (testing: as if this copy never arrived)
                if (!ok) break;
                if (elect_one()) {
                    load_w(k, s, w0);
                    if constexpr (!FUSED) load_x(k, s, x0);
                }
                __syncwarp();
            }
        }
        // Never leave with copies in flight into this CTA's shared memory.
        for (int k = g - S < 0 ? 0 : g - S; k < g; ++k)
            tc::mbar_wait(full_bar(k % S), (k / S) & 1, err, tc::ERR_DRAIN, lim, false);
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA: the whole warp walks along, one lane issues ----
        int g = 0, j = 0;
        bool ok = true;
        for (long long t = first_tile; ok && t < tiles; t += tile_step, ++j) {
            int x0, w0;
            tile_at(t, x0, w0);
            const int acc = j & 1;
            // Tile j - 2's sums have been read.
            if (j >= 2 && !warp_wait(acc_free_bar(acc), ((j >> 1) - 1) & 1, err, tc::ERR_MMA_WAIT, lim)) {
                ok = false;
                break;
            }
            if (FUSED && !warp_wait(x_ready_bar, 0, err, tc::ERR_MMA_WAIT, lim)) {
                ok = false;
                break;
            }
            tc::tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(acc * NT);
            for (int k = k_first; k < k_last; ++k, ++g) {
                const int s = g % S;
                ok = warp_wait(full_bar(s), (g / S) & 1, err, tc::ERR_MMA_WAIT, lim);
                if (!ok) break;
                tc::tc_fence_after();
                if (elect_one()) {
                    const uint32_t at = sbase + s * L::STAGE_BYTES, sf = at + L::W_BYTES;
                    uint32_t xc = sf + L::SF_BYTES, xf = xc + L::X_BYTES;
                    if constexpr (FUSED) {
                        xc = sbase + L::X_OFFSET + (k - k_first) * L::X_BYTES;
                        xf = sbase + L::X_OFFSET + (k_last - k_first) * L::X_BYTES + (k - k_first) * L::SF_BYTES;
                    }
                    const uint32_t sfw = tmem + L::SF_BASE + (uint32_t)((g & 1) * L::SF_COLS), sfx = sfw + 8;
                    const int left = p.blocks - k * TC_BLOCKS;  // blocks from here on
                    const uint64_t wd = tc::kmajor_sw128_desc(at), xd = tc::kmajor_sw128_desc(xc);
                    // A tile of 64 rows may start in the middle of its group's scales.
                    const uint32_t sfx_at = sfx + (uint32_t)(NT < 128 ? (x0 % 128) / 32 : 0);
                    // Two atoms of scales, each for two MMAs of two blocks.  (The MMAs that still
                    // read this buffer come earlier in the tensor core's order.)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        if (left > 4 * a) {
                            copy_atom(sfw + 4 * a, sf + a * ATOM_BYTES);
                            copy_atom(sfx + 4 * a, xf + a * ATOM_BYTES);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (left > 2 * i)
                            mma_mxf4(d, wd + 2u * i, xd + 2u * i, mxf4_idesc(NT, 2 * (i & 1)), sfw + 4 * (i >> 1),
                                     sfx_at + 4 * (i >> 1), k > k_first || i > 0);
                    tc::umma_commit(empty_bar(s));
                    if (k + 1 == k_last) tc::umma_commit(acc_full_bar(acc));
                }
                __syncwarp();
            }
        }
        if (!ok) {  // give up: nothing issued may still be running at teardown
            if (elect_one()) tc::umma_commit(drain_bar);
            __syncwarp();
            tc::mbar_wait(drain_bar, 0, err, tc::ERR_DRAIN, lim, false);
        }
        __syncwarp();
    } else {
        // ---- epilogue: warps of two sets of four, a set takes every other chunk ----
        const int q = warp & 3, set = (warp - 2) >> 2;
        if constexpr (FUSED) {
            const int stages = k_last - k_first;
            uint8_t *const codes = smem + L::X_OFFSET;
            quantize_tokens<NT, T>(p, codes, codes + stages * L::X_BYTES, stages, (long long)k_first * TC_DEPTH,
                                   (int)threadIdx.x - 64, 32 * EPI_WARPS);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor core reads them
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(x_ready_bar);
        }
        int j = 0;
        for (long long t = first_tile; t < tiles; t += tile_step, ++j) {
            int x0, w0;
            tile_at(t, x0, w0);
            const int acc = j & 1, n = w0 + 32 * q + lane;
            const float bias = p.bias && n < p.N ? p.bias[n] : 0.0f;  // (on its way during the wait)
            if (!warp_wait(acc_full_bar(acc), (j >> 1) & 1, err, tc::ERR_EPILOGUE, lim)) break;
            tc::tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * NT);
            T *const out = static_cast<T *>(p.c) + (long long)x0 * p.ldc + n;
            // (N even: a pair is inside or outside as a whole)
            const bool pairs = p.c_pairs && (p.N & 1) == 0;
            constexpr int CHUNKS = NT / L::CHUNK;
#pragma unroll 1
            for (int i = set; i < CHUNKS; i += 2) {
                const int c0 = i * L::CHUNK;
                uint32_t r[L::CHUNK];
                tmem_load(src + (uint32_t)c0, r);
                if (i + 2 >= CHUNKS) {  // this warp has read its part
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(acc_free_bar(acc));
                }
                if (MODE != WHOLE && ranks > 1) {
                    // Column c of the tile: 128 sums, one for each row of B.
                    float *const part = reinterpret_cast<float *>(smem) + c0 * TC_ROWS + 32 * q + lane;
#pragma unroll
                    for (int c = 0; c < L::CHUNK; ++c) part[c * TC_ROWS] = __uint_as_float(r[c]);
                } else {
                    store_chunk(p, out + c0 * p.ldc, r, bias, p.M - x0 - c0, n < p.N, pairs);
                }
            }
        }
        __syncwarp();
    }

    if (MODE != WHOLE && ranks > 1) {
        // Every CTA of the cluster adds up its share of the tile over the ranks, in rank order:
        // four rows of B (columns of C) of one row of A at a time.  (A rank that gave up leaves its
        // memory as it was; the error word says that C is undefined.)
        cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        int x0, w0;
        tile_at(first_tile, x0, w0);
        const int columns = min(NT, p.M - x0), from = columns * rank / ranks, to = columns * (rank + 1) / ranks;
        for (int i = threadIdx.x; i < (to - from) * (TC_ROWS / 4); i += TC_THREADS) {
            const int c = from + i / (TC_ROWS / 4), row = i % (TC_ROWS / 4) * 4, n = w0 + row;
            if (n >= p.N) continue;
            float4 part[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < ranks)
                    part[r] = *reinterpret_cast<const float4 *>(
                        cluster.map_shared_rank(reinterpret_cast<float *>(smem) + c * TC_ROWS + row, r));
            float sum[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < ranks) {
                    sum[0] += part[r].x;
                    sum[1] += part[r].y;
                    sum[2] += part[r].z;
                    sum[3] += part[r].w;
                }
            T *const out = static_cast<T *>(p.c) + (long long)(x0 + c) * p.ldc + n;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= p.N) break;
                const float bias = p.bias ? p.bias[n + e] : 0.0f;
                float o = p.beta != 0.0f ? finish<T, true, false>(p, out + e, sum[e], bias)
                                         : finish<T, false, false>(p, out + e, sum[e], bias);
                if (p.relu) o = relu(o);
                out[e] = from_float<T>(o);
            }
        }
        cluster.sync();
    }

    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::TMEM_COLS) : "memory");
    }
}

// ---- pairs of CTAs ----------------------------------------------------------------------

// Large products: a cluster of two CTAs works on 256 rows of B x 256 rows of A with
// tcgen05.mma.cta_group::2.  Each holds 128 rows of both operands in its shared memory and
// the sums of its own 128 rows of B in its tensor memory, so a stage brings 35 KB to each SM
// where one CTA alone needs 51 KB for as many sums: L2's bandwidth is what bounds that (the
// 51 KB stages came at 24 TB/s).  CTA 0 issues for both; its `full` barriers count the
// bytes that arrive in either CTA.
template <int NT>
struct PairTile {
    static constexpr int W_BYTES = 128 * 128, X_BYTES = NT / 2 * 128;  // bytes of either operand's rows
    static constexpr int SF_BYTES = 3 * 2 * ATOM_BYTES;  // own rows of B, both groups of A
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + SF_BYTES;
    static constexpr int STAGES = NT == 256 ? 6 : 7;
    static constexpr int ACC_STEP = 192, SF_BASE = ACC_STEP + NT, SF_COLS = 24;
    static constexpr int BAR_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int SMEM_BYTES = 1024 + BAR_OFFSET + (2 * STAGES + 6) * 8 + 8;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    static_assert(STAGE_BYTES % 1024 == 0, "the swizzle's alignment");
};

struct PairArgs {
    CUtensorMap w, x;    // codes: (bytes along K, rows), boxes of 128 x 128
    CUtensorMap sw, sx;  // scales: (words of an atom, atoms along K, groups of 128 rows)
    TcArgs t;            // the rest (its own maps and scale pointers are not used)
};

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void arrive_at(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// TMA loads of a CTA pair: into this CTA's memory, counted by a barrier of either CTA.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void pair_copy_atom(uint32_t tmem, uint32_t smem_addr)
{
    const uint64_t desc = (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` of both CTAs when the MMAs and copies issued so far are complete.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// The copies of a pair's CTA 1 are counted by CTA 0's barriers.  Where CTA 0 gives up some stages before CTA 1 (no more than the
// ring holds), these have to expect what CTA 1 has on its way, or nobody waits for it: CTA 1 tells how many stages it
// has asked for (tell_asked, at its producer's end), and CTA 0's producer, `ok` or having given up behind g, waits
// for that here and returns it; g where it is less or not told.  Having given up, not before the error is known: the barriers
// then let the MMA go on with a part of its operands missing.  (The count comes as a copy does, with its bytes on a
// barrier, and like one it is always waited for.  By a store and an arrival that releases it 4096 cubed took 0.3 us longer.)
__device__ __forceinline__ void tell_asked(uint32_t slot, uint32_t bar, int g)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(map_to_rank(slot, 0)), "r"(g),
                 "r"(map_to_rank(bar, 0))
                 : "memory");
}

__device__ __forceinline__ int asked_by_other(uint32_t slot, uint32_t bar, int g, bool ok, unsigned *err, unsigned long long lim)
{
    if (!ok) {
        const uint64_t t0 = tc::global_timer();
        while (*(volatile unsigned *)err == 0u)
            if (tc::global_timer() - t0 > 2 * lim) atomicOr(err, tc::ERR_PRODUCER);
    }
    if (elect_one()) tc::mbar_arrive_expect_tx(bar, 4);
    __syncwarp();
    // (CTA 1 is past its own waits soon after an error.)
    const bool told = tc::mbar_wait(bar, 0, err, tc::ERR_DRAIN, 2 * lim, false);
    if (!__all_sync(0xFFFFFFFFu, told)) return g;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    int asked;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(asked) : "r"(slot) : "memory");
    return max(g, __shfl_sync(0xFFFFFFFFu, asked, 0));
}

template <int NT, class T>
__global__ void __launch_bounds__(TC_THREADS, 1)
    mxfp4_pair_kernel(const __grid_constant__ PairArgs args, unsigned *err)
{
    using L = PairTile<NT>;
    constexpr int S = L::STAGES;
    const TcArgs &p = args.t;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = tc::cvta_smem(smem), bars = sbase + L::BAR_OFFSET;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto acc_full_bar = [&](int a) { return bars + 8u * (2 * S + a); };
    auto acc_free_bar = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (2 * S + 4), asked_bar = bars + 8u * (2 * S + 5);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + L::BAR_OFFSET + 8 * (2 * S + 6));
    const uint32_t asked_slot = bars + 8u * (2 * S + 6) + 4;  // of CTA 0: the stages that CTA 1 has asked for

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int rank = (int)cluster.block_rank();
    const unsigned long long lim = p.wait_limit_ns;
    const int stages_k = (p.blocks + TC_BLOCKS - 1) / TC_BLOCKS;
    const long long tiles = (long long)p.tiles_x * p.tiles_w;
    const long long first_tile = blockIdx.x / 2, tile_step = gridDim.x / 2;
    auto tile_at = [&](long long t, int &x0, int &w0) {  // as above; w0: the pair's first row of B
        const long long per_group = 8ll * p.tiles_w, group = t / per_group, in_group = t - group * per_group;
        const int height = min(p.tiles_x - (int)group * 8, 8);
        x0 = ((int)group * 8 + (int)(in_group % height)) * NT;
        w0 = (int)(in_group / height) * 256;
    };

    if (warp == 0 && lane == 0) {
        prefetch_map(&args.w);
        prefetch_map(&args.x);
        prefetch_map(&args.sw);
        prefetch_map(&args.sx);
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(full_bar(s), 1);
            tc::mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(acc_full_bar(a), 1);
            tc::mbar_init(acc_free_bar(a), 2 * EPI_WARPS);
        }
        tc::mbar_init(drain_bar, 1);
        tc::mbar_init(asked_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::cvta_smem(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc::tc_fence_before();
    cluster.sync();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);
    after_previous_kernel();

    if (warp == 0) {
        // ---- producer, one in each CTA ----
        int g = 0;
        bool ok = true;
        for (long long t = first_tile; ok && t < tiles; t += tile_step) {
            int x0, w0;
            tile_at(t, x0, w0);
            for (int k = 0; k < stages_k; ++k, ++g) {
                const int s = g % S, round = g / S;
                ok = (round == 0 || warp_wait(empty_bar(s), (round - 1) & 1, err, tc::ERR_PRODUCER, lim)) &&
                     (g != p.withhold || rank == 1);  // (testing: as if this copy never arrived)
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t at = sbase + s * L::STAGE_BYTES, sf = at + L::W_BYTES + L::X_BYTES;
                    if (rank == 0) tc::mbar_arrive_expect_tx(full_bar(s), 2 * L::STAGE_BYTES);
                    const uint32_t bar = map_to_rank(full_bar(s), 0);
                    pair_load_2d(at, &args.w, bar, k * 128, w0 + 128 * rank);
                    pair_load_2d(at + L::W_BYTES, &args.x, bar, k * 128, x0 + NT / 2 * rank);
                    pair_load_3d(sf, &args.sw, bar, 0, 2 * k, w0 / 128 + rank);
                    pair_load_3d(sf + 2 * ATOM_BYTES, &args.sx, bar, 0, 2 * k, x0 / 128);
                }
                __syncwarp();
            }
        }
        // Never leave with copies in flight into either CTA's shared memory.
        if (rank == 1) {
            if (elect_one()) tell_asked(asked_slot, asked_bar, g);
        } else {
            for (const int asked = asked_by_other(asked_slot, asked_bar, g, ok, err, lim); g < asked; ++g)
                if (elect_one()) tc::mbar_arrive_expect_tx(full_bar(g % S), L::STAGE_BYTES);
        }
        __syncwarp();
        if (rank == 0)
            for (int k = g - S < 0 ? 0 : g - S; k < g; ++k)
                tc::mbar_wait(full_bar(k % S), (k / S) & 1, err, tc::ERR_DRAIN, lim, false);
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA, by CTA 0 for both ----
        if (rank == 0) {
            int g = 0, j = 0;
            bool ok = true;
            for (long long t = first_tile; ok && t < tiles; t += tile_step, ++j) {
                int x0, w0;
                tile_at(t, x0, w0);
                const int acc = j & 1, before = NT == 256 ? j - 1 : j - 2;
                if (before >= 0 && !warp_wait(acc_free_bar(before & 1), (before >> 1) & 1, err, tc::ERR_MMA_WAIT, lim)) {
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * L::ACC_STEP);
                for (int k = 0; k < stages_k; ++k, ++g) {
                    const int s = g % S;
                    ok = warp_wait(full_bar(s), (g / S) & 1, err, tc::ERR_MMA_WAIT, lim);
                    if (!ok) break;
                    tc::tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = sbase + s * L::STAGE_BYTES, sf = at + L::W_BYTES + L::X_BYTES;
                        const uint32_t sfw = tmem + L::SF_BASE + (uint32_t)((g & 1) * L::SF_COLS), sfx = sfw + 8;
                        const int left = p.blocks - k * TC_BLOCKS;
                        const uint64_t wd = tc::kmajor_sw128_desc(at), xd = tc::kmajor_sw128_desc(at + L::W_BYTES);
                        const uint32_t sfx_at = sfx + (uint32_t)(x0 % 128) / 32;  // a tile may start inside its group
                        constexpr uint32_t tall = (uint32_t)(TC_ROWS >> 4) << 24;  // 256 rows in place of 128
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            if (left > 4 * a) {
                                pair_copy_atom(sfw + 4 * a, sf + a * ATOM_BYTES);
                                pair_copy_atom(sfx + 8 * a, sf + (2 + a) * ATOM_BYTES);
                                pair_copy_atom(sfx + 8 * a + 4, sf + (4 + a) * ATOM_BYTES);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (left > 2 * i)
                                pair_mma(d, wd + 2u * i, xd + 2u * i, mxf4_idesc(NT, 2 * (i & 1)) + tall,
                                         sfw + 4 * (i >> 1), sfx_at + 8 * (i >> 1), k > 0 || i > 0);
                        pair_commit(empty_bar(s));
                        if (k + 1 == stages_k) pair_commit(acc_full_bar(acc));
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // give up: nothing issued may still be running at teardown
                if (elect_one()) pair_commit(drain_bar);
                __syncwarp();
                tc::mbar_wait(drain_bar, 0, err, tc::ERR_DRAIN, lim, false);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue, each CTA its own 128 rows of B ----
        const int q = warp & 3, set = (warp - 2) >> 2;
        const bool pairs = p.c_pairs && (p.N & 1) == 0;
        int j = 0;
        for (long long t = first_tile; t < tiles; t += tile_step, ++j) {
            int x0, w0;
            tile_at(t, x0, w0);
            const int acc = j & 1, n = w0 + 128 * rank + 32 * q + lane;
            const float bias = p.bias && n < p.N ? p.bias[n] : 0.0f;  // (on its way during the wait)
            if (!warp_wait(acc_full_bar(acc), (j >> 1) & 1, err, tc::ERR_EPILOGUE, lim)) break;
            tc::tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * L::ACC_STEP);
            T *const out = static_cast<T *>(p.c) + (long long)x0 * p.ldc + n;
#pragma unroll 1
            for (int i = set; i < NT / 32; i += 2) {
                const int c0 = (NT == 256 && acc == 0 ? 7 - i : i) * 32;
                uint32_t r[32];
                tmem_load(src + (uint32_t)c0, r);
                if (NT == 256 ? i == set : i + 2 >= NT / 32) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(map_to_rank(acc_free_bar(acc), 0));
                }
                store_chunk(p, out + c0 * p.ldc, r, bias, p.M - x0 - c0, n < p.N, pairs);
            }
        }
        __syncwarp();
    }

    // Neither CTA leaves while the other may still reach its memory.
    tc::tc_fence_before();
    cluster.sync();
    if (warp == 1) {
        tc::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace mx
}  // namespace fgemm
