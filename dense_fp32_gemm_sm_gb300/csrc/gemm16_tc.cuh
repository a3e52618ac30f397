// gemm16_tc.cuh -- products of 16-bit matrices (BF16 or F16) on the tensor cores of sm_103a
// (tcgen05.mma kind::f16, FP32 accumulators), with a layer's epilogue, for one matrix or a
// weight for each group of rows.
//
//   P = alpha op(A) op(B);   Y = act(P + bias) + beta R, or Y = P act'(Z) with Y's column sums
//
// The MMA's rows are columns of Y (128 a CTA) and its columns are rows of Y (up to 256): an
// accumulator lane is then a column of Y, a warp's 32 lanes are neighbours in a row of Y, and the
// epilogue reads R and Z and stores Y and Z straight from registers, for any leading dimension
// and alignment; a column sum is a sum in one lane; and a short tile (the end of a group, few
// tokens) takes an MMA of as many columns as it has rows, in steps of 16.
//
// A stage is 64 deep: 128 bytes a row, the 128-byte swizzle's row.  Either operand may be stored
// along the depth (K-major boxes of 64 x rows) or across it (boxes of 64 rows x 64 deep); the
// MMA takes both.  One warp streams stages by TMA, one issues MMAs, eight store the sums of the
// tile before.
//
// Groups (experts) come as a device array of row offsets, which the host does not see: every CTA
// reads it after its wait for the kernel before, and walks the tiles of all groups; a group
// without rows has none.  Offsets are clamped to 0 .. M and to each other, so that wrong ones reach
// no other memory.  Where the rows of a group are the depth (the weights' gradient), a group's
// last stage reaches into the next group: its rows from the group's end up to the MMA's 16 are
// overwritten with zeros in shared memory, in both operands (0 * NaN).
#pragma once

#include "gemm16.h"
#include "gemm16_device.cuh"
#include "mxfp4_tc.cuh"

namespace fgemm {
namespace h16 {

constexpr int TILE_F = 128;      // columns of Y a CTA: tensor-memory lanes
constexpr int DEPTH = 64;        // 16-bit elements of a stage: 128 bytes
constexpr int THREADS = 320;     // producer, MMA, eight epilogue warps
constexpr int EPI_WARPS = 8;
constexpr int MAX_STAGES = 12;
constexpr int W_BYTES = TILE_F * 128;
constexpr int BLOCK_BYTES = 64 * 128;  // a box of an operand stored across the depth
constexpr int ROWS_SWEPT = 8;          // tiles of rows that are swept along the columns together

struct Args {
    CUtensorMap w, x;  // op(B): columns of Y; op(A): rows of Y
    Product q;
    int w_across, x_across;  // stored across the depth
    int nt, step;            // most rows of a tile; rows of a tile of the one product
    int tiles_t, tiles_f;    // of one product (RAGGED_ROWS: tiles_t is not known here)
    int x_box;               // rows of a box of A stored along the depth
    int stages, stage_bytes, acc_step, tmem_cols;
    int table;               // offset in shared memory of the groups' table
    int y_pairs, z_pairs;    // pairs of columns are aligned
    unsigned long long wait_limit_ns;
    int withhold;
};

// Offsets in shared memory behind the ring: barriers, then the slot for tensor memory's address.
__host__ __device__ constexpr int bar_bytes(int stages) { return (3 * stages + 5) * 8 + 8; }

// MMA descriptors.  Along the depth: as of the other tensor-core kernels.  Across it: boxes of 64 elements x
// 64 deep, 128 bytes an entry of depth; 8 of depth are 1024 bytes apart (stride), 64 elements a box (leading).
__device__ __forceinline__ uint64_t across_desc(uint32_t smem_addr)
{
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(BLOCK_BYTES >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// A wait for an arrival of the other CTA of a pair, whose writes it makes visible.
__device__ __forceinline__ bool cluster_wait(uint32_t bar, uint32_t parity, unsigned *err, unsigned code,
                                             unsigned long long limit_ns)
{
    const uint64_t t0 = tc::global_timer();
    for (uint32_t spin = 1;; ++spin) {
        uint32_t done;
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n"
            "}\n"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (__all_sync(0xFFFFFFFFu, done)) return true;
        if ((spin & 255u) == 0) {
            bool stop = *(volatile unsigned *)err != 0u;
            if (!stop && tc::global_timer() - t0 > limit_ns) {
                atomicOr(err, code);
                stop = true;
            }
            if (__any_sync(0xFFFFFFFFu, stop)) return false;
        }
    }
}

// A tile: rows t0 .. t0 + valid of the output, columns from f0, group e, depth k0 .. k0 + depth;
// row_tile: its number among all tiles of rows.
struct Tile {
    int t0, valid, f0, e, k0, depth, row_tile;
};

// The tiles of a product, for each role by itself.  Eight tiles of rows are swept along the columns
// together, so that the tiles in flight share operands in L2.
struct Walk {
    const Args &p;
    const int *begin, *first;  // table: a group's first row, its first tile
    int tile_f, group;

    __device__ Walk(const Args &args, const int *table, int columns)
        : p(args), begin(table), first(table + args.q.groups + 1), tile_f(columns), group(0)
    {
    }

    __device__ __forceinline__ int tiles() const
    {
        if (p.q.ragged == RAGGED_ROWS) return first[p.q.groups];
        return p.tiles_t * p.tiles_f * (p.q.ragged == RAGGED_DEPTH ? p.q.groups : 1);
    }

    __device__ __forceinline__ Tile at(int t)
    {
        Tile o;
        int tiles_t = p.tiles_t, step = p.step, rows = p.q.M, row0 = 0, row_tile0 = 0;
        o.e = 0;
        o.k0 = 0;
        o.depth = p.q.K;
        if (p.q.ragged == RAGGED_ROWS) {
            while (t >= first[group + 1]) ++group;  // (t only grows)
            o.e = group;
            tiles_t = (first[group + 1] - first[group]) / p.tiles_f;
            t -= first[group];
            row0 = begin[group];
            rows = begin[group + 1] - row0;
            step = ((rows + tiles_t - 1) / tiles_t + 31) & ~31;
            step = min(step, p.nt);
            row_tile0 = first[group] / p.tiles_f;
        } else if (p.q.ragged == RAGGED_DEPTH) {
            const int per = p.tiles_t * p.tiles_f;
            o.e = t / per;
            t -= o.e * per;
            o.k0 = begin[o.e];
            o.depth = begin[o.e + 1] - o.k0;
        }
        const int per_sweep = ROWS_SWEPT * p.tiles_f, sweep = t / per_sweep, in = t - sweep * per_sweep;
        const int height = min(tiles_t - sweep * ROWS_SWEPT, ROWS_SWEPT);
        const int i = sweep * ROWS_SWEPT + in % height;
        o.f0 = in / height * tile_f;
        o.t0 = row0 + i * step;
        o.valid = min(step, rows - i * step);
        o.row_tile = row_tile0 + i;
        if (p.q.alpha == 0.0f) o.depth = 0;
        return o;
    }
};

// The groups' table from the offsets, by one warp: monotone first rows, then (RAGGED_ROWS) first tiles.
__device__ __forceinline__ void make_table(const Args &p, int *table, int lane)
{
    const int E = p.q.groups, limit = p.q.ragged == RAGGED_DEPTH ? p.q.K : p.q.M;
    int *const begin = table, *const first = table + E + 1;
    int most = max(0, min(p.q.offsets[0], limit)), tiles = 0;
    if (lane == 0) {
        begin[0] = most;
        first[0] = 0;
    }
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int end = e < E ? max(0, min(p.q.offsets[e + 1], limit)) : 0;
        end = max(end, most);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int other = __shfl_up_sync(0xFFFFFFFFu, end, d);
            if (lane >= d) end = max(end, other);
        }
        const int before = __shfl_up_sync(0xFFFFFFFFu, end, 1), rows = end - (lane == 0 ? most : before);
        int sum = p.q.ragged == RAGGED_ROWS ? (rows + p.nt - 1) / p.nt * p.tiles_f : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int other = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += other;
        }
        if (e < E) {
            begin[e + 1] = end;
            first[e + 1] = tiles + sum;
        }
        most = __shfl_sync(0xFFFFFFFFu, end, 31);
        tiles += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
}

// ---- epilogue ---------------------------------------------------------------------------

// Elements [row c][this lane's column], c < rows, into v.
template <class T>
__device__ __forceinline__ void load_rows(float (&v)[32], const T *src, long long ld, int rows, bool in)
{
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = in && c < rows ? to_float(src[c * ld]) : 0.0f;
}

// Store v to rows c < rows of this lane's column.  16-bit types, where pairs of columns are aligned:
// lanes 2i and 2i + 1 exchange their values of two rows, and each stores both columns of one.
template <class T>
__device__ __forceinline__ void store_rows(T *out, long long ld, const float (&v)[32], int rows, bool in, bool pairs)
{
    if constexpr (sizeof(T) == 2) {
        if (pairs) {
            const int odd = threadIdx.x & 1;
            T *dst = out + (odd ? ld - 1 : 0);
#pragma unroll
            for (int c = 0; c < 32; c += 2, dst += 2 * ld) {
                const T a = from_float<T>(v[c]), b = from_float<T>(v[c + 1]);
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
#pragma unroll
    for (int c = 0; c < 32; ++c, out += ld)
        if (c < rows) *out = from_float<T>(v[c]);
}

// 32 sums of this lane's column (rows from `row` on) to their place (stride_y is 0 unless each group has an output); returns the sum of what Y
// holds of them, before its rounding.
template <class T, class O>
__device__ __forceinline__ float finish_rows(const Args &p, float (&v)[32], long long row, int n, int e, float bias, int rows,
                                             bool in)
{
    const Product &q = p.q;
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = fmaf(q.alpha, v[c], bias);
    if (q.slope) {
        if (q.act != FGEMM_ACT_NONE) {
            float z[32];
            load_rows(z, static_cast<const T *>(q.z) + row * q.ldz + n, q.ldz, rows, in);
            if (q.act == FGEMM_ACT_RELU) {
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = through(v[c], z[c], FGEMM_ACT_RELU);
            } else if (q.act == FGEMM_ACT_GELU) {
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = through(v[c], z[c], FGEMM_ACT_GELU);
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = through(v[c], z[c], FGEMM_ACT_SILU);
            }
        }
    } else {
        if (q.z) store_rows(static_cast<T *>(q.z) + row * q.ldz + n, q.ldz, v, rows, in, p.z_pairs);
        if (q.act == FGEMM_ACT_RELU) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = relu(v[c]);
        } else if (q.act == FGEMM_ACT_GELU) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = gelu(v[c]);
        } else if (q.act == FGEMM_ACT_SILU) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = silu(v[c]);
        }
        if (q.beta != 0.0f) {
            float r[32];
            load_rows(r, static_cast<const O *>(q.r) + e * q.stride_y + row * q.ldr + n, q.ldr, rows, in);
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = fmaf(q.beta, r[c], v[c]);
        }
    }
    store_rows(static_cast<O *>(q.y) + e * q.stride_y + row * q.ldy + n, q.ldy, v, rows, in, p.y_pairs);
    float sum = 0.0f;
    if (q.partial) {
#pragma unroll
        for (int c = 0; c < 32; ++c) sum += c < rows ? v[c] : 0.0f;
    }
    return sum;
}

// The same for one element.
template <class T, class O>
__device__ __forceinline__ void finish_one(const Args &p, float sum, long long row, int n, int e)
{
    const Product &q = p.q;
    float v = q.alpha * sum;
    if (q.slope) {
        if (q.act != FGEMM_ACT_NONE) v = through(v, to_float(static_cast<const T *>(q.z)[row * q.ldz + n]), q.act);
    } else {
        if (q.bias) v += q.bias[(long long)e * q.N + n];
        if (q.z) static_cast<T *>(q.z)[row * q.ldz + n] = from_float<T>(v);
        v = activate(v, q.act);
        if (q.beta != 0.0f) v = fmaf(q.beta, to_float(static_cast<const O *>(q.r)[e * q.stride_y + row * q.ldr + n]), v);
    }
    static_cast<O *>(q.y)[e * q.stride_y + row * q.ldy + n] = from_float<O>(v);
}

// Zero rows `from` .. `to` (entries of depth) of `blocks` boxes stored across the depth, by a warp.
__device__ __forceinline__ void zero_depth(uint32_t base, int blocks, int from, int to, int lane)
{
    const int per = (to - from) * 8;
    for (int i = lane; i < blocks * per; i += 32) {
        const int b = i / per, o = i - b * per;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + b * BLOCK_BYTES + from * 128 + o * 16), "r"(0)
                     : "memory");
    }
}

// A ring position and its phase.
struct Slot {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
};

// PAIR: a cluster of two CTAs works on 256 columns of Y with cta_group::2; each holds its own 128
// columns of op(B) and half of the tile's rows of op(A).  CTA 0 issues for both; its `full`
// barriers count what arrives in either.  Else `ranks` CTAs of a cluster divide the depth of one
// tile, or a CTA walks whole tiles.
template <bool PAIR, class T, class O>
__global__ void __launch_bounds__(THREADS, 1) gemm16_kernel(const __grid_constant__ Args p, unsigned *err)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, bar_offset = S * p.stage_bytes;
    const uint32_t sbase = tc::cvta_smem(smem), bars = sbase + bar_offset;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto fixed_bar = [&](int s) { return bars + 8u * (2 * S + s); };
    auto acc_full_bar = [&](int a) { return bars + 8u * (3 * S + a); };
    auto acc_free_bar = [&](int a) { return bars + 8u * (3 * S + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (3 * S + 4);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + bar_offset + 8 * (3 * S + 5));
    int *const table = reinterpret_cast<int *>(smem + p.table);

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const unsigned long long lim = p.wait_limit_ns;
    const bool split = !PAIR && ranks > 1;

    if (warp == 0 && lane == 0) {
        mx::prefetch_map(&p.w);
        mx::prefetch_map(&p.x);
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(full_bar(s), 1);
            tc::mbar_init(empty_bar(s), 1);
            tc::mbar_init(fixed_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(acc_full_bar(a), 1);
            tc::mbar_init(acc_free_bar(a), (PAIR ? 2 : 1) * EPI_WARPS);
        }
        tc::mbar_init(drain_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::cvta_smem(tmem_slot)),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::cvta_smem(tmem_slot)),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    after_previous_kernel();
    if (p.q.ragged != RAGGED_NONE && warp == 2) make_table(p, table, lane);
    tc::tc_fence_before();
    if constexpr (PAIR)
        cluster.sync();
    else
        __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);

    constexpr int COLUMNS = PAIR ? 2 * TILE_F : TILE_F;
    Walk walk(p, table, COLUMNS);
    const int tiles = walk.tiles();
    const int first_tile = (int)blockIdx.x / ranks, tile_step = (int)gridDim.x / ranks;
    const bool fix_depth = p.q.ragged == RAGGED_DEPTH;
    // A tile's stages that are this CTA's.
    auto stages_of = [&](const Tile &o, int &from) {
        const int all = (int)(((long long)o.depth + DEPTH - 1) / DEPTH);
        from = 0;
        if (!split) return all;
        from = (int)((long long)all * rank / ranks);
        return (int)((long long)all * (rank + 1) / ranks) - from;
    };
    // MMA columns of a tile, and the rows of op(A) that this CTA brings for them.
    auto mma_cols = [&](const Tile &o) { return PAIR ? (o.valid + 31) & ~31 : (o.valid + 15) & ~15; };
    // Whether a stage with `left` of its depth to come ends inside the MMA's 16.
    auto wants_fix = [&](int left) { return fix_depth && left < DEPTH && (left & 15) != 0; };

    if (warp == 0) {
        // ---- producer (one in each CTA): the whole warp walks along, one lane issues ----
        Slot at;
        int g = 0;
        bool ok = true;
        uint32_t own_phase = 0, own_used = 0;  // rank 1 of a pair: stages that its own barriers count
        for (int t = first_tile; ok && t < tiles; t += tile_step) {
            const Tile o = walk.at(t);
            int from;
            const int n = stages_of(o, from), cols = mma_cols(o), own = PAIR ? cols / 2 : cols;
            const int boxes = p.x_across ? (own + 63) / 64 : (own + p.x_box - 1) / p.x_box;
            const uint32_t box_bytes = p.x_across ? BLOCK_BYTES : p.x_box * 128;
            const uint32_t bytes = W_BYTES + boxes * box_bytes;
            const int f = o.f0 + (PAIR ? TILE_F * rank : 0), x0 = o.t0 + (PAIR ? own * rank : 0);
            for (int k = from; k < from + n; ++k, ++g) {
                ok = mx::warp_wait(empty_bar(at.s), at.phase ^ 1, err, tc::ERR_PRODUCER, lim) &&
                     g != p.withhold;  // (testing: as if this copy never arrived)
                if (!ok) break;
                const bool fix = PAIR && wants_fix(o.depth - k * DEPTH);
                if (mx::elect_one()) {
                    const uint32_t w_at = sbase + at.s * p.stage_bytes, x_at = w_at + W_BYTES;
                    const int depth = o.k0 + k * DEPTH, e = fix_depth ? 0 : o.e;
                    if (!PAIR || fix) {
                        const uint32_t bar = full_bar(at.s);
                        tc::mbar_arrive_expect_tx(bar, bytes);
                        if (p.w_across) {
                            tc::tma_load_3d(w_at, &p.w, bar, f, depth, e);
                            tc::tma_load_3d(w_at + BLOCK_BYTES, &p.w, bar, f + 64, depth, e);
                        } else {
                            tc::tma_load_3d(w_at, &p.w, bar, depth, f, e);
                        }
                        for (int b = 0; b < boxes; ++b) {
                            if (p.x_across)
                                mx::tma_load_2d(x_at + b * BLOCK_BYTES, &p.x, bar, x0 + 64 * b, depth);
                            else
                                mx::tma_load_2d(x_at + b * box_bytes, &p.x, bar, depth, x0 + p.x_box * b);
                        }
                    } else {
                        if (rank == 0) tc::mbar_arrive_expect_tx(full_bar(at.s), 2 * bytes);
                        const uint32_t bar = mx::map_to_rank(full_bar(at.s), 0);
                        if (p.w_across) {
                            mx::pair_load_3d(w_at, &p.w, bar, f, depth, e);
                            mx::pair_load_3d(w_at + BLOCK_BYTES, &p.w, bar, f + 64, depth, e);
                        } else {
                            mx::pair_load_3d(w_at, &p.w, bar, depth, f, e);
                        }
                        for (int b = 0; b < boxes; ++b) {
                            if (p.x_across)
                                mx::pair_load_2d(x_at + b * BLOCK_BYTES, &p.x, bar, x0 + 64 * b, depth);
                            else
                                mx::pair_load_2d(x_at + b * box_bytes, &p.x, bar, depth, x0 + p.x_box * b);
                        }
                    }
                }
                __syncwarp();
                if (fix && rank == 1) {
                    own_used |= 1u << at.s;
                    own_phase ^= 1u << at.s;
                }
                at.next(S);
            }
        }
        // Never leave with copies in flight into either CTA's shared memory.
        if (!PAIR || rank == 0) {
            for (int k = g - S < 0 ? 0 : g - S; k < g; ++k)
                tc::mbar_wait(full_bar(k % S), (k / S) & 1, err, tc::ERR_DRAIN, lim, false);
        } else {
            for (int s = 0; s < S; ++s)
                if (own_used >> s & 1) tc::mbar_wait(full_bar(s), (own_phase >> s & 1) ^ 1, err, tc::ERR_DRAIN, lim, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA (of a pair: by CTA 0 for both) ----
        Slot at;
        bool ok = true;
        uint32_t fix_phase = 0;
        if (!PAIR || rank == 0) {
            int j = 0;
            const uint32_t fmt = sizeof(T) == 2 && p.q.type == FGEMM_BF16 ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t idesc0 = (1u << 4) | fmt | ((uint32_t)p.w_across << 15) | ((uint32_t)p.x_across << 16) |
                                    ((uint32_t)(COLUMNS >> 4) << 24);
            for (int t = first_tile; ok && t < tiles; t += tile_step) {
                const Tile o = walk.at(t);
                int from;
                const int n = stages_of(o, from), cols = mma_cols(o);
                if (n == 0) continue;
                const int acc = j & 1;
                // Tile j - 2's sums have been read.
                if (j >= 2 && !mx::warp_wait(acc_free_bar(acc), ((j >> 1) - 1) & 1, err, tc::ERR_MMA_WAIT, lim)) {
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * p.acc_step), idesc = idesc0 | ((uint32_t)(cols >> 3) << 17);
                for (int k = from; k < from + n; ++k) {
                    ok = mx::warp_wait(full_bar(at.s), at.phase, err, tc::ERR_MMA_WAIT, lim);
                    if (!ok) break;
                    const int left = o.depth - k * DEPTH, steps = min(DEPTH / 16, (left + 15) / 16);
                    const uint32_t w_at = sbase + at.s * p.stage_bytes, x_at = w_at + W_BYTES;
                    if (wants_fix(left)) {
                        zero_depth(w_at, 2, left, 16 * steps, lane);
                        zero_depth(x_at, ((PAIR ? cols / 2 : cols) + 63) / 64, left, 16 * steps, lane);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor core reads them
                        __syncwarp();
                        if (PAIR) {
                            ok = cluster_wait(fixed_bar(at.s), fix_phase >> at.s & 1, err, tc::ERR_MMA_WAIT, lim);
                            fix_phase ^= 1u << at.s;
                            if (!ok) break;
                        }
                    }
                    tc::tc_fence_after();
                    if (mx::elect_one()) {
                        const uint64_t wd = p.w_across ? across_desc(w_at) : tc::kmajor_sw128_desc(w_at);
                        const uint64_t xd = p.x_across ? across_desc(x_at) : tc::kmajor_sw128_desc(x_at);
                        // 16 of depth: 32 bytes along it, 16 rows of 128 bytes across it.
                        const uint32_t wi = p.w_across ? 128u : 2u, xi = p.x_across ? 128u : 2u;
                        for (int i = 0; i < steps; ++i)
                            mma<PAIR>(d, wd + wi * i, xd + xi * i, idesc, k > from || i > 0);
                        if constexpr (PAIR) {
                            mx::pair_commit(empty_bar(at.s));
                            if (k + 1 == from + n) mx::pair_commit(acc_full_bar(acc));
                        } else {
                            tc::umma_commit(empty_bar(at.s));
                            if (k + 1 == from + n) tc::umma_commit(acc_full_bar(acc));
                        }
                    }
                    __syncwarp();
                    at.next(S);
                }
                ++j;
            }
            if (!ok) {  // give up: nothing issued may still be running at teardown
                if (mx::elect_one()) {
                    if constexpr (PAIR)
                        mx::pair_commit(drain_bar);
                    else
                        tc::umma_commit(drain_bar);
                }
                __syncwarp();
                tc::mbar_wait(drain_bar, 0, err, tc::ERR_DRAIN, lim, false);
            }
        } else if (fix_depth) {
            // CTA 1 of a pair overwrites its own part of the stages that a group ends in.
            for (int t = first_tile; ok && t < tiles; t += tile_step) {
                const Tile o = walk.at(t);
                int from;
                const int n = stages_of(o, from), left = o.depth - (n - 1) * DEPTH;
                for (int k = 0; k + 1 < n; ++k) at.next(S);
                if (n == 0) continue;
                if (wants_fix(left)) {
                    ok = mx::warp_wait(full_bar(at.s), fix_phase >> at.s & 1, err, tc::ERR_MMA_WAIT, lim);
                    fix_phase ^= 1u << at.s;
                    if (!ok) break;
                    const uint32_t w_at = sbase + at.s * p.stage_bytes;
                    const int to = (left + 15) & ~15;
                    zero_depth(w_at, 2, left, to, lane);
                    zero_depth(w_at + W_BYTES, (mma_cols(o) / 2 + 63) / 64, left, to, lane);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mx::arrive_at(mx::map_to_rank(fixed_bar(at.s), 0));
                }
                at.next(S);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: warps of two sets of four, a set takes every other chunk of 32 rows ----
        const int q = warp & 3, set = (warp - 2) >> 2;
        int j = 0;
        for (int t = first_tile; t < tiles; t += tile_step) {
            const Tile o = walk.at(t);
            int from;
            const bool products = stages_of(o, from) > 0;
            const int acc = j & 1, n = o.f0 + (PAIR ? TILE_F * rank : 0) + 32 * q + lane;
            const bool in = n < p.q.N;
            // (on its way during the wait)
            const float bias = p.q.bias && in && !split ? p.q.bias[(long long)o.e * p.q.N + n] : 0.0f;
            if (products && !mx::warp_wait(acc_full_bar(acc), (j >> 1) & 1, err, tc::ERR_EPILOGUE, lim)) break;
            tc::tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * p.acc_step);
            float sum = 0.0f;
#pragma unroll 1
            for (int c0 = 32 * set; c0 < o.valid; c0 += 64) {
                uint32_t r[32];
                if (products) {
                    tc::tmem_ld_32cols(src + (uint32_t)c0, r);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) r[c] = 0;
                }
                float v[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
                if (split) {  // row c of the tile: 128 sums, one for each column
                    float *const part = reinterpret_cast<float *>(smem) + c0 * TILE_F + 32 * q + lane;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c0 + c < o.valid) part[c * TILE_F] = v[c];
                } else {
                    sum += finish_rows<T, O>(p, v, (long long)o.t0 + c0, n, o.e, bias, o.valid - c0, in);
                }
            }
            if (products) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        mx::arrive_at(mx::map_to_rank(acc_free_bar(acc), 0));
                    else
                        tc::mbar_arrive(acc_free_bar(acc));
                }
                ++j;
            }
            const long long part = 2ll * o.row_tile + set;
            if (p.q.partial && in && part < p.q.partials) p.q.partial[part * p.q.N + n] = sum;
        }
        __syncwarp();
    }

    if (split) {
        // Every CTA of the cluster adds up its share of the tile's rows over the ranks, in rank order.
        // (A rank that gave up leaves its memory as it was; the error word says that Y is undefined.)
        cluster.sync();
        if (first_tile < tiles) {
            Walk again(p, table, COLUMNS);
            const Tile o = again.at(first_tile);
            const int from = o.valid * rank / ranks, to = o.valid * (rank + 1) / ranks;
            for (int i = threadIdx.x; i < (to - from) * TILE_F; i += THREADS) {
                const int c = from + i / TILE_F, f = i % TILE_F, n = o.f0 + f;
                if (n >= p.q.N) continue;
                float part[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < ranks) part[r] = *cluster.map_shared_rank(reinterpret_cast<float *>(smem) + c * TILE_F + f, r);
                float sum = part[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < ranks) sum += part[r];
                finish_one<T, O>(p, sum, (long long)o.t0 + c, n, o.e);
            }
        }
        cluster.sync();
    }

    if (p.q.partial_start && blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= p.q.groups; e += THREADS)
            p.q.partial_start[e] = p.q.ragged == RAGGED_ROWS ? 2 * (walk.first[e] / p.tiles_f) : 2 * p.tiles_t * e;
    }

    // No CTA of a pair leaves while the other may still reach its memory.
    tc::tc_fence_before();
    if constexpr (PAIR)
        cluster.sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

}  // namespace h16
}  // namespace fgemm
