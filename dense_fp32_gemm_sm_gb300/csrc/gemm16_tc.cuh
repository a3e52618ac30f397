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
// A stage is one or two blocks of a depth of 64: 128 bytes a row, the 128-byte swizzle's row.  (Two
// where room for three such stages is left: a stage's way through the barriers takes the producer
// and the MMA warp some 170 ns, which is what bounds short tiles.)  Either operand may be stored
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
constexpr int DEPTH = 64;        // 16-bit elements of a block: 128 bytes
constexpr int SETS = 2;  // of four epilogue warps: one for 32 lanes of tensor memory each
__host__ __device__ constexpr int threads_of(bool pair) { return 64 + 128 * SETS + (pair ? 32 : 0); }  // producer, MMA, epilogue; mender
constexpr int CHUNK = 16;      // accumulator columns that a warp finishes at a time
constexpr int Z_SLOTS = 4;     // of a warp's ring of Z: chunks of 16 rows by 32 columns
constexpr int Z_SLOT_BYTES = CHUNK * 64;

constexpr int MAX_STAGES = 12;
constexpr int W_BYTES = TILE_F * 128;
constexpr int BOX_BYTES = 64 * 128;  // a box of an operand stored across the depth
constexpr int MAX_BOXES = 4;            // of op(A), a stage and CTA
constexpr int ROWS_SWEPT = 8;          // tiles of rows that are swept along the columns together

struct Args {
    CUtensorMap w, x;  // op(B): columns of Y; op(A): rows of Y
    Product q;
    int w_across, x_across;  // stored across the depth
    int nt, step;            // most rows of a tile; rows of a tile of the one product
    int tiles_t, tiles_f;    // of one product (RAGGED_ROWS: tiles_t is not known here)
    int x_box;               // rows of a box of A stored along the depth
    int stages, stage_bytes, acc_step, tmem_cols;
    int blocks, block_bytes;  // 64-deep blocks of a stage (1 or 2), each of op(B), then of op(A)
    int table, join;         // offsets in shared memory: the groups' table, the sums that ranks send each other
    int y_pairs, z_pairs, r_pairs;  // pairs of columns are aligned
    int z_ring;  // offset in shared memory of the rings of Z whose slope is taken; 0: Z comes to registers
    unsigned long long wait_limit_ns;
    int withhold;
};

// Offsets in shared memory behind the ring: barriers, then a word for tensor memory's address and one for a count of stages.
__host__ __device__ constexpr int bar_bytes(int stages) { return (4 * stages + 6) * 8 + 8; }

// MMA descriptors.  Along the depth: as of the other tensor-core kernels.  Across it: boxes of 64 elements x
// 64 deep, 128 bytes an entry of depth; 8 of depth are 1024 bytes apart (stride), 64 elements a box (leading).
__device__ __forceinline__ uint64_t across_desc(uint32_t smem_addr)
{
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(BOX_BYTES >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
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

// A value that is the same in all lanes, kept in a register and known to be uniform.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// Whether the phase has completed, without waiting.
__device__ __forceinline__ uint32_t test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done;
}

// A bounded wait for a whole warp, with the same answer in all lanes, known to be uniform.  CLUSTER: what
// another CTA wrote before it arrived is visible.  The clock is read only after some polls: reading it
// takes longer than most waits.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned *err, unsigned code,
                                          unsigned long long limit_ns)
{
    uint64_t t0 = 0;
    for (uint32_t spin = 1;; ++spin) {
        uint32_t done;
        if constexpr (CLUSTER)
            asm volatile(
                "{\n"
                ".reg .pred p;\n"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                "selp.u32 %0, 1, 0, p;\n"
                "}\n"
                : "=r"(done)
                : "r"(bar), "r"(parity)
                : "memory");
        else
            done = tc::mbar_try_wait(bar, parity);
        if (__all_sync(0xFFFFFFFFu, done)) return true;
        if ((spin & 63u) == 0) {
            bool stop = *(volatile unsigned *)err != 0u;
            const uint64_t now = tc::global_timer();
            if (t0 == 0) t0 = now;
            if (!stop && now - t0 > limit_ns) {
                atomicOr(err, code);
                stop = true;
            }
            if (__any_sync(0xFFFFFFFFu, stop)) return false;
        }
    }
}

// Arrive on a barrier of another CTA of the cluster, without releasing writes to it: with
// .release.cluster the arrival waits for this thread's stores to global memory (3000 cycles a tile).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void store_remote(uint32_t cluster_addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// A tile: rows t0 .. t0 + valid of the output, columns from f0, group e, depth k0 .. k0 + depth;
// row_tile: its number among all tiles of rows.
struct Tile {
    int t0, valid, f0, e, k0, depth, row_tile;
};

// The tiles of a product, for each role (a warp) by itself.  Eight tiles of rows are swept along the
// columns together, so that the tiles in flight share operands in L2.  Each lane finds one of the CTA's
// next 32 tiles: found one by one they took every role 1400 cycles a tile, divisions for the most part.
// Pairs: the tiles that a last round has too few of are divided into 2 or 4 by rows, as long as there are pairs for
// them: a tile of 64 rows takes half the time of one of 256.  (4096 cubed, 28 tiles in the last round, 82.6 us to
// 79.1; 8192 x 11008 x 4096 with GELU, 8 of them, 417 to 409; shapes with none as before.)
struct Walk {
    const Args &p;
    const int *begin, *first;  // table: a group's first row, its first tile
    int tile_f, start, step, total, group;
    int whole, parts;  // tiles that are not divided; of a divided one
    Tile mine;

    __device__ Walk(const Args &args, const int *table, int columns, int first_tile, int tile_step)
        : p(args), begin(table), first(table + args.q.groups + 1), tile_f(columns), start(first_tile), step(tile_step), group(0)
    {
        if (p.q.ragged == RAGGED_ROWS)
            total = __shfl_sync(0xFFFFFFFFu, first[p.q.groups], 0);
        else
            total = p.tiles_t * p.tiles_f * (p.q.ragged == RAGGED_DEPTH ? p.q.groups : 1);
        whole = total;
        parts = 1;
        const int rest = total % step;
        // (Column sums have room for a tile's.)
        if (columns > TILE_F && rest != total && rest * 2 <= step && p.nt >= 64 && !p.q.partial) {
            parts = rest * 4 <= step && p.nt >= 128 ? 4 : 2;
            whole -= rest;
            total = whole + rest * parts;
        }
        mine = Tile{};
    }

    // Whether there is a j-th tile of this CTA, and what it is.  j: 0, 1, 2, ...
    __device__ __forceinline__ bool get(int j, Tile &o)
    {
        if (start + (long long)j * step >= total) return false;
        if (j % 32 == 0) mine = find((int)min(start + (long long)(j + (int)(threadIdx.x & 31)) * step, total - 1ll));
        // (Through shuffles, so that loops over a tile are known to be uniform: in others an MMA takes 128
        // cycles to issue, and 16 of depth of a 128 x 16 tile as long as of a 256 x 256 one.)
        int *const to = reinterpret_cast<int *>(&o);
        const int *const from = reinterpret_cast<const int *>(&mine);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Tile) / sizeof(int)); ++i) to[i] = __shfl_sync(0xFFFFFFFFu, from[i], j % 32);
        return true;
    }

    // Tile t; a lane asks for ever later ones.
    __device__ __forceinline__ Tile find(int t)
    {
        Tile o;
        int tiles_t = p.tiles_t, height_t = p.step, rows = p.q.M, row0 = 0, row_tile0 = 0, part = 0;
        const bool divided = t >= whole;
        if (divided) {
            part = (t - whole) % parts;
            t = whole + (t - whole) / parts;
        }
        o.e = 0;
        o.k0 = 0;
        o.depth = p.q.K;
        if (p.q.ragged == RAGGED_ROWS) {
            while (t >= first[group + 1]) ++group;
            o.e = group;
            tiles_t = (first[group + 1] - first[group]) / p.tiles_f;
            t -= first[group];
            row0 = begin[group];
            rows = begin[group + 1] - row0;
            height_t = min((int)(((unsigned)rows + tiles_t - 1) / tiles_t + 31) & ~31, p.nt);
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
        o.t0 = row0 + i * height_t;
        o.valid = min(height_t, rows - i * height_t);
        o.row_tile = row_tile0 + i;
        if (divided) {
            const int height_p = ((o.valid + parts - 1) / parts + 31) & ~31;
            o.t0 += part * height_p;
            o.valid = max(min(height_p, o.valid - part * height_p), 0);
        }
        if (p.q.alpha == 0.0f || o.valid == 0) o.depth = 0;
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
        int sum = p.q.ragged == RAGGED_ROWS ? (int)(((unsigned)rows + p.nt - 1) / p.nt) * p.tiles_f : 0;
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

// Elements [row c][this lane's column], c < rows, on their way to registers: loaded here, taken as
// floats later.  16-bit types, where pairs of columns are aligned: lanes 2i and 2i + 1 load both columns of
// a row each, and exchange them then.
template <int N>
struct Ahead {
    uint32_t raw[N];

    template <class T>
    __device__ __forceinline__ void load(const T *src, long long ld, int rows, bool in, bool pairs)
    {
        if constexpr (sizeof(T) == 2) {
            if (pairs) {
                const int odd = threadIdx.x & 1, last = in ? rows - odd : 0;
                src += odd ? ld - 1 : 0;
#pragma unroll
                for (int c = 0; c < N; c += 2, src += 2 * ld)
                    raw[c] = c < last ? *reinterpret_cast<const uint32_t *>(src) : 0u;
                return;
            }
        }
        const int last = in ? rows : 0;
#pragma unroll
        for (int c = 0; c < N; ++c, src += ld) {
            if constexpr (sizeof(T) == 2)
                raw[c] = c < last ? *reinterpret_cast<const uint16_t *>(src) : 0u;
            else
                raw[c] = c < last ? __float_as_uint(to_float(*src)) : 0u;
        }
    }

    template <class T>
    __device__ __forceinline__ void take(float (&v)[N], bool pairs) const
    {
        if constexpr (sizeof(T) == 2) {
            if (pairs) {
                const bool odd = threadIdx.x & 1;
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, raw[c], 1);
                    const uint32_t first = odd ? other >> 16 : raw[c], second = odd ? raw[c] >> 16 : other;
                    v[c] = from_bits<T>(first);
                    v[c + 1] = from_bits<T>(second);
                }
                return;
            }
        }
#pragma unroll
        for (int c = 0; c < N; ++c) {
            if constexpr (sizeof(T) == 2)
                v[c] = from_bits<T>(raw[c]);
            else
                v[c] = __uint_as_float(raw[c]);
        }
    }
};

// Store v to rows c < rows of this lane's column.  16-bit types, where pairs of columns are aligned:
// lanes 2i and 2i + 1 exchange their values of two rows, and each stores both columns of one.
template <class T, int N>
__device__ __forceinline__ void store_rows(T *out, long long ld, const float (&v)[N], int rows, bool in, bool pairs)
{
    if constexpr (sizeof(T) == 2) {
        if (pairs) {
            const int odd = threadIdx.x & 1, last = in ? rows - odd : 0;
            const uint32_t select = odd ? 0x3276u : 0x5410u;
            T *dst = out + (odd ? ld - 1 : 0);
#pragma unroll
            for (int c = 0; c < N; c += 2, dst += 2 * ld) {
                const uint32_t own = pack<T>(v[c], v[c + 1]), other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
                if (c < last) *reinterpret_cast<uint32_t *>(dst) = __byte_perm(own, other, select);
            }
            return;
        }
    }
    if (!in) return;
#pragma unroll
    for (int c = 0; c < N; ++c, out += ld)
        if (c < rows) *out = from_float<T>(v[c]);
}

// What the epilogue needs of the arguments, in registers: from the constant bank each of them would
// cost a chunk of rows 40 cycles and more (a chunk of 16 rows took 1400 cycles).
enum { WITH_Z = 16, WITH_R = 32, WITH_SUMS = 64, SLOPE = 128, Y_PAIRS = 256, Z_PAIRS = 512, R_PAIRS = 1024 };
// The kernel comes in three kinds, PLAIN (bias and activation), FORWARD (with Z or R) and GRADIENT (a slope or
// column sums): the code of a chunk is short enough then that jumps over what a call does not want cost
// little (1353 x 6488 x 72: 12.5 us in place of 10.3 where all were one).
enum Kind { PLAIN, FORWARD, GRADIENT };
template <Kind KIND>
struct Epilogue {
    float alpha, beta;
    int mode;  // act, and the above
    long long ldy, ldz, ldr;

    __device__ __forceinline__ explicit Epilogue(const Args &p)
    {
        const Product &q = p.q;
        alpha = __shfl_sync(0xFFFFFFFFu, q.alpha, 0);
        beta = __shfl_sync(0xFFFFFFFFu, q.beta, 0);
        ldy = __shfl_sync(0xFFFFFFFFu, q.ldy, 0);
        ldz = __shfl_sync(0xFFFFFFFFu, q.ldz, 0);
        ldr = __shfl_sync(0xFFFFFFFFu, q.ldr, 0);
        const int z = q.slope ? q.act != FGEMM_ACT_NONE : q.z != nullptr;
        mode = uniform(q.act | (z ? WITH_Z : 0) | (!q.slope && q.beta != 0.0f ? WITH_R : 0) | (q.partial ? WITH_SUMS : 0) |
                       (p.y_pairs ? Y_PAIRS : 0) | (p.z_pairs ? Z_PAIRS : 0) | (p.r_pairs ? R_PAIRS : 0));
    }
    __device__ __forceinline__ int act() const { return mode & 15; }
    __device__ __forceinline__ bool has(int what) const
    {
        if (what == SLOPE) return KIND == GRADIENT;
        if (KIND == PLAIN && what == WITH_Z) return false;
        if (KIND != FORWARD && what == WITH_R) return false;
        if (KIND != GRADIENT && what == WITH_SUMS) return false;
        return (mode & what) != 0;
    }

    // What finish_rows reads, Z for a slope or R.
    template <class T, class O, int N>
    __device__ __forceinline__ void load(Ahead<N> &ahead, const T *z, const O *r, int rows, bool in) const
    {
        if (has(SLOPE)) {
            if (has(WITH_Z)) ahead.load(z, ldz, rows, in, has(Z_PAIRS));
        } else if (has(WITH_R)) {
            ahead.load(r, ldr, rows, in, has(R_PAIRS));
        }
    }
};

// N sums of this lane's column to `rows` rows of it, the first at y (and z); ahead: what of Z or R goes in.
// Returns the sum of what Y holds of them, before its rounding.
template <class T, class O, Kind KIND, int N>
__device__ __forceinline__ float finish_rows(const Epilogue<KIND> &q, float (&v)[N], const Ahead<N> &ahead, O *y, T *z, float bias,
                                             int rows, bool in)
{
#pragma unroll
    for (int c = 0; c < N; c += 2) split(fma(two(v[c], v[c + 1]), both(q.alpha), both(bias)), v[c], v[c + 1]);
    const int act = q.act();
    if (q.has(SLOPE)) {
        if (q.has(WITH_Z)) {
            float x[N];
            ahead.template take<T>(x, q.has(Z_PAIRS));
            if (act == FGEMM_ACT_RELU) {
#pragma unroll
                for (int c = 0; c < N; ++c) v[c] = gate(v[c], x[c]);
            } else if (act == FGEMM_ACT_GELU) {
#pragma unroll
                for (int c = 0; c < N; c += 2) split(mul(two(v[c], v[c + 1]), gelu_slope(x[c], x[c + 1])), v[c], v[c + 1]);
            } else {
#pragma unroll
                for (int c = 0; c < N; ++c) v[c] *= silu_slope(x[c]);
            }
        }
    } else {
        if (q.has(WITH_Z)) store_rows(z, q.ldz, v, rows, in, q.has(Z_PAIRS));
        if (act == FGEMM_ACT_RELU) {
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] = relu(v[c]);
        } else if (act == FGEMM_ACT_GELU) {
#pragma unroll
            for (int c = 0; c < N; c += 2) gelu(v[c], v[c + 1]);
        } else if (act == FGEMM_ACT_SILU) {
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] = silu(v[c]);
        }
        if (q.has(WITH_R)) {
            float x[N];
            ahead.template take<O>(x, q.has(R_PAIRS));
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] = fmaf(q.beta, x[c], v[c]);
        }
    }
    store_rows(y, q.ldy, v, rows, in, q.has(Y_PAIRS));
    float sum = 0.0f;
    if (q.has(WITH_SUMS)) {
#pragma unroll
        for (int c = 0; c < N; ++c) sum += c < rows ? v[c] : 0.0f;
    }
    return sum;
}

// Zero rows `from` .. `to` (entries of depth, at most 15) of `boxes` boxes stored across the depth, by a warp.
__device__ __forceinline__ void zero_depth(uint32_t base, int boxes, int from, int to, int lane)
{
    for (int b = 0; b < boxes; ++b)
        for (int row = from + (lane >> 3); row < to; row += 4)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + b * BOX_BYTES + row * 128 + (lane & 7) * 16), "r"(0)
                         : "memory");
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

// 16 bytes to shared memory, on their way when this returns.
__device__ __forceinline__ void copy_16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// 16 sums of each lane from tensor memory.
__device__ __forceinline__ void load_sums(uint32_t taddr, bool products, float (&v)[CHUNK])
{
    static_assert(CHUNK == 16, "columns");
    if (!products) {
#pragma unroll
        for (int c = 0; c < CHUNK; ++c) v[c] = 0.0f;
        return;
    }
    uint32_t r[CHUNK];
    mx::tmem_load(taddr, r);
#pragma unroll
    for (int c = 0; c < CHUNK; ++c) v[c] = __uint_as_float(r[c]);
}

// The way back.
__device__ __forceinline__ void store_sums(uint32_t taddr, const float (&v)[CHUNK])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

// In CTA 0 of a pair whose producer has given up behind g stages: those up to `asked`, which CTA 1 has asked for, are
// expected by the barriers that count them, too.
static __device__ __noinline__ void follow(const Args &p, const int *table, int first_tile, int tile_step, uint32_t full0, int g,
                                           int asked)
{
    const int stage_depth = p.blocks * DEPTH;
    const int x_step = p.x_across ? 64 : p.x_box;
    const bool fix_depth = p.q.ragged == RAGGED_DEPTH;
    Walk walk(p, table, 2 * TILE_F, first_tile, tile_step);
    Tile o{};
    for (int tile = 0, at = 0; at < asked && walk.get(tile, o); ++tile) {
        const int n = (int)(((unsigned)o.depth + stage_depth - 1) / stage_depth), own = ((o.valid + 31) & ~31) / 2;
        const uint32_t bytes = W_BYTES + (own + x_step - 1) / x_step * x_step * 128;
        for (int k = 0; k < n && at < asked; ++k, ++at) {
            if (at < g) continue;
            const int left = o.depth - (!fix_depth ? k : k == 0 ? n - 1 : k - 1) * stage_depth;
            const uint32_t full = full0 + 8 * (at % p.stages);
            if ((threadIdx.x & 31) == 0) {
                if (fix_depth && left < stage_depth && (left & 15) != 0)
                    tc::mbar_arrive(full);  // (the end of a group: counted by CTA 1 itself)
                else
                    tc::mbar_arrive_expect_tx(full, stage_depth > DEPTH && left > DEPTH ? 2 * bytes : bytes);
            }
        }
        __syncwarp();
    }
}

// PAIR: two CTAs work on 256 columns of Y with cta_group::2; each holds its own 128 columns of
// op(B) and half of the tile's rows of op(A).  CTA 0 issues for both; its `full` barriers count what
// arrives in either.  Else the `ranks` CTAs of a cluster divide the depth of one tile, or (ranks 1) a CTA
// walks whole tiles.
// LONG: the accumulators take a depth of LONG_DEPTH (768) at a time, and the epilogue's warps add these
// sums up in their registers.  The tensor core cuts where FP32 addition rounds: over a depth of
// 2048, sums come out 2.1e-6 off (2-norm, random operands), of 768 at a time 0.6e-6, which counts where
// they are kept in FP32 and, of a depth beyond one_go(), in 16 bits.  (4096 x 11008 of a depth of 2048: 122 us
// in turns, 119 in one go.)
template <bool PAIR, class T, class O, bool LONG, Kind KIND>
__global__ void __launch_bounds__(threads_of(PAIR), 1) gemm16_kernel(const __grid_constant__ Args p, unsigned *err)
{
    constexpr int THREADS = threads_of(PAIR);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, bar_offset = S * p.stage_bytes;
    const uint32_t sbase = tc::cvta_smem(smem), bars = sbase + bar_offset;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    // A pair's stages that a group ends in: what each CTA brings is counted by its own `tail`, and mended.
    auto fixed_bar = [&](int s) { return bars + 8u * (2 * S + s); };
    auto tail_bar = [&](int s) { return bars + 8u * (3 * S + s); };
    auto acc_full_bar = [&](int a) { return bars + 8u * (4 * S + a); };
    auto acc_free_bar = [&](int a) { return bars + 8u * (4 * S + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (4 * S + 4), asked_bar = drain_bar + 8;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + bar_offset + 8 * (4 * S + 6));
    const uint32_t asked_slot = asked_bar + 12;  // of CTA 0 of a pair: the stages that CTA 1 has asked for
    int *const table = reinterpret_cast<int *>(smem + p.table);

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int ctas = __shfl_sync(0xFFFFFFFFu, (int)cluster.num_blocks(), 0), cta = __shfl_sync(0xFFFFFFFFu, (int)cluster.block_rank(), 0);
    // Which part of the depth, or which half of a pair (whose CTA 0 leads).
    const int ranks = PAIR ? 1 : ctas, rank = PAIR ? 0 : cta, half = PAIR ? cta : 0;
    const unsigned long long lim = p.wait_limit_ns;
    const bool split = !PAIR && ranks > 1;

    if (warp == 0 && lane == 0) {
        mx::prefetch_map(&p.w);
        mx::prefetch_map(&p.x);
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(full_bar(s), 1);
            tc::mbar_init(empty_bar(s), 1);
            tc::mbar_init(fixed_bar(s), 2);
            tc::mbar_init(tail_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(acc_full_bar(a), 1);
            tc::mbar_init(acc_free_bar(a), (PAIR ? 2 : 1) * 4 * SETS);
        }
        tc::mbar_init(drain_bar, 1);
        tc::mbar_init(asked_bar, 1);
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
    tc::tc_fence_before();
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);

    // The first tiles are found, where the arguments say which they are, while the kernel before this one
    // ends, and each role waits for that when it is ready to go.
    constexpr int COLUMNS = PAIR ? 2 * TILE_F : TILE_F;
    const int first_tile = (int)blockIdx.x / ctas, tile_step = (int)gridDim.x / ctas;
    if (p.q.ragged != RAGGED_NONE) {
        after_previous_kernel();
        if (warp == 2) make_table(p, table, lane);
        __syncthreads();
    }
    Walk walk(p, table, COLUMNS, first_tile, tile_step);
    Tile first{};
    const bool any = walk.get(0, first);  // (else there is nothing for this CTA, or its cluster)
    const bool waits = p.q.ragged == RAGGED_NONE;
    const int stage_depth = uniform(p.blocks) * DEPTH;
    const bool fix_depth = p.q.ragged == RAGGED_DEPTH;
    // A tile's stages that are this CTA's.
    auto stages_of = [&](const Tile &o, int &from) {
        const int all = (int)(((unsigned)o.depth + stage_depth - 1) >> (stage_depth == DEPTH ? 6 : 7));
        from = 0;
        if (!split) return all;
        from = (int)((long long)all * rank / ranks);
        return (int)((long long)all * (rank + 1) / ranks) - from;
    };
    // MMA columns of a tile, and the rows of op(A) that this CTA brings for them.
    auto mma_cols = [&](const Tile &o) { return PAIR ? (o.valid + 31) & ~31 : (o.valid + 15) & ~15; };
    // The k-th of a tile's n stages.  Where depths are ragged the last one comes first: it may have to be
    // mended, while the tensor core is still at the tile before.
    auto order = [&](int k, int n) { return !fix_depth ? k : k == 0 ? n - 1 : k - 1; };
    // Whether a stage with `left` of its depth to come ends inside the MMA's 16.
    auto wants_fix = [&](int left) { return fix_depth && left < stage_depth && (left & 15) != 0; };
    // That end of a stage becomes 0, in this CTA's part of both operands (x_boxes of op(A)).
    auto fix = [&](uint32_t at, int left, int x_boxes) {
        const uint32_t block = at + (left / DEPTH) * p.block_bytes;
        const int first_row = left % DEPTH, to = (first_row + 15) & ~15;
        zero_depth(block, 2, first_row, to, lane);
        zero_depth(block + W_BYTES, x_boxes, first_row, to, lane);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor core reads them
        __syncwarp();
    };

    if (warp == 0) {
        // ---- producer (one in each CTA): the whole warp walks along, one lane issues ----
        // What the loop needs of the arguments is in registers, and the next barrier is looked at before
        // this stage's copies are issued: the loop is a chain of short latencies.
        const int withhold = uniform(p.withhold), w_across = uniform(p.w_across), x_across = uniform(p.x_across);
        const uint32_t stage_bytes = uniform(p.stage_bytes), block_bytes = uniform(p.block_bytes);
        const uint32_t full0 = full_bar(0), empty0 = empty_bar(0), lead0 = PAIR ? mx::map_to_rank(full0, 0) : full0;
        const int x_step = x_across ? 64 : uniform(p.x_box);
        const uint32_t box_bytes = (uint32_t)x_step * 128;
        // From one box of op(A) to the next.
        const int x_d0 = x_across ? x_step : 0, x_d1 = x_across ? 0 : x_step;
        Slot at;
        uint32_t place = sbase;  // of the stage
        int g = 0;
        bool ok = true, ready = true;
        uint32_t tail_phase = 0, tail_used = 0;  // of the tail barriers
        Tile o = first;
        int from, n = stages_of(o, from);
        if (waits) after_previous_kernel();
        bool more = any;
        for (int tile = 1; ok && more; ++tile) {
            const int cols = mma_cols(o), own = PAIR ? cols / 2 : cols;
            const int boxes = (own + x_step - 1) / x_step, e = fix_depth ? 0 : o.e;
            const uint32_t bytes = W_BYTES + boxes * box_bytes;
            const int f = o.f0 + TILE_F * half, x0 = o.t0 + own * half;
            for (int k = 0; k < n; ++k, ++g) {
                const int skip = (from + order(k, n)) * stage_depth, depth = o.k0 + skip, left = o.depth - skip;
                ok = (ready || warp_wait(empty0 + 8 * at.s, at.phase ^ 1, err, tc::ERR_PRODUCER, lim)) &&
                     (g != withhold || half == 1);  // (testing: as if this copy never arrived)
                if (!ok) break;
                const bool tail = PAIR && wants_fix(left);
                const uint32_t here = place, full = full0 + 8 * at.s, lead = lead0 + 8 * at.s;
                const uint32_t bar = tail ? tail_bar(at.s) : full;
                const bool two = stage_depth > DEPTH && left > DEPTH;
                if (tail) {
                    tail_used |= 1u << at.s;
                    tail_phase ^= 1u << at.s;
                }
                at.next(S);
                place = at.s == 0 ? sbase : place + stage_bytes;
                const uint32_t next = test_wait(empty0 + 8 * at.s, at.phase ^ 1);
                if (mx::elect_one()) {
                    if (!PAIR || tail)
                        tc::mbar_arrive_expect_tx(bar, two ? 2 * bytes : bytes);
                    else if (half == 0)
                        tc::mbar_arrive_expect_tx(bar, two ? 4 * bytes : 2 * bytes);
                    if (tail && half == 0) tc::mbar_arrive(full);  // (this use of it passes)
#pragma unroll
                    for (int block = 0; block < 2; ++block) {
                        if (block == 1 && !two) break;
                        const uint32_t w_at = here + block * block_bytes, x_at = w_at + W_BYTES;
                        const int d = depth + block * DEPTH;
                        const int w_c0 = w_across ? f : d, w_c1 = w_across ? d : f;
                        const int x_c0 = x_across ? x0 : d, x_c1 = x_across ? d : x0;
                        if (!PAIR || tail) {
                            tc::tma_load_3d(w_at, &p.w, bar, w_c0, w_c1, e);
                            if (w_across) tc::tma_load_3d(w_at + BOX_BYTES, &p.w, bar, w_c0 + 64, w_c1, e);
#pragma unroll
                            for (int b = 0; b < MAX_BOXES; ++b)
                                if (b < boxes) mx::tma_load_2d(x_at + b * box_bytes, &p.x, bar, x_c0 + b * x_d0, x_c1 + b * x_d1);
                        } else {
                            mx::pair_load_3d(w_at, &p.w, lead, w_c0, w_c1, e);
                            if (w_across) mx::pair_load_3d(w_at + BOX_BYTES, &p.w, lead, w_c0 + 64, w_c1, e);
#pragma unroll
                            for (int b = 0; b < MAX_BOXES; ++b)
                                if (b < boxes) mx::pair_load_2d(x_at + b * box_bytes, &p.x, lead, x_c0 + b * x_d0, x_c1 + b * x_d1);
                        }
                    }
                }
                __syncwarp();
                ready = __all_sync(0xFFFFFFFFu, next);
            }
            more = walk.get(tile, o);
            n = stages_of(o, from);
        }
        if constexpr (PAIR) {
            if (half == 1) {
                if (lane == 0) mx::tell_asked(asked_slot, asked_bar, g);
            } else {
                const int asked = mx::asked_by_other(asked_slot, asked_bar, g, ok, err, lim);
                if (asked > g) follow(p, table, first_tile, tile_step, full0, g, asked);
                g = asked;
            }
        }
        // Never leave with copies in flight into either CTA's shared memory.
        if (half == 0)
            for (int k = g - S < 0 ? 0 : g - S; k < g; ++k)
                tc::mbar_wait(full_bar(k % S), (k / S) & 1, err, tc::ERR_DRAIN, lim, false);
        for (int s = 0; s < S; ++s)
            if (tail_used >> s & 1) tc::mbar_wait(tail_bar(s), (tail_phase >> s & 1) ^ 1, err, tc::ERR_DRAIN, lim, false);
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA (of a pair: by CTA 0 for both) ----
        Slot at;
        bool ok = true;
        uint32_t fix_phase = 0;
        if (waits) after_previous_kernel();
        if (half == 0) {
            const uint32_t fmt = p.q.type == FGEMM_BF16 ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t idesc0 = uniform((int)((1u << 4) | fmt | ((uint32_t)p.w_across << 15) | ((uint32_t)p.x_across << 16) |
                                                  ((uint32_t)(COLUMNS >> 4) << 24)));
            // 16 of depth: 32 bytes along it, 16 rows of 128 bytes across it.
            const uint32_t wi = uniform(p.w_across ? 128 : 2), xi = uniform(p.x_across ? 128 : 2);
            const uint32_t stage_bytes = uniform(p.stage_bytes), acc_step = uniform(p.acc_step);
            const uint32_t block_step = uniform(p.block_bytes >> 4);
            const int long_stages = LONG_DEPTH / stage_depth;
            const uint32_t full0 = full_bar(0), empty0 = empty_bar(0);
            // (Addresses count modulo 256 KB: above are the bits that tell the CTAs of a cluster apart.)
            const uint64_t w_desc = p.w_across ? across_desc(0) : tc::kmajor_sw128_desc(0);
            const uint64_t x_desc = p.x_across ? across_desc(0) : tc::kmajor_sw128_desc(0);
            uint32_t place = sbase;
            int j = 0;
            bool ready = false;
            Tile o = first;
            bool more = any;
            for (int tile = 1; ok && more; more = walk.get(tile++, o)) {
                int from;
                const int n = stages_of(o, from), cols = mma_cols(o);
                const uint32_t idesc = idesc0 | ((uint32_t)(cols >> 3) << 17);
                uint32_t d = 0;
                int since = 0;  // stages that this accumulator holds
                for (int k = 0; k < n; ++k) {
                    const int left = o.depth - (from + order(k, n)) * stage_depth;
                    const int acc = j & 1;
                    if (since == 0) {  // the sums before the last ones have been read
                        ok = j < 2 || warp_wait(acc_free_bar(acc), ((j >> 1) - 1) & 1, err, tc::ERR_MMA_WAIT, lim);
                        if (!ok) break;
                        d = tmem + (uint32_t)acc * acc_step;
                    }
                    ok = ready || warp_wait(full0 + 8 * at.s, at.phase, err, tc::ERR_MMA_WAIT, lim);
                    if (!ok) break;
                    const bool last = k + 1 == n || (LONG && since + 1 == long_stages);
                    const int steps = (min(stage_depth, left) + 15) >> 4;
                    if (wants_fix(left)) {
                        if constexpr (PAIR) {  // the menders of both CTAs have been there
                            ok = warp_wait<true>(fixed_bar(at.s), fix_phase >> at.s & 1, err, tc::ERR_MMA_WAIT, lim);
                            fix_phase ^= 1u << at.s;
                            if (!ok) break;
                        } else {
                            fix(place, left, (cols + 63) / 64);
                        }
                    }
                    const uint64_t wd = w_desc + ((place >> 4) & 0x3FFFu), xd = x_desc + (((place + W_BYTES) >> 4) & 0x3FFFu);
                    const uint32_t empty = empty0 + 8 * at.s;
                    at.next(S);
                    place = at.s == 0 ? sbase : place + stage_bytes;
                    const uint32_t next = test_wait(full0 + 8 * at.s, at.phase);
                    tc::tc_fence_after();
                    if (mx::elect_one()) {
#pragma unroll
                        for (int i = 0; i < 2 * DEPTH / 16; ++i) {
                            const uint32_t block = i < DEPTH / 16 ? 0 : block_step;
                            if (i < steps)
                                mma<PAIR>(d, wd + (block + wi * (i % (DEPTH / 16))), xd + (block + xi * (i % (DEPTH / 16))), idesc,
                                          since > 0 || i > 0);
                        }
                        if constexpr (PAIR) {
                            mx::pair_commit(empty);
                            if (last) mx::pair_commit(acc_full_bar(acc));
                        } else {
                            tc::umma_commit(empty);
                            if (last) tc::umma_commit(acc_full_bar(acc));
                        }
                    }
                    __syncwarp();
                    ready = __all_sync(0xFFFFFFFFu, next);
                    since = last ? 0 : since + 1;
                    j += last;
                }
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
        }
        __syncwarp();
    } else if (PAIR && warp == 2 + 4 * SETS) {
        // ---- mender (one in each CTA of a pair): overwrites its CTA's part of the stages that a group ends in,
        // as soon as they are there ----
        if (fix_depth) {
            Slot at;
            uint32_t phases = 0;
            Tile o = first;
            bool more = any, ok = true;
            for (int tile = 1; ok && more; more = walk.get(tile++, o)) {
                int from;
                const int n = stages_of(o, from), left = o.depth - (from + order(0, n)) * stage_depth;
                if (n > 0 && wants_fix(left)) {
                    ok = warp_wait(tail_bar(at.s), phases >> at.s & 1, err, tc::ERR_MMA_WAIT, lim);
                    if (!ok) break;
                    phases ^= 1u << at.s;
                    fix(sbase + at.s * p.stage_bytes, left, (mma_cols(o) / 2 + 63) / 64);
                    if (lane == 0) mx::arrive_at(mx::map_to_rank(fixed_bar(at.s), 0));
                }
                for (int k = 0; k < n; ++k) at.next(S);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: sets of four warps; the sets take the chunks of rows in turn ----
        const int q = warp & 3, set = (warp - 2) >> 2;
        auto give_back = [&](int acc) {  // this warp has read an accumulator
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    arrive_remote(mx::map_to_rank(acc_free_bar(acc), 0));
                else
                    tc::mbar_arrive(acc_free_bar(acc));
            }
        };
        const Epilogue<KIND> epi(p);
        const float *const biases = p.q.bias;
        const bool staged = KIND == GRADIENT && PAIR && uniform(p.z_ring) != 0;
        const uint32_t ring = sbase + p.z_ring + (warp - 2) * (Z_SLOTS * Z_SLOT_BYTES);
        const int N = uniform(p.q.N), acc_step = uniform(p.acc_step);
        const long long stride_y = __shfl_sync(0xFFFFFFFFu, p.q.stride_y, 0);
        int j = 0;
        Tile o = first;
        if (waits) after_previous_kernel();
        bool more = any;
        for (int tile = 1; more; more = walk.get(tile++, o)) {
            int from;
            const int stages = stages_of(o, from), n = o.f0 + TILE_F * half + 32 * q + lane;
            const int turns = LONG ? (int)(((unsigned)(stages * stage_depth) + LONG_DEPTH - 1) / LONG_DEPTH) : stages > 0;
            const bool in = n < N;
            // (on its way during the wait)
            const float bias = biases && in ? biases[(long long)o.e * N + n] : 0.0f;
            O *const y = static_cast<O *>(p.q.y) + o.e * stride_y + o.t0 * epi.ldy + n;
            T *const z = static_cast<T *>(p.q.z) + o.t0 * epi.ldz + n;
            const O *const r_at = static_cast<const O *>(p.q.r) + o.e * stride_y + o.t0 * epi.ldr + n;
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
            float sum = 0.0f;
            const int share = (o.valid + ranks - 1) / ranks;  // rows that a rank of the cluster joins
            auto load_ahead = [&](Ahead<CHUNK> &ahead, int c0) {
                if (c0 < o.valid && !split) epi.load(ahead, z + c0 * epi.ldz, r_at + c0 * epi.ldr, o.valid - c0, in);
            };
            auto finish = [&](float (&v)[CHUNK], const Ahead<CHUNK> &ahead, int c0) {
                if (split) {  // to the rank that joins the row: by rank, row, 128 columns
                    int to = c0 / share, row = c0 - to * share;
                    const uint32_t mine = sbase + p.join + (uint32_t)(rank * share * TILE_F + 32 * q + lane) * 4;
                    uint32_t at = mx::map_to_rank(mine, to);
#pragma unroll
                    for (int c = 0; c < CHUNK; ++c) {
                        if (c0 + c < o.valid) store_remote(at + (uint32_t)row * TILE_F * 4, v[c]);
                        if (++row == share) {
                            row = 0;
                            to = min(to + 1, ranks - 1);
                            at = mx::map_to_rank(mine, to);
                        }
                    }
                } else {
                    sum += finish_rows<T, O, KIND>(epi, v, ahead, y + c0 * epi.ldy, z + c0 * epi.ldz, bias, o.valid - c0, in);
                }
            };
            // What of Z or R the first chunk takes comes during the wait, each next chunk's during the one before
            // (the gradient of 8192 x 4096, depth 2048, through GELU: 174 us without, 119 with).
            Ahead<CHUNK> ahead;
            if (!LONG && !staged) load_ahead(ahead, CHUNK * set);
            // Or (pairs, rows of Z on 16 bytes) four chunks are on their way through shared memory: a chunk takes less
            // time than memory does to answer, which the tensor core waits for where a tile's last sums keep it from the
            // turn after the next one.  (Groups of 512 x 4096, depth 2048, with column sums: through ReLU 123 us, by
            // registers 137 to 145; GELU 141 and 146; SiLU 136 and 141 to 146.  Without sums no turns, and 110 either way.)
            auto send_for = [&](int c0) {
                const int row = c0 + (lane >> 2), c = 8 * (lane & 3) - lane;
                const T *const src = z + row * epi.ldz + c;
                const uint32_t dst = ring + (c0 / (SETS * CHUNK) % Z_SLOTS) * Z_SLOT_BYTES + lane * 16;
                if (n + c < N && row < o.valid) copy_16(dst, src);
                if (n + c < N && row + 8 < o.valid) copy_16(dst + Z_SLOT_BYTES / 2, src + 8 * epi.ldz);
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            if (staged) {
                __syncwarp();  // (the tile before has been read)
#pragma unroll
                for (int i = 0; i < Z_SLOTS; ++i) send_for(CHUNK * (SETS * i + set));
            }
            bool ok = true;
            if constexpr (LONG) {
                // All turns but the last are added up in registers, and then with the last one where its
                // sums are, in tensor memory.
                if (turns > 1) {
                    constexpr int MOST = (PAIR ? 256 : 64) / CHUNK / SETS;
                    float sums[MOST][CHUNK];
#pragma unroll
                    for (int i = 0; i < MOST; ++i)
#pragma unroll
                        for (int c = 0; c < CHUNK; ++c) sums[i][c] = 0.0f;
#pragma unroll 1
                    for (int turn = 0; ok && turn < turns; ++turn) {
                        ok = warp_wait(acc_full_bar(j & 1), (j >> 1) & 1, err, tc::ERR_EPILOGUE, lim);
                        if (!ok) break;
                        tc::tc_fence_after();
                        const bool last = turn + 1 == turns;
#pragma unroll
                        for (int i = 0; i < MOST; ++i) {
                            const int c0 = CHUNK * (SETS * i + set);
                            if (c0 < o.valid) {
                                const uint32_t at = lanes + (uint32_t)((j & 1) * acc_step + c0);
                                float v[CHUNK];
                                load_sums(at, true, v);
#pragma unroll
                                for (int c = 0; c < CHUNK; ++c) sums[i][c] += v[c];
                                if (last) store_sums(at, sums[i]);
                            }
                        }
                        if (!last) {
                            give_back(j & 1);
                            ++j;
                        }
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
            }
            if (LONG && !staged) load_ahead(ahead, CHUNK * set);
            // (A wait for a whole tile's depth, of which a stage takes 0.3 us: 2^31 rows take 5 s.)
            if (!LONG || turns == 1)
                ok = turns == 0 || warp_wait(acc_full_bar(j & 1), (j >> 1) & 1, err, tc::ERR_EPILOGUE, lim + 1024ull * stages);
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int c0 = CHUNK * set; c0 < o.valid; c0 += SETS * CHUNK) {
                float v[CHUNK];
                load_sums(lanes + (uint32_t)((j & 1) * acc_step + c0), turns > 0, v);
                if (staged) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(Z_SLOTS - 1) : "memory");
                    __syncwarp();
                    const uint8_t *const slot = smem + (ring - sbase) + (c0 / (SETS * CHUNK) % Z_SLOTS) * Z_SLOT_BYTES;
                    Ahead<CHUNK> now;
                    now.load(reinterpret_cast<const T *>(slot) + lane, 32, o.valid - c0, in, true);
                    __syncwarp();
                    send_for(c0 + Z_SLOTS * SETS * CHUNK);
                    finish(v, now, c0);
                } else {
                    const Ahead<CHUNK> now = ahead;
                    load_ahead(ahead, c0 + SETS * CHUNK);
                    finish(v, now, c0);
                }
            }
            if (turns > 0) {
                give_back(j & 1);
                ++j;
            }
            const long long row = (long long)SETS * o.row_tile + set;
            if (KIND == GRADIENT && p.q.partial && in && row < p.q.partials) p.q.partial[row * p.q.N + n] = sum;
        }
        if (staged) asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }

    if (split) {
        // Every CTA of the cluster has been sent its share of the tile's rows by all ranks (its own room
        // for them is apart from the stages, which it may still use meanwhile) and adds them up, in rank
        // order.  (A rank that gave up sends nothing; the error word says that Y is undefined.)
        const Epilogue<KIND> epi(p);
        float bias = 0.0f;
        const int q = warp & 3, set = (warp - 2) >> 2, n = first.f0 + TILE_F * half + 32 * q + lane;
        if (warp >= 2 && any && p.q.bias && n < p.q.N) bias = p.q.bias[(long long)first.e * p.q.N + n];
        cluster.sync();
        if (warp >= 2 && any) {
            const int share = (first.valid + ranks - 1) / ranks, rows = min(share, first.valid - rank * share);
            const float *const part = reinterpret_cast<const float *>(smem + p.join) + 32 * q + lane;
            constexpr int FEW = 8;
#pragma unroll 1
            for (int c0 = FEW * set; c0 < rows; c0 += SETS * FEW) {
                const long long row = first.t0 + rank * share + c0, base = first.e * p.q.stride_y + n;
                T *const z = static_cast<T *>(p.q.z) + n + row * epi.ldz;
                Ahead<FEW> ahead;
                epi.load(ahead, z, static_cast<const O *>(p.q.r) + base + row * epi.ldr, rows - c0, n < p.q.N);
                float v[FEW];
#pragma unroll
                for (int c = 0; c < FEW; ++c) v[c] = 0.0f;
#pragma unroll 2
                for (int r = 0; r < ranks; ++r) {
#pragma unroll
                    for (int c = 0; c < FEW; ++c)
                        if (c0 + c < rows) v[c] += part[(r * share + c0 + c) * TILE_F];
                }
                finish_rows<T, O, KIND>(epi, v, ahead, static_cast<O *>(p.q.y) + base + row * epi.ldy, z, bias, rows - c0, n < p.q.N);
            }
        }
    }

    if (KIND == GRADIENT && p.q.partial_start && blockIdx.x == 0) {
        for (int e = threadIdx.x; e <= p.q.groups; e += THREADS)
            p.q.partial_start[e] = SETS * (p.q.ragged == RAGGED_ROWS ? walk.first[e] / p.tiles_f : p.tiles_t * e);
    }

    // No CTA of a pair leaves while the other may still reach its memory.  (What ranks send each other has
    // arrived.)
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
