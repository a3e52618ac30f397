// gemm16_launch.cuh -- host side of the 16-bit products: tensor maps and the launch of one kernel
// instance.  Each operand type's instances are compiled in a unit of their own.
#pragma once

#include <atomic>
#include <cstring>

#include "ctx_id.h"
#include "fgemm_internal.h"
#include "gemm16_tc.cuh"
#include "mxfp4_launch.h"
#include "tc_host.h"

namespace fgemm {
namespace h16 {

// A matrix (or `batch` of them) of rows x cols 16-bit elements as a tensor map with boxes of 64
// elements (the 128-byte swizzle's row) x box_rows; beyond the matrix it reads 0.  dims: 2 or 3.
static bool make_map(CUtensorMap *map, const void *x, bool bf16, int dims, long long rows, long long cols, long long ld,
                     long long batch, long long stride, int box_rows)
{
    const auto encode = tc_encode_fn();
    if (!encode) return false;
    const cuuint64_t size[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    // (One row or one matrix: the stride is not used, but has to be a multiple of 16 bytes.)
    const cuuint64_t pitch = rows > 1 ? (cuuint64_t)ld * 2 : ((cuuint64_t)cols * 2 + 15) / 16 * 16;
    const cuuint64_t strides[2] = {pitch, batch > 1 ? (cuuint64_t)stride * 2 : pitch};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims,
                  const_cast<void *>(x), size, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a launch needs besides its arguments: the error word, the SM count, and the kernel opted in to
// its shared memory, once per context (`Kernel` keeps instances' records apart).
constexpr int MOST_SMEM = 227 * 1024;
template <class Kernel, Kernel kernel>
static bool prepare(unsigned **err, int *sms)
{
    static std::atomic<unsigned long long> ready_ctx[64];
    int dev = 0;
    *err = tc_error_word();
    if (!*err || cudaGetDevice(&dev) != cudaSuccess || device_sm_count(sms) != 0) return false;
    std::atomic<unsigned long long> &ready = ready_ctx[dev & 63];
    const unsigned long long ctx = current_context_id();
    if (ctx != 0 && ready.load(std::memory_order_acquire) == ctx) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_SMEM) != cudaSuccess) return false;
    ready.store(current_context_id(), std::memory_order_release);
    return true;
}

static bool paired(const void *p, long long ld, fgemm_dtype t) { return t != FGEMM_F32 && reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0; }

template <bool PAIR, class T, class O, bool LONG, Kind KIND>
static fgemm_status launch_instance(const Product &q, const Plan &plan, cudaStream_t stream)
{
    constexpr auto kernel = &gemm16_kernel<PAIR, T, O, LONG, KIND>;
    unsigned *err = nullptr;
    int sms = 0;
    if (!prepare<decltype(kernel), kernel>(&err, &sms)) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    constexpr int columns = PAIR ? 2 * TILE_F : TILE_F;
    const int ctas = PAIR ? 2 : plan.ranks;
    if (ctas < 1 || ctas > 8 || (LONG && !PAIR && plan.nt > 64)) return FGEMM_ERR_NOT_SUPPORTED;
    Args p;
    std::memset(&p, 0, sizeof(p));
    p.q = q;
    p.w_across = !q.tb;
    p.x_across = q.ta;
    p.nt = plan.nt;
    const long long row_tiles = ((long long)q.M + p.nt - 1) / p.nt, tiles_f = ((long long)q.N + columns - 1) / columns;
    // Tiles of one product are of like sizes: 4100 rows by 256 are 17 of 256 (the last of 4), or of 242.
    const long long even = ((long long)q.M + row_tiles - 1) / row_tiles;
    p.step = (int)((even + 31) / 32 * 32 < p.nt ? (even + 31) / 32 * 32 : p.nt);
    if (q.ragged != RAGGED_ROWS) p.nt = p.step;
    long long tiles = row_tiles * tiles_f;
    if (q.ragged == RAGGED_DEPTH) tiles *= q.groups;
    if (q.ragged == RAGGED_ROWS) tiles = (row_tiles + (q.groups < q.M ? q.groups : q.M)) * tiles_f;  // at most
    if (tiles * ctas > 0x7FFFFFFF) return FGEMM_ERR_NOT_SUPPORTED;
    p.tiles_t = (int)row_tiles;
    p.tiles_f = (int)tiles_f;
    const int own = PAIR ? p.nt / 2 : p.nt;  // rows of op(A) that a CTA brings
    // Boxes: a whole tile's where all tiles are alike, else half of it, so that a short tile brings little more.  (As 64 rows
    // they bring 128 for 96: groups of 500 x 4096, depth 4096, 59 us in place of 52.)
    p.x_box = q.ragged == RAGGED_ROWS && own > 64 ? own / 2 : own;
    const int x_bytes = q.ta ? (own + 63) / 64 * BOX_BYTES : (own + p.x_box - 1) / p.x_box * p.x_box * 128;
    p.block_bytes = (W_BYTES + x_bytes + 1023) / 1024 * 1024;
    const int table_bytes = q.ragged == RAGGED_NONE ? 0 : 2 * 4 * (q.groups + 1);
    const int join_bytes = !PAIR && plan.ranks > 1 ? (p.nt + plan.ranks) * TILE_F * 4 : 0;  // (shares are rounded up)
    const int room = MOST_SMEM - 1024 - table_bytes - join_bytes - bar_bytes(MAX_STAGES) - 40;
    p.blocks = room >= 6 * p.block_bytes ? 2 : 1;
    p.stage_bytes = p.blocks * p.block_bytes;
    p.stages = room / p.stage_bytes < MAX_STAGES ? room / p.stage_bytes : MAX_STAGES;
    // Rings of Z where they cost no stage.  (Groups of 500 x 4096, depth 4096, 192 rows a tile, through ReLU: 56.5 us with four stages,
    // 62 with three and rings; of 128 x 2048, depth 1024: 72 without rings, 65 with them.)
    const int z_bytes = 4 * SETS * Z_SLOTS * Z_SLOT_BYTES;
    const bool z_ring = PAIR && KIND == GRADIENT && q.act != FGEMM_ACT_NONE && q.N % 8 == 0 && q.ldz % 8 == 0 &&
                        reinterpret_cast<uintptr_t>(q.z) % 16 == 0 && room - z_bytes >= p.stages * p.stage_bytes;
    if (p.stages < 2) return FGEMM_ERR_NOT_SUPPORTED;
    p.table = p.stages * p.stage_bytes + (bar_bytes(p.stages) + 15) / 16 * 16;
    p.join = p.table + (table_bytes + 15) / 16 * 16;
    p.z_ring = z_ring ? (p.join + join_bytes + 15) / 16 * 16 : 0;
    const int smem = 1024 + (z_ring ? p.z_ring + z_bytes : p.join + join_bytes);
    p.acc_step = PAIR ? 256 : p.nt;
    p.tmem_cols = 32;
    while (p.tmem_cols < 2 * p.acc_step) p.tmem_cols *= 2;
    if (p.tmem_cols > 512) return FGEMM_ERR_NOT_SUPPORTED;
    p.y_pairs = paired(q.y, q.ldy, q.out_type) && q.stride_y % 2 == 0 && q.N % 2 == 0;
    p.z_pairs = paired(q.z, q.ldz, q.type) && q.N % 2 == 0;
    p.r_pairs = paired(q.r, q.ldr, q.out_type) && q.stride_y % 2 == 0 && q.N % 2 == 0;
    p.wait_limit_ns = tc_wait_limit_ns();
    p.withhold = tc_withheld_k_block();
    if (q.K > 0 && q.alpha != 0.0f) {
        const bool bf16 = q.type == FGEMM_BF16;
        const long long batch = q.ragged == RAGGED_ROWS ? q.groups : 1;
        if (!make_map(&p.w, q.b, bf16, 3, q.tb ? q.N : q.K, q.tb ? q.K : q.N, q.ldb, batch, q.stride_b,
                      q.tb ? TILE_F : DEPTH) ||
            !make_map(&p.x, q.a, bf16, 2, q.ta ? q.K : q.M, q.ta ? q.M : q.K, q.lda, 1, 0, q.ta ? DEPTH : p.x_box))
            return FGEMM_ERR_NOT_SUPPORTED;
    }
    const long long most = PAIR ? sms / 2 : sms;
    const dim3 grid((unsigned)(ctas * ((!PAIR && plan.ranks > 1) || tiles < most ? tiles : most)));
    return mx::launch(kernel, grid, threads_of(PAIR), (size_t)smem, stream, (unsigned)ctas, p, err) == cudaSuccess ? FGEMM_OK
                                                                                                        : FGEMM_ERR_LAUNCH;
}

template <bool PAIR, class T, class O, bool LONG>
static fgemm_status launch_kind(const Product &q, const Plan &plan, cudaStream_t stream)
{
    if (q.slope && (q.act != FGEMM_ACT_NONE || q.partial)) return launch_instance<PAIR, T, O, LONG, GRADIENT>(q, plan, stream);
    if (!q.slope && (q.z || q.beta != 0.0f)) return launch_instance<PAIR, T, O, LONG, FORWARD>(q, plan, stream);
    return launch_instance<PAIR, T, O, LONG, PLAIN>(q, plan, stream);
}

template <class T, class O>
fgemm_status launch_product_type(const Product &q, const Plan &plan, cudaStream_t stream)
{
    if (plan.in_turns)
        return plan.pair ? launch_kind<true, T, O, true>(q, plan, stream) : launch_kind<false, T, O, true>(q, plan, stream);
    return plan.pair ? launch_kind<true, T, O, false>(q, plan, stream) : launch_kind<false, T, O, false>(q, plan, stream);
}

}  // namespace h16
}  // namespace fgemm
