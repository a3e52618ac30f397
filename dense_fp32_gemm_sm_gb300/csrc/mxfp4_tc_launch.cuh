// mxfp4_tc_launch.cuh -- host side of the MXFP4 product: tensor maps and the launch of one
// kernel instance.  Each output type's instances are compiled in a unit of their own.
#pragma once

#include <atomic>
#include <cstring>

#include "ctx_id.h"
#include "fgemm_internal.h"
#include "mxfp4_launch.h"
#include "mxfp4_tc.cuh"
#include "tc_host.h"

namespace fgemm {
namespace mx {

// Codes of a quantised matrix as a tensor map: rows of whole blocks, boxes of 128 bytes
// (the 128-byte swizzle's row) x box_rows; beyond the last block and row it reads 0.
static bool make_codes_map(CUtensorMap *map, const uint8_t *codes, long long rows, long long blocks, long long ld, int box_rows)
{
    const auto encode = tc_encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(16 * blocks), (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales as a tensor map of whole atoms: (128 words, atoms along K, 128-row groups), boxes of
// two atoms of `groups` groups; beyond the matrix it reads 0.
static bool make_scales_map(CUtensorMap *map, const uint8_t *scales, long long rows, long long atoms, int groups)
{
    const auto encode = tc_encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[3] = {ATOM_BYTES / 4, (cuuint64_t)atoms, (cuuint64_t)((rows + ATOM_ROWS - 1) / ATOM_ROWS)};
    const cuuint64_t strides[2] = {ATOM_BYTES, (cuuint64_t)(atoms * ATOM_BYTES)};
    const cuuint32_t box[3] = {ATOM_BYTES / 4, 2, (cuuint32_t)groups}, estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(scales), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The arguments that do not depend on the kernel, for tiles of tile_x rows of A and tile_w of B.
static void fill_args(TcArgs &p, const GemmArgs &g, int tile_x, int tile_w)
{
    const long long blocks = blocks_of(g.K);
    p.w_scales = g.b_scales;
    p.x_scales = g.a_scales;
    p.c = g.c;
    p.bias = g.bias;
    p.ldc = g.ldc;
    p.atoms = atoms_of(blocks);
    p.M = g.M;
    p.N = g.N;
    p.blocks = (int)blocks;
    p.K = g.K;
    p.dependent = g.dependent;
    p.alpha = g.alpha;
    p.beta = g.beta;
    p.relu = g.relu;
    p.c_pairs = reinterpret_cast<uintptr_t>(g.c) % 4 == 0 && g.ldc % 2 == 0;
    p.tiles_x = (int)(((long long)g.M + tile_x - 1) / tile_x);
    p.tiles_w = (int)(((long long)g.N + tile_w - 1) / tile_w);
    p.wait_limit_ns = tc_wait_limit_ns();
    p.withhold = tc_withheld_k_block();
}

// What a launch needs besides its arguments: the error word, the SM count, and the kernel
// opted in to its shared memory, once per context (`Kernel` keeps instances' records apart).
template <class Kernel, Kernel kernel>
static bool prepare(int smem_bytes, unsigned **err, int *sms)
{
    static std::atomic<unsigned long long> ready_ctx[64];
    int dev = 0;
    *err = tc_error_word();
    if (!*err || cudaGetDevice(&dev) != cudaSuccess || device_sm_count(sms) != 0) return false;
    std::atomic<unsigned long long> &ready = ready_ctx[dev & 63];
    const unsigned long long ctx = current_context_id();
    if (ctx != 0 && ready.load(std::memory_order_acquire) == ctx) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) != cudaSuccess) return false;
    ready.store(current_context_id(), std::memory_order_release);
    return true;
}

// Pairs of CTAs, tiles of 256 rows of B by NT of A.
template <int NT, class T>
static fgemm_status launch_pairs(const GemmArgs &g, cudaStream_t stream)
{
    using L = PairTile<NT>;
    unsigned *err = nullptr;
    int sms = 0;
    constexpr auto kernel = &mxfp4_pair_kernel<NT, T>;
    if (!prepare<decltype(kernel), kernel>(L::SMEM_BYTES, &err, &sms)) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    PairArgs p;
    std::memset(&p, 0, sizeof(p));
    fill_args(p.t, g, NT, 256);
    if (!make_codes_map(&p.w, g.b, g.N, p.t.blocks, g.ldb, 128) || !make_codes_map(&p.x, g.a, g.M, p.t.blocks, g.lda, NT / 2) ||
        !make_scales_map(&p.sw, g.b_scales, g.N, p.t.atoms, 1) || !make_scales_map(&p.sx, g.a_scales, g.M, p.t.atoms, 2))
        return FGEMM_ERR_NOT_SUPPORTED;
    const long long tiles = (long long)p.t.tiles_x * p.t.tiles_w, most = sms / 2;
    const dim3 grid((unsigned)(2 * (tiles < most ? tiles : most)));
    return launch(kernel, grid, TC_THREADS, L::SMEM_BYTES, stream, 2, p, err) == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
}

// One CTA a tile (WHOLE), or a cluster of `ranks`.  x, ldx: the unquantised A of SPLIT_FUSED.
template <int NT, class T, int MODE>
static fgemm_status launch_instance(const GemmArgs &g, const void *x, long long ldx, int ranks, cudaStream_t stream)
{
    using L = TcTile<NT, MODE>;
    constexpr auto kernel = &mxfp4_tc_kernel<NT, T, MODE>;
    unsigned *err = nullptr;
    int sms = 0;
    TcArgs p;
    std::memset(&p, 0, sizeof(p));
    fill_args(p, g, NT, TC_ROWS);
    const int stages = (p.blocks + TC_BLOCKS - 1) / TC_BLOCKS;
    // A rank without stages would leave its sums unwritten.
    if (MODE != WHOLE && (ranks < 1 || ranks > 8 || ranks > stages)) return FGEMM_ERR_NOT_SUPPORTED;
    const int smem = L::SMEM_BYTES + (MODE == SPLIT_FUSED ? (stages + ranks - 1) / ranks * L::FUSED_BYTES : 0);
    constexpr int most = MODE == SPLIT_FUSED ? L::SMEM_BYTES + FUSED_SMEM : L::SMEM_BYTES;
    if (smem > most) return FGEMM_ERR_NOT_SUPPORTED;
    if (!prepare<decltype(kernel), kernel>(most, &err, &sms)) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    if (!make_codes_map(&p.w, g.b, g.N, p.blocks, g.ldb, TC_ROWS)) return FGEMM_ERR_NOT_SUPPORTED;
    if (MODE == SPLIT_FUSED) {
        p.x_plain = x;
        p.ldx = ldx;
        p.x_vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * (long long)sizeof(T) % 16 == 0;
    } else if (!make_codes_map(&p.x, g.a, g.M, p.blocks, g.lda, NT)) {
        return FGEMM_ERR_NOT_SUPPORTED;
    }
    const long long tiles = (long long)p.tiles_x * p.tiles_w;
    if (MODE != WHOLE && tiles * ranks > 0x7FFFFFFF) return FGEMM_ERR_NOT_SUPPORTED;
    const dim3 grid((unsigned)(MODE != WHOLE ? tiles * ranks : tiles < sms ? tiles : sms));
    return launch(kernel, grid, TC_THREADS, (size_t)smem, stream, MODE != WHOLE ? (unsigned)ranks : 1u, p, err) == cudaSuccess
               ? FGEMM_OK
               : FGEMM_ERR_LAUNCH;
}

// The product as planned (see GemmPlan).
template <class T>
fgemm_status launch_tc_type(const GemmArgs &g, GemmPlan plan, cudaStream_t stream)
{
    switch (plan.nt) {
    case PAIRS_256: return launch_pairs<256, T>(g, stream);
    case PAIRS_192: return launch_pairs<192, T>(g, stream);
    case 128: return launch_instance<128, T, WHOLE>(g, nullptr, 0, 0, stream);
    case 64: return launch_instance<64, T, SPLIT>(g, nullptr, 0, plan.ranks, stream);
    case 32: return launch_instance<32, T, SPLIT>(g, nullptr, 0, plan.ranks, stream);
    default: return launch_instance<16, T, SPLIT>(g, nullptr, 0, plan.ranks, stream);
    }
}

// The same with A as x (M x K, unquantised, element type T, at most LINEAR_ROWS rows).
template <class T>
fgemm_status launch_fused_type(const GemmArgs &g, const void *x, long long ldx, int ranks, cudaStream_t stream)
{
    return launch_instance<16, T, SPLIT_FUSED>(g, x, ldx, ranks, stream);
}

}  // namespace mx
}  // namespace fgemm
