// mxfp4_tc_launch.cuh -- host side of the MXFP4 product: tensor maps and the launch of one
// kernel instance.  Each output type's instances are compiled in a unit of their own.
#pragma once

#include <atomic>
#include <cstring>

#include "ctx_id.h"
#include "fgemm_internal.h"
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

template <int NT, class T, bool SPLIT>
static fgemm_status launch_instance(const GemmArgs &g, int ranks, cudaStream_t stream)
{
    using L = TcTile<NT>;
    const auto kernel = mxfp4_tc_kernel<NT, T, SPLIT>;
    static std::atomic<unsigned long long> ready_ctx[64];
    int dev = 0, sms = 0;
    unsigned *const err = tc_error_word();
    if (!err || cudaGetDevice(&dev) != cudaSuccess || device_sm_count(&sms) != 0) {
        (void)cudaGetLastError();
        return FGEMM_ERR_LAUNCH;
    }
    std::atomic<unsigned long long> &ready = ready_ctx[dev & 63];
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ready.load(std::memory_order_acquire) != ctx) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_BYTES) != cudaSuccess) {
            (void)cudaGetLastError();
            return FGEMM_ERR_LAUNCH;
        }
        ready.store(current_context_id(), std::memory_order_release);
    }
    TcArgs p;
    std::memset(&p, 0, sizeof(p));
    const long long blocks = blocks_of(g.K);
    if (!make_codes_map(&p.w, g.b, g.N, blocks, g.ldb, TC_ROWS) || !make_codes_map(&p.x, g.a, g.M, blocks, g.lda, NT))
        return FGEMM_ERR_NOT_SUPPORTED;
    p.w_scales = g.b_scales;
    p.x_scales = g.a_scales;
    p.c = g.c;
    p.bias = g.bias;
    p.ldc = g.ldc;
    p.atoms = atoms_of(blocks);
    p.M = g.M;
    p.N = g.N;
    p.blocks = (int)blocks;
    p.alpha = g.alpha;
    p.beta = g.beta;
    p.relu = g.relu;
    p.c_pairs = reinterpret_cast<uintptr_t>(g.c) % 4 == 0 && g.ldc % 2 == 0;
    p.tiles_x = (int)(((long long)g.M + NT - 1) / NT);
    p.tiles_w = (int)(((long long)g.N + TC_ROWS - 1) / TC_ROWS);
    p.wait_limit_ns = tc_wait_limit_ns();
    p.withhold = tc_withheld_k_block();
    const long long tiles = (long long)p.tiles_x * p.tiles_w;
    if (!SPLIT) {
        kernel<<<(unsigned)(tiles < sms ? tiles : sms), TC_THREADS, L::SMEM_BYTES, stream>>>(p, err);
    } else {
        if (tiles * ranks > 0x7FFFFFFF) return FGEMM_ERR_NOT_SUPPORTED;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(tiles * ranks));
        cfg.blockDim = dim3(TC_THREADS);
        cfg.dynamicSmemBytes = L::SMEM_BYTES;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ranks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, kernel, p, err) != cudaSuccess) {
            (void)cudaGetLastError();
            return FGEMM_ERR_LAUNCH;
        }
    }
    return cudaGetLastError() == cudaSuccess ? FGEMM_OK : FGEMM_ERR_LAUNCH;
}

// The product with tiles of `nt` rows of A, each over a cluster of `ranks` CTAs (0: whole
// tiles, persistent CTAs).
template <class T>
fgemm_status launch_tc_type(const GemmArgs &g, int nt, int ranks, cudaStream_t stream)
{
    if (ranks == 0)
        return nt == 256 ? launch_instance<256, T, false>(g, 0, stream) : launch_instance<128, T, false>(g, 0, stream);
    switch (nt) {
    case 16: return launch_instance<16, T, true>(g, ranks, stream);
    case 32: return launch_instance<32, T, true>(g, ranks, stream);
    case 64: return launch_instance<64, T, true>(g, ranks, stream);
    default: return launch_instance<128, T, true>(g, ranks, stream);
    }
}

}  // namespace mx
}  // namespace fgemm
