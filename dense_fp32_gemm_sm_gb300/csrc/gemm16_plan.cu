// gemm16_plan.cu -- how a 16-bit product runs: the estimated time of each candidate, from its tiles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fgemm_internal.h"
#include "gemm16.h"

namespace fgemm {
namespace h16 {
namespace {

double up(double a, double b) { return (double)(((long long)a + (long long)b - 1) / (long long)b); }
double most(double a, double b) { return a > b ? a : b; }
double least(double a, double b) { return a < b ? a : b; }

// The estimate in us.  Fitted to 660 measurements of 60 products (1 to 8192 rows, 80 to 11008 columns, depths of 72
// to 11008, both ends cold in L2): the plan of the least estimate took 1.6 % longer than the best one on average.
//   64 of depth through a pair's barriers 0.139 us and more with the rows of its tile, through one CTA's
//   0.103; a tile's epilogue; what all CTAs bring through L2 at 14 TB/s; the launch, and the joining of ranks.
struct Work {
    double row_tiles, rows;  // tiles of rows (all groups'), rows of one
    double N, blocks;        // columns, 64-deep blocks of a product
    double products;         // weights' gradient: groups, each with all tiles; else 1
    double bytes;            // operands and output, once
};

double estimate(const Work &w, bool pair, int ranks, int sms)
{
    const double tiles = w.row_tiles * w.products * up(w.N, pair ? 256 : 128);
    const double stage = (pair ? 32768 : 16384) + 128 * w.rows, share = up(w.blocks, ranks);
    const double memory = most(tiles * ranks * share * stage / 14.2e6, w.bytes / 10.1e6);
    const double waves = pair ? up(tiles, sms / 2) : up(tiles * ranks, sms);
    const double depth = share * (pair ? most(0.133, 0.1385 + 0.00074 * w.rows) : 0.1034);
    const double epilogue = (pair ? 0.01135 : 0.00573) * w.rows;
    const double t = (pair ? 3.03 : 3.18) + most(waves * most(depth, epilogue) + least(depth, epilogue), memory);
    return ranks > 1 ? t + 0.62 + 0.0316 * w.rows : t;
}

}  // namespace

Plan plan_product(long long M, long long N, long long K, int ragged, long long groups, bool sums, bool fine, int sms)
{
    static const int pair_rows[] = {256, 224, 192, 160, 128, 96, 64}, rows[] = {64, 32, 16}, all_ranks[] = {1, 2, 3, 4, 5, 6, 8};
    const double used = (double)(ragged == RAGGED_ROWS ? (groups < M ? groups : M) : 1);
    const double depth = ragged == RAGGED_DEPTH ? (double)K / (double)groups : (double)K;
    // Column sums: the room for partial ones is two rows for every SUMS_ROWS rows and two a group.
    const int least_rows = sums ? SUMS_ROWS : 1;
    Plan best{0, 0, 1, 1, 0};
    double least_time = 0;
    const auto consider = [&](bool pair, int nt, int ranks) {
        Work w;
        // Groups of rows whose sizes the host does not know: half a tile more for each that has rows.
        w.row_tiles = ragged == RAGGED_ROWS && groups > 1 ? most(used, up((double)M, nt) + used / 2) : up((double)M, nt);
        w.rows = least(nt, 32 * up(up((double)M, w.row_tiles), 32));
        w.N = (double)N;
        w.blocks = up(depth, 64) + (ragged == RAGGED_DEPTH && groups > 1 ? 0.5 : 0.0);
        w.products = ragged == RAGGED_DEPTH ? (double)groups : 1.0;
        w.bytes = 2.0 * (M * (double)K + used * K * (double)N) + 2.0 * w.products * M * (double)N;
        // A cluster's ranks all run at once or not at all: no more of them than SMs.
        const double ctas = w.row_tiles * w.products * up(w.N, 128);
        if (ranks > 1 && (ctas * ranks > sms || w.blocks < 2 * ranks)) return;
        const double t = estimate(w, pair, ranks, sms);
        if (best.nt == 0 || t < least_time) {
            // Two CTAs an SM where there are more tiles than SMs: the epilogue of one beside the products of the other.
            best = Plan{pair, nt, ranks, !pair && ctas > sms ? 2 : 1, 0};
            least_time = t;
        }
    };
    for (const int nt : pair_rows)
        if (nt < 2 * M || nt == 64) consider(true, nt, 1);
    for (const int nt : rows) {
        if (nt < least_rows || (nt >= 2 * M && nt > 16 && nt > least_rows)) continue;
        for (const int ranks : all_ranks) {
            if (ranks > 1 && (sums || ragged == RAGGED_DEPTH)) break;
            consider(false, nt, ranks);
        }
    }
    best.in_turns = fine && K > 512;
    return best;
}

fgemm_status launch_product(const Product &q, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) return FGEMM_ERR_LAUNCH;
    const Plan plan = plan_product(q.M, q.N, q.K, q.ragged, q.groups, q.partial != nullptr,
                                   q.partial != nullptr || q.out_type == FGEMM_F32, sms);
    return q.type == FGEMM_BF16 ? launch_product_type<__nv_bfloat16>(q, plan, stream)
                                : launch_product_type<__half>(q, plan, stream);
}

}  // namespace h16
}  // namespace fgemm
