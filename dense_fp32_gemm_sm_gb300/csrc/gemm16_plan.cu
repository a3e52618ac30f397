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
// to 11008, operands not in L2), before the kernel came in kinds and divided a last round's tiles, which are counted as a whole
// round here.  On 80 other products of these ranges with GELU, as the kernel is now, the plan of the least estimate is the
// best one for 55, and takes 1.9 % longer on average, 20 % at most.
//   64 of depth through a pair's barriers 0.151 us and more with the rows of its tile, through one CTA's
//   0.151; a tile's epilogue and its way through the roles; what all CTAs bring through L2 at 15.8 TB/s, and from memory
//   at 6.6; the launch, and the joining of ranks.
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
    const double memory = most(tiles * ranks * share * stage / 15.8e6, w.bytes / 6.6e6);
    const double waves = pair ? up(tiles, sms / 2) : up(tiles * ranks, sms);
    const double depth = share * (pair ? most(0.151, 0.117 + 0.00065 * w.rows) : 0.151);
    const double epilogue = (pair ? 0.22 + 0.0104 * w.rows : 0.56 + 0.0097 * w.rows);
    const double t = (pair ? 2.52 : 1.81) + most(waves * most(depth, epilogue) + least(depth, epilogue), memory);
    return ranks > 1 ? t + 1.22 + 0.0187 * w.rows : t;
}

}  // namespace

Plan plan_product(long long M, long long N, long long K, int ragged, long long groups, bool sums, long long one_go, int sms)
{
    static const int pair_rows[] = {256, 224, 192, 160, 128, 96, 64}, rows[] = {64, 32, 16}, all_ranks[] = {1, 2, 3, 4, 5, 6, 8};
    const double used = (double)(ragged == RAGGED_ROWS ? (groups < M ? groups : M) : 1);
    const double depth = ragged == RAGGED_DEPTH ? (double)K / (double)groups : (double)K;
    // Column sums: the room for partial ones is two rows for every SUMS_ROWS rows and two a group.
    const int least_rows = sums ? SUMS_ROWS : 1;
    Plan best{0, 0, 1, 0};
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
        // A cluster's ranks all run at once or not at all, on SMs of one part of the GPU: no more of them than SMs, of more
        // than two than four fifths (24 clusters of six did not fit at once, 14.7 us in place of 8.5, nor on another GPU 48 of
        // three, 11.8 in place of 6.6).
        const double ctas = w.row_tiles * w.products * up(w.N, 128) * ranks;
        if (ranks > 1 && (ctas > sms || (ranks > 2 && ctas > 0.8 * sms) || w.blocks < 2 * ranks)) return;
        const double t = estimate(w, pair, ranks, sms);
        if (best.nt == 0 || t < least_time) {
            best = Plan{pair, nt, ranks, 0};
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
    best.in_turns = K > one_go;
    return best;
}

namespace {

// The last plans of this thread: weighing the candidates takes 1 us of a call's 4.
struct Planned {
    long long M, N, K;
    int ragged, groups, sums, go, sms;
    Plan plan;
};

Plan planned(const Product &q, int sms)
{
    static thread_local Planned last[8];
    static thread_local unsigned next = 0;
    const int sums = q.partial != nullptr, go = (int)one_go(q.out_type, sums != 0);
    for (const Planned &p : last)
        if (p.M == q.M && p.N == q.N && p.K == q.K && p.ragged == q.ragged && p.groups == q.groups && p.sums == sums &&
            p.go == go && p.sms == sms)
            return p.plan;
    Planned &p = last[next++ % 8];
    p = Planned{q.M, q.N, q.K, q.ragged, q.groups, sums, go, sms,
                plan_product(q.M, q.N, q.K, q.ragged, q.groups, sums != 0, go, sms)};
    return p.plan;
}

}  // namespace

fgemm_status launch_product(const Product &q, cudaStream_t stream)
{
    int sms = 0;
    if (device_sm_count(&sms) != 0) return FGEMM_ERR_LAUNCH;
    const Plan plan = planned(q, sms);
    if (q.type == FGEMM_BF16)
        return q.out_type == FGEMM_F32 ? launch_product_type<__nv_bfloat16, float>(q, plan, stream)
                                       : launch_product_type<__nv_bfloat16, __nv_bfloat16>(q, plan, stream);
    return q.out_type == FGEMM_F32 ? launch_product_type<__half, float>(q, plan, stream)
                                   : launch_product_type<__half, __half>(q, plan, stream);
}

}  // namespace h16
}  // namespace fgemm
