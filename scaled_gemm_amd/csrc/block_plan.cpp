// Which kernel a block-scaled product launches, and how routing cuts its
// tokens, chosen on the host from the call's extents alone.
#include "block.h"

#include <cmath>

namespace ptpc {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tiled kernels and what a K block of 128 costs in them, in microseconds, with
// the launch at 3: `full`, a workgroup's share of a CU when all are busy, and `alone`,
// one workgroup on a CU of an otherwise idle GPU (its loads' latency over the blocks
// in flight, or a CU's fill rate).  The two widest tiles have no `alone`: a CU holds
// one of them, and a round of them is priced as a full one however many CUs it leaves
// idle (one on an idle GPU takes 0.78 and 1.3).  Measured over 1 to 8192 tokens, layers
// of 1024 x 1024 to 8192 x 10240 and 8 to 256 experts (72 shapes): the cheapest kernel
// by these numbers ran within 0.5% of the fastest of the six on average, 9% at most;
// over 90 others of 512 to 65536 rows, K from 256 on, within 0.9%, 14% at most.
struct TileCost {
    BlockPlan plan;
    int64_t rows, cols;
    double alone, full;
};
constexpr double kWholeRounds = 0.0;            // in the place of `alone`
constexpr TileCost kTiles[] = {
    {BlockPlan::k32x64, 32, 64, 0.155, 0.153},
    {BlockPlan::k64x64, 64, 64, 0.20, 0.237},
    {BlockPlan::k64x128, 64, 128, 0.287, 0.41},
    {BlockPlan::k128x128, 128, 128, 0.475, 0.64},
    {BlockPlan::k128x256, 128, 256, kWholeRounds, 1.07},
    {BlockPlan::k256x256, 256, 256, kWholeRounds, 1.75},
};
constexpr double kCus = 256.0, kLaunch = 3.0;
// The few-row kernel: 16 columns a workgroup, whose eight waves share the K blocks.
constexpr double kFewAlone = 0.09, kFewFull = 0.16, kFewLaunch = 3.3;

double tile_cost(const TileCost& t, double row_tiles, int64_t Co, int64_t nks) {
    const double load = row_tiles * (double)ceil_div(Co, t.cols) / kCus;
    const double up = std::ceil(load);
    if (t.alone == kWholeRounds) return kLaunch + (double)nks * t.full * up;
    const double busy = t.full * (load + up) / 2;
    const double idle = t.alone + (t.full - t.alone) * (load < 1.0 ? load : 1.0);
    return kLaunch + (double)nks * (busy > idle ? busy : idle);
}

}  // namespace

BlockPlan block_gemm_plan(int64_t T, int64_t E, int64_t Ci, int64_t Co) {
    // (Ci == 0 writes zeros: tiles for the results, as for one K block)
    const int64_t nks = Ci > 0 ? scale_blocks(Ci) : 1;
    // Experts: as many have rows as T rows dealt out at random reach, and each has
    // half a tile of rows that are not there (the tiled kernels skip products, not
    // loads, of a half that is empty).
    const double some = E > 0 ? (double)E * (1.0 - std::pow(1.0 - 1.0 / (double)E, (double)T)) : 1.0;
    BlockPlan best = BlockPlan::k256x256;
    double least = 0.0;
    for (const TileCost& t : kTiles) {
        double tiles = (double)ceil_div(T, t.rows);
        if (E > 0) {
            const double each = (double)T / some / (double)t.rows + 0.5;
            tiles = some * (each > 1.0 ? each : 1.0);
        }
        const double c = tile_cost(t, tiles, Co, nks);
        if (least == 0.0 || c < least) {
            least = c;
            best = t.plan;
        }
    }
    if (E == 0 && T <= kFewRows16) {
        const double load = (double)ceil_div(Co, 16) / kCus;
        const double each = load * kFewFull > kFewAlone ? load * kFewFull : kFewAlone;
        if (kFewLaunch + (double)nks * each < least) best = BlockPlan::kFew;
    }
    return best;
}

const char* block_plan_name(BlockPlan p) {
    switch (p) {
        case BlockPlan::k256x256: return "block_gemm_kernel<256,256>";
        case BlockPlan::k128x256: return "block_gemm_kernel<128,256>";
        case BlockPlan::k128x128: return "block_gemm_kernel<128,128>";
        case BlockPlan::k64x128: return "block_gemm_kernel<64,128>";
        case BlockPlan::k64x64: return "block_gemm_kernel<64,64>";
        case BlockPlan::k32x64: return "block_gemm_kernel<32,64>";
        case BlockPlan::kFew: return "block_few_kernel";
    }
    return nullptr;
}

int64_t block_gemm_grid(BlockPlan p, int64_t T, int64_t E, int64_t Co) {
    if (p == BlockPlan::kFew) return ceil_div(Co, 16);
    for (const TileCost& t : kTiles)
        if (t.plan == p)
            return (E > 0 ? max_expert_tiles(T, E, t.rows) : ceil_div(T, t.rows)) *
                   ceil_div(Co, t.cols);
    return 0;
}

RoutePlan route_plan(int64_t T) {
    RoutePlan p;
    p.chunk = 16;                                  // a token for each wave
    while (ceil_div(T, p.chunk) > kRouteMaxChunks) p.chunk *= 2;
    p.chunks = T > 0 ? ceil_div(T, p.chunk) : 1;       // without tokens: the offsets
    return p;
}

}  // namespace ptpc
