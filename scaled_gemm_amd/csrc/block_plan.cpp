// Which kernel a block-scaled product launches, and how routing cuts its
// tokens, chosen on the host from the call's extents alone.
#include "block.h"

namespace ptpc {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

BlockPlan block_gemm_plan(int64_t T, int64_t E, int64_t Ci, int64_t Co) {
    (void)Ci;
    // mean rows of one weight
    const int64_t m = ceil_div(T, E);
    if (m <= 16) return BlockPlan::kFew16;
    if (m <= 32) return BlockPlan::kFew32;
    if (m <= 64) return BlockPlan::kFew64;
    const int64_t cus = 256;
    if (E * ceil_div(m, 256) * ceil_div(Co, 256) >= cus) return BlockPlan::k256x256;
    if (E * ceil_div(m, 128) * ceil_div(Co, 256) >= cus) return BlockPlan::k128x256;
    if (E * ceil_div(m, 128) * ceil_div(Co, 128) >= cus) return BlockPlan::k128x128;
    return BlockPlan::k64x128;
}

const char* block_plan_name(BlockPlan p) {
    switch (p) {
        case BlockPlan::k256x256: return "block_gemm_kernel<256,256>";
        case BlockPlan::k128x256: return "block_gemm_kernel<128,256>";
        case BlockPlan::k128x128: return "block_gemm_kernel<128,128>";
        case BlockPlan::k64x128: return "block_gemm_kernel<64,128>";
        case BlockPlan::kFew64: return "block_few_kernel<64>";
        case BlockPlan::kFew32: return "block_few_kernel<32>";
        case BlockPlan::kFew16: return "block_few_kernel<16>";
    }
    return nullptr;
}

BlockTile block_tile(BlockPlan p) {
    switch (p) {
        case BlockPlan::k256x256: return {256, 256};
        case BlockPlan::k128x256: return {128, 256};
        case BlockPlan::k128x128: return {128, 128};
        case BlockPlan::k64x128: return {64, 128};
        case BlockPlan::kFew64: return {64, 32};
        case BlockPlan::kFew32: return {32, 32};
        case BlockPlan::kFew16: return {16, 32};
    }
    return {1, 1};
}

int64_t block_gemm_grid(BlockPlan p, int64_t T, int64_t E, int64_t Co) {
    const BlockTile t = block_tile(p);
    return (E > 0 ? max_expert_tiles(T, E, t.rows) : ceil_div(T, t.rows)) * ceil_div(Co, t.cols);
}

RoutePlan route_plan(int64_t T) {
    RoutePlan p;
    p.chunk = 64;
    if (T > p.chunk) p.chunk = 32;
    while (ceil_div(T, p.chunk) > kRouteMaxChunks) p.chunk *= 2;
    p.chunks = T > 0 ? ceil_div(T, p.chunk) : 1;       // without tokens: the offsets
    return p;
}

}  // namespace ptpc
