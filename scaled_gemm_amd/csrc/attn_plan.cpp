// Which kernel an attention call launches and how its keys are split over
// workgroups, chosen on the host from the call's extents alone.
#include "attn.h"

namespace ptpc {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

}  // namespace

PagedPlan paged_plan(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                     const CacheView& c) {
    PagedPlan p{};
    const int64_t G = q_heads / c.kv_heads;
    const int64_t rows = min64(max64(max_q, 1), T) * G;
    p.few = rows <= kFewRows;
    if (p.few) {
        p.tile_rows = (int)rows;
        p.items = B * c.kv_heads;
    } else {
        p.tile_rows = rows <= kSmallTile ? kSmallTile : kLargeTile;
        // every sequence has at most one tile that is not full
        p.items = (T * G / p.tile_rows + B) * c.kv_heads;
    }
    // Ranges of keys: enough workgroups for kRounds rounds of the GPU where the
    // keys allow it, none shorter than kMinChunk.
    const int64_t step = 128;
    const int64_t slots = p.few ? kFewSlots : p.tile_rows == kSmallTile ? 512 : 256;
    const int64_t target = slots * (p.few ? kFewRounds : kTileRounds);
    const int64_t least = p.few ? kFewMinChunk : kTileMinChunk;
    int64_t chunk = ceil_div(max64(max_kv, 1), max64(target / p.items, 1));
    chunk = max64(chunk, least);
    chunk = max64(chunk, ceil_div(max64(max_kv, 1), kMaxSplits));
    chunk = ceil_div(chunk, step) * step;
    int64_t splits = max_q > 0 ? ceil_div(max64(max_kv, 1), chunk) : 1;
    const int64_t part = p.tile_rows * (int64_t)(c.D + 2) * 4;       // bytes of one range's sums
    if (splits > 1 && (p.items * splits > kMaxBlocks || p.items * splits * part > kMaxWorkspace)) {
        splits = max64(1, min64(kMaxBlocks / p.items, kMaxWorkspace / (p.items * part)));
        chunk = ceil_div(ceil_div(max_kv, splits), step) * step;
        splits = ceil_div(max_kv, chunk);
    }
    p.splits = (int)splits;
    p.chunk = (int)min64(chunk, INT32_MAX / 2);
    p.blocks = p.items * splits;
    p.workspace = splits > 1 ? p.items * splits * part : 0;
    return p;
}

size_t attn_paged_workspace(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                            const CacheView& c) {
    return (size_t)paged_plan(T, B, max_q, max_kv, q_heads, c).workspace;
}

}  // namespace ptpc
