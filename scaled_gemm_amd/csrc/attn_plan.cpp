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
    const int64_t keys = max64(max_kv, 1), step = 128;
    int64_t chunk;
    if (p.few) {
        // up to 32 rows a workgroup, more rows in equal parts
        p.row_tiles = (int)ceil_div(rows, kFewTile);
        p.tile_rows = (int)ceil_div(rows, p.row_tiles);
        p.items = B * c.kv_heads * p.row_tiles;
        // Ranges for eight rounds of the GPU (ragged lengths even out), but of kFewChunk keys
        // at least where that leaves one round: a workgroup's start, its first loads and the
        // join of its waves cost as much as hundreds of keys.  Measured: 32 sequences over up
        // to 8192 keys, 8 key heads, 83 us with ranges of 512 keys, 78 with 1024, 75 with 2048
        // and 4096; 32 over up to 8192 E4M3 keys, 16 key heads of 64, 50 us with 2048, 63 with
        // 4096; 35 rows of 16 sequences over up to 4096, 4 key heads, 33 us with two rounds (512
        // keys), 26 with one (1024); 96 over up to 32768 E4M3 keys, 8 key heads, 445 us with
        // eight rounds (6144 keys), 501 with two.
        const int64_t all = p.items * keys;
        chunk = max64(all / (kFewSlots * 8), min64(kFewChunk, all / kFewSlots));
    } else {
        p.row_tiles = 1;
        p.tile_rows = rows <= kSmallTile ? kSmallTile : kLargeTile;
        // every sequence has at most one tile that is not full
        const int64_t tiles = B == 1 ? ceil_div(T * G, p.tile_rows) : T * G / p.tile_rows + B;
        p.items = tiles * c.kv_heads;
        const int64_t slots = p.tile_rows == kSmallTile ? 512 : 256;
        if (B > 1) {
            // lengths may differ: ranges for eight rounds of the GPU (four 70B chunks over up
            // to 16384 keys: 422 us with four rounds, 385 us with eight)
            chunk = ceil_div(keys, max64(slots * 8 / p.items, 1));
        } else {
            // One sequence: the number of ranges whose rounds take the fewest keys, a range's
            // start and its fp32 part counted as kRangeCost keys.  Measured with 0, 128, 512 and
            // 2048: 300 tokens of 64 heads over 4096 keys 89, 65, 65 and 65 us (without a cost,
            // ranges that save nothing), 64 tokens of 32 heads over 2048 keys 29, 29, 29 and 58
            // (too dear: no ranges where they help); 16 to 1000 tokens over 8192 to 32768 keys
            // level.
            int64_t best = 1, cost = INT64_MAX;
            for (int64_t n = 1; n <= 64; ++n) {
                const int64_t each = ceil_div(ceil_div(keys, n), step) * step + (n > 1 ? kRangeCost : 0);
                const int64_t t = ceil_div(p.items * n, slots) * each;
                if (t < cost) {
                    cost = t;
                    best = n;
                }
            }
            chunk = ceil_div(keys, best);
        }
        // Measured with 128, 256, 512 and 1024 keys at least, 32 query and 8 key heads: 8
        // sequences of 64 tokens over up to 2048 keys 48, 38, 36 and 45 us, 2 of 300 over up to
        // 1200 43, 35, 37 and 47, 4 of 40 over up to 1500 E4M3 keys 28, 30, 37 and 46, one of 64
        // over 2048 28, 26, 29 and 40; 8 of 9 over up to 4096 E4M3 keys, 64 query heads, 43, 36,
        // 32 and 35.
        chunk = max64(chunk, kTileMinChunk);
    }
    chunk = max64(chunk, ceil_div(keys, kMaxSplits));
    chunk = max64(ceil_div(chunk, step) * step, step);
    int64_t splits = max_q > 0 ? ceil_div(keys, chunk) : 1;
    const int64_t part = p.tile_rows * (int64_t)(c.D + 2) * 4;       // bytes of one range's sums
    if (splits > 1 && (p.items * splits > kMaxSplitBlocks || p.items * splits * part > kMaxWorkspace)) {
        splits = max64(1, min64(kMaxSplitBlocks / p.items, kMaxWorkspace / (p.items * part)));
        chunk = ceil_div(ceil_div(max_kv, splits), step) * step;
        splits = ceil_div(max_kv, chunk);
    }
    p.splits = (int)splits;
    p.chunk = (int)chunk;                     // max_kv <= 2^30
    p.blocks = p.items * splits;
    p.workspace = splits > 1 ? p.items * splits * part : 0;
    return p;
}

size_t attn_paged_workspace(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                            const CacheView& c) {
    return (size_t)paged_plan(T, B, max_q, max_kv, q_heads, c).workspace;
}

}  // namespace ptpc
