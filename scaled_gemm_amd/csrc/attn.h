// Internal launchers of the attention operators (host side).  Arguments are
// validated before these are called; each launcher only enqueues kernels on
// the given stream and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ptpc {

// The paged cache as the kernels see it (include/ptpc.h: ptpc_kv_cache).
struct CacheView {
    uint8_t* k;            // bf16 or E4M3 rows of D elements
    uint8_t* v;
    float* dk;             // scales, E4M3 caches only
    float* dv;
    int32_t pages;
    int32_t kv_heads;
    int32_t page_shift;    // log2(page_size)
    int32_t D;
    bool fp8;
};

struct RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float* table;
    int64_t n_pos;
    int32_t rot_dim;
    bool interleaved;
    const int32_t* positions;
    const int64_t* slots;
    int64_t T;
    int32_t q_heads;
    CacheView cache;
    uint16_t* q_out;
    int64_t ldqo;
};
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t s);

// Attention of T rows of q.  Keys and values: the cache through page_table
// (paged) or rows of k / v packed like q (prompt: page_table == nullptr).
struct AttnArgs {
    const uint16_t* q;
    int64_t ldq;
    const int32_t* cu;
    int64_t T;
    int32_t B;
    int32_t q_heads, kv_heads, D;
    float scale;
    uint16_t* out;
    int64_t ldo;
    // prompt
    const uint16_t *k, *v;
    int64_t ldk, ldv;
    // paged
    CacheView cache;
    const int32_t* page_table;
    int64_t ld_table;
    int32_t table_keys;    // table_pages * page_size, at most 2^31 - 1
    const int32_t* kv_lens;
    int64_t max_q, max_kv;
    float* ws;
};
// Launch of a paged call.  A workgroup takes the query rows (token, query head
// of the group) of one sequence and key head, tile_rows at a time, over one
// range of `chunk` keys; ranges beyond the first of a tile leave fp32 parts in
// the workspace, which a second kernel joins.
constexpr int64_t kFewRows = 64;          // up to here: waves split the keys, not the rows
constexpr int64_t kFewTile = 32;          // rows of a workgroup then
constexpr int64_t kSmallTile = 128, kLargeTile = 256;
constexpr int64_t kFewSlots = 512;        // workgroups the GPU runs at once (two a CU)
constexpr int64_t kFewChunk = 2048, kTileMinChunk = 512, kRangeCost = 512;   // keys
constexpr int64_t kMaxSplits = 128;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;         // times 512 threads < 2^32
constexpr int64_t kMaxSplitBlocks = int64_t(1) << 16;    // more items than half of it: no split
constexpr int64_t kMaxWorkspace = int64_t(1) << 28;      // bytes
// Most rows (T * q_heads) and (sequence, key head) pairs of one call.
constexpr int64_t kMaxRowHeads = int64_t(1) << 28, kMaxPairs = int64_t(1) << 20;
struct PagedPlan {
    bool few;
    int tile_rows;
    int row_tiles;         // few rows: tiles the launch has for each sequence and key head
    int chunk;             // keys of a range, a multiple of 128
    int splits;            // ranges (the last one is open-ended)
    int64_t items;         // (tile, key head) pairs
    int64_t blocks;        // items * splits
    int64_t workspace;     // bytes, 0 if splits == 1
};
PagedPlan paged_plan(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                     const CacheView& c);
size_t attn_paged_workspace(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t q_heads,
                            const CacheView& c);
hipError_t launch_attn_paged(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_tiles(const AttnArgs& a, const PagedPlan& p, hipStream_t s);
hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t s);

}  // namespace ptpc
