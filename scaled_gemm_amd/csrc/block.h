// Internal launchers of the block-scaled FP8 operators and the experts (host
// side).  Arguments are validated before these are called; each launcher only
// enqueues kernels on the given stream and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ptpc {

// Elements of a scale's block: along K, and along the columns of a weight.
constexpr int64_t kScaleBlock = 128;
constexpr int64_t scale_blocks(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// count: rows from *count on are left alone (NULL: none are).
hipError_t launch_quant_act_block(const uint16_t* x, int64_t T, int64_t C, int64_t ldx, bool gate,
                                  const int32_t* count, uint8_t* qx, int64_t ldq, float* sx,
                                  int64_t lds, hipStream_t s);

// Weights of E experts (1: a plain layer).  Source elements (expert e, k, o) at
// e * se + k * sk + o * so; packed as ptpc_quant_weight packs, expert after
// expert, with scales [E][blocks of Co][blocks of Ci].
hipError_t launch_quant_weight_block(const uint16_t* w, int64_t E, int64_t Ci, int64_t Co,
                                     int64_t ldw, int64_t se, uint8_t* packed, float* sw,
                                     hipStream_t s);
struct PackArgs {
    const uint8_t* codes;
    int64_t se, sk, so;            // strides of the codes
    const float* scales;
    int64_t te, tk, to;            // strides of the scales [E][blocks of Ci][blocks of Co]
    int64_t E, Ci, Co;
    uint8_t* packed;
    float* sw;
};
hipError_t launch_pack_weight_block(const PackArgs& a, hipStream_t s);
// One workgroup of 256 threads a block of 128 x 128, rows of kWeightGridX of them: a
// grid's x holds fewer than 2^32 threads, and weights have up to 2^24 blocks.
constexpr int64_t kWeightGridX = int64_t(1) << 20;
inline dim3 weight_grid(int64_t blocks) {
    return dim3((unsigned)(blocks < kWeightGridX ? blocks : kWeightGridX),
                (unsigned)((blocks + kWeightGridX - 1) / kWeightGridX));
}

// One product, dense or by experts.  Dense: out[t] from row t.  Experts:
// output row i in offsets[e] .. offsets[e+1]-1 belongs to expert e, and reads
// row i of qx, or (rows != NULL) row rows[i] / top_k.
struct BlockGemmArgs {
    const uint8_t* qx;
    int64_t ldq;
    const float* sx;               // [blocks of Ci] rows of T_in scales, pitch lds
    int64_t lds;
    const uint8_t* wp;
    const float* sw;
    int64_t T;                     // output rows (T, or the pairs)
    int64_t T_in;                  // rows of qx
    int64_t Ci, Co;
    uint16_t* out;
    int64_t ldo;
    // experts
    const int32_t* offsets;        // NULL: dense
    const int32_t* rows;           // NULL: rows of qx are in the output's order
    int32_t E;
    int32_t top_k;
};

// Kernel and tile of a product, chosen on the host from its extents alone:
// T output rows, E experts (0: one weight, dense).
enum class BlockPlan : int { k256x256, k128x256, k128x128, k64x128, k64x64, k32x64, kFew };
constexpr int64_t kFewRows16 = 16;     // rows of the few-row kernel
BlockPlan block_gemm_plan(int64_t T, int64_t E, int64_t Ci, int64_t Co);
const char* block_plan_name(BlockPlan p);
// Workgroups of a product; a launch has at most kMaxGrid of up to 512 threads
// (2^32 threads are the limit of a grid).
constexpr int64_t kMaxGrid = int64_t(1) << 22;
int64_t block_gemm_grid(BlockPlan p, int64_t T, int64_t E, int64_t Co);
hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s);
hipError_t launch_block_gemm_few(const BlockGemmArgs& a, hipStream_t s);

// Most row tiles of bm rows that E experts with R rows in all can need.
constexpr int64_t max_expert_tiles(int64_t R, int64_t E, int64_t bm) {
    return R / bm + (E < R ? E : R);
}

// Routing of T tokens to E experts and the sorted layout of their pairs.
struct RouteArgs {
    const void* logits;
    bool bf16;
    int64_t ldl;
    const float* bias;             // NULL: none
    int64_t T;
    int32_t E, K;
    bool sigmoid, renorm;
    int32_t groups, top_groups, group_top;
    float scale;
    int32_t first, local;          // the experts that are laid out
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* rows;
    int32_t* slots;
    int32_t* ws;                   // [chunks][local] counts
};
constexpr int64_t kMaxExperts = 512;    // eight a lane; one thread each in the layout
constexpr int64_t kRouteMaxChunks = 256;
// Tokens of one workgroup and the workgroups (one: a single launch does it all).
struct RoutePlan {
    int64_t chunk, chunks;
};
RoutePlan route_plan(int64_t T);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

hipError_t launch_combine(const uint16_t* y, int64_t ldy, int64_t R, const int32_t* slots,
                          const float* weights, int64_t T, int32_t K, int64_t C, uint16_t* out,
                          int64_t ldo, hipStream_t s);

}  // namespace ptpc
