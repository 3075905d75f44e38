// C ABI of the block-scaled FP8 operators and the experts: argument validation
// on the host, then kernel launches on the caller's stream (contract:
// include/ptpc.h).
#include "ptpc.h"

#include <hip/hip_runtime.h>

#include <cstdlib>
#include <cstring>

#include "block.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// PTPC_FAULT=launch in the environment: every call that would launch work
// returns PTPC_ERR_HIP instead (error-path tests, as for the GEMM calls).
bool forced_launch_failure() {
    const char* f = std::getenv("PTPC_FAULT");
    return f != nullptr && std::strcmp(f, "launch") == 0;
}

ptpc_status from_hip(hipError_t e) { return e == hipSuccess ? PTPC_OK : PTPC_ERR_HIP; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// The limits of the other GEMM calls: tiles are addressed with 32-bit offsets,
// tile counts and rows stay in 32 bits.
constexpr int64_t kMaxK = int64_t(1) << 17;
constexpr int64_t kMaxPitch = int64_t(1) << 22;
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxOutputs = int64_t(1) << 36;
constexpr int64_t kMaxPairs = int64_t(1) << 28;
constexpr int64_t kMaxScaleBlocks = int64_t(1) << 24;
// Scales of one row of tokens are addressed in 64 bits; the pitch is bounded
// only to keep products in range.
constexpr int64_t kMaxScalePitch = int64_t(1) << 28;
// Rows that a gather reaches with one 32-bit offset.
constexpr int64_t kMaxGather = int64_t(1) << 31;
constexpr int64_t kMaxTopK = 64;

ptpc_status check_weight(int64_t E, int64_t Ci, int64_t Co) {
    if (E < 0 || Ci < 0 || Co < 0) return PTPC_ERR_SHAPE;
    if (E > ptpc::kMaxExperts || Ci % 16 != 0 || Co % 16 != 0 || Ci > kMaxK || Co > kMaxRows ||
        E * ptpc::scale_blocks(Ci) * ptpc::scale_blocks(Co) > kMaxScaleBlocks)
        return PTPC_ERR_UNSUPPORTED;
    return PTPC_OK;
}

// What both products check: `T` rows of qx, `R` rows of out.
ptpc_status check_product(const uint8_t* qx, int64_t ldq, const float* sx, int64_t lds,
                          const void* wp, const float* sw, int64_t T, int64_t R, int64_t E,
                          int64_t Ci, int64_t Co, const void* out, int64_t ldo) {
    if (T < 0 || R < 0 || ldq < Ci || ldo < Co || lds < T) return PTPC_ERR_SHAPE;
    const ptpc_status st = check_weight(E, Ci, Co);
    if (st != PTPC_OK) return st;
    if (T > kMaxRows || R > kMaxRows || ldq > kMaxPitch || ldo > kMaxPitch ||
        lds > kMaxScalePitch || R * Co > kMaxOutputs)
        return PTPC_ERR_UNSUPPORTED;
    if (R == 0 || Co == 0 || E == 0) return PTPC_OK;
    if (out == nullptr || (Ci > 0 && T > 0 && (qx == nullptr || sx == nullptr)) ||
        (Ci > 0 && (wp == nullptr || sw == nullptr)))
        return PTPC_ERR_NULL;
    if (!aligned(out, 16) || ldo % 8 != 0 ||
        (Ci > 0 && (!aligned(qx, 16) || !aligned(wp, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
                    ldq % 16 != 0)))
        return PTPC_ERR_ALIGN;
    return PTPC_OK;
}

}  // namespace

extern "C" {

ptpc_status ptpc_quant_act_block(const void* x, int64_t T, int64_t Ci, int64_t ldx, int gate,
                                 const int32_t* count, uint8_t* qx, int64_t ldq, float* sx,
                                 int64_t lds, void* stream) {
    if (T < 0 || Ci < 0 || ldx < Ci || ldq < Ci || lds < T) return PTPC_ERR_SHAPE;
    if (Ci % 16 != 0 || T > kMaxRows || ldx > kMaxPitch || ldq > kMaxPitch || lds > kMaxScalePitch)
        return PTPC_ERR_UNSUPPORTED;
    if (gate && ldx < 2 * Ci) return PTPC_ERR_SHAPE;
    if (T == 0 || Ci == 0) return PTPC_OK;
    if (x == nullptr || qx == nullptr || sx == nullptr) return PTPC_ERR_NULL;
    if (!aligned(x, 16) || !aligned(qx, 16) || !aligned(sx, 4) || !aligned(count, 4) ||
        ldx % 8 != 0 || ldq % 16 != 0)
        return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    return from_hip(ptpc::launch_quant_act_block(static_cast<const uint16_t*>(x), T, Ci, ldx,
                                                 gate != 0, count, qx, ldq, sx, lds,
                                                 as_stream(stream)));
}

ptpc_status ptpc_quant_weight_block(const void* w, int64_t E, int64_t Ci, int64_t Co, int64_t ldw,
                                    int64_t we, void* w_packed, float* sw, void* stream) {
    if (ldw < Co || we < 0) return PTPC_ERR_SHAPE;
    const ptpc_status st = check_weight(E, Ci, Co);
    if (st != PTPC_OK) return st;
    if (ldw > kMaxPitch) return PTPC_ERR_UNSUPPORTED;
    if (E == 0 || Ci == 0 || Co == 0) return PTPC_OK;
    if (w == nullptr || w_packed == nullptr || sw == nullptr) return PTPC_ERR_NULL;
    if (!aligned(w, 16) || !aligned(w_packed, 16) || !aligned(sw, 4) || ldw % 8 != 0 ||
        (E > 1 && we % 8 != 0))
        return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    return from_hip(ptpc::launch_quant_weight_block(static_cast<const uint16_t*>(w), E, Ci, Co, ldw,
                                                    E > 1 ? we : 0,
                                                    static_cast<uint8_t*>(w_packed), sw,
                                                    as_stream(stream)));
}

ptpc_status ptpc_pack_weight_block(const uint8_t* codes, int64_t ce, int64_t ck, int64_t co,
                                   const float* scales, int64_t se, int64_t sk, int64_t so,
                                   int64_t E, int64_t Ci, int64_t Co, void* w_packed, float* sw,
                                   void* stream) {
    if (ce < 0 || ck < 0 || co < 0 || se < 0 || sk < 0 || so < 0) return PTPC_ERR_SHAPE;
    const ptpc_status st = check_weight(E, Ci, Co);
    if (st != PTPC_OK) return st;
    if ((ck != 1 && co != 1) || ck > kMaxRows || co > kMaxRows || sk > kMaxRows || so > kMaxRows ||
        ce > (int64_t(1) << 42) || se > (int64_t(1) << 42))
        return PTPC_ERR_UNSUPPORTED;
    if (E == 0 || Ci == 0 || Co == 0) return PTPC_OK;
    if (codes == nullptr || scales == nullptr || w_packed == nullptr || sw == nullptr)
        return PTPC_ERR_NULL;
    if (!aligned(w_packed, 16) || !aligned(sw, 4) || !aligned(scales, 4)) return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    const ptpc::PackArgs a{codes, ce, ck, co, scales, se, sk, so, E, Ci, Co,
                           static_cast<uint8_t*>(w_packed), sw};
    return from_hip(ptpc::launch_pack_weight_block(a, as_stream(stream)));
}

ptpc_status ptpc_gemm_block(const uint8_t* qx, int64_t ldq, const float* sx, int64_t lds,
                            const void* w_packed, const float* sw, int64_t T, int64_t Ci,
                            int64_t Co, void* out, int64_t ldo, void* stream) {
    const ptpc_status st =
        check_product(qx, ldq, sx, lds, w_packed, sw, T, T, 1, Ci, Co, out, ldo);
    if (st != PTPC_OK || T == 0 || Co == 0) return st;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    const ptpc::BlockGemmArgs a{qx, ldq, sx, lds, static_cast<const uint8_t*>(w_packed), sw, T, T,
                                Ci, Co, static_cast<uint16_t*>(out), ldo, nullptr, nullptr, 1, 1};
    return from_hip(ptpc::launch_block_gemm(a, as_stream(stream)));
}

ptpc_status ptpc_gemm_experts(const uint8_t* qx, int64_t ldq, const float* sx, int64_t lds,
                              const void* w_packed, const float* sw, const int32_t* offsets,
                              const int32_t* rows, int64_t top_k, int64_t E, int64_t T, int64_t R,
                              int64_t Ci, int64_t Co, void* out, int64_t ldo, void* stream) {
    if (rows == nullptr && T != R) return PTPC_ERR_SHAPE;
    const ptpc_status st =
        check_product(qx, ldq, sx, lds, w_packed, sw, T, R, E, Ci, Co, out, ldo);
    if (st != PTPC_OK || R == 0 || Co == 0 || E == 0) return st;
    if (ptpc::block_gemm_grid(ptpc::block_gemm_plan(R, E, Ci, Co), R, E, Co) > ptpc::kMaxGrid ||
        (rows != nullptr && (top_k < 1 || top_k > kMaxTopK || T * ldq > kMaxGather)))
        return PTPC_ERR_UNSUPPORTED;
    if (offsets == nullptr) return PTPC_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(rows, 4)) return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    const ptpc::BlockGemmArgs a{qx, ldq, sx, lds, static_cast<const uint8_t*>(w_packed), sw, R, T,
                                Ci, Co, static_cast<uint16_t*>(out), ldo, offsets, rows,
                                (int32_t)E, (int32_t)(rows != nullptr ? top_k : 1)};
    return from_hip(ptpc::launch_block_gemm(a, as_stream(stream)));
}

size_t ptpc_route_experts_workspace_bytes(int64_t T, int64_t local) {
    if (T <= 0 || local <= 0 || T > kMaxPairs || local > ptpc::kMaxExperts) return 0;
    const ptpc::RoutePlan p = ptpc::route_plan(T);
    return p.chunks > 1 ? (size_t)(p.chunks * local * 4) : 0;
}

ptpc_status ptpc_route_experts(const void* logits, int bf16, int64_t ldl, const float* bias,
                               int64_t T, int64_t E, int64_t top_k, int sigmoid, int64_t groups,
                               int64_t top_groups, int64_t group_top, int renorm, float scale,
                               int64_t first, int64_t local, int32_t* ids, float* weights,
                               int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace,
                               size_t workspace_bytes, void* stream) {
    if (T < 0 || E < 0 || top_k < 0 || ldl < E || groups < 1 || top_groups < 1 ||
        top_groups > groups || first < 0 || local < 0 || first > E || local > E - first)
        return PTPC_ERR_SHAPE;
    if (E < 1 || E > ptpc::kMaxExperts || top_k < 1 || top_k > kMaxTopK || local < 1 ||
        groups > 64 || E % groups != 0 || top_k > top_groups * (E / groups) || group_top < 1 ||
        group_top > 2 || ldl > kMaxPitch || T > kMaxPairs || T * top_k > kMaxPairs)
        return PTPC_ERR_UNSUPPORTED;
    if (offsets == nullptr ||
        (T > 0 && (logits == nullptr || ids == nullptr || weights == nullptr || rows == nullptr ||
                   slots == nullptr)))
        return PTPC_ERR_NULL;
    if (!aligned(logits, bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) ||
        !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
        return PTPC_ERR_ALIGN;
    const size_t need = ptpc_route_experts_workspace_bytes(T, local);
    if (need > 0) {
        if (workspace == nullptr) return PTPC_ERR_NULL;
        if (workspace_bytes < need) return PTPC_ERR_SHAPE;
        if (!aligned(workspace, 16)) return PTPC_ERR_ALIGN;
    }
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    const ptpc::RouteArgs a{logits, bf16 != 0, ldl, bias, T, (int32_t)E, (int32_t)top_k,
                            sigmoid != 0, renorm != 0, (int32_t)groups, (int32_t)top_groups,
                            (int32_t)group_top, scale, (int32_t)first, (int32_t)local, ids, weights,
                            offsets, rows, slots, static_cast<int32_t*>(workspace)};
    return from_hip(ptpc::launch_route(a, as_stream(stream)));
}

ptpc_status ptpc_combine_experts(const void* y, int64_t ldy, int64_t R, const int32_t* slots,
                                 const float* weights, int64_t T, int64_t top_k, int64_t C,
                                 void* out, int64_t ldo, void* stream) {
    if (R < 0 || T < 0 || top_k < 0 || C < 0 || ldy < C || ldo < C) return PTPC_ERR_SHAPE;
    if (C % 16 != 0 || R > kMaxPairs || T > kMaxPairs || top_k < 1 || top_k > kMaxTopK ||
        T * top_k > kMaxPairs || ldy > kMaxPitch || ldo > kMaxPitch || T * C > kMaxOutputs)
        return PTPC_ERR_UNSUPPORTED;
    if (T == 0 || C == 0) return PTPC_OK;
    if (slots == nullptr || weights == nullptr || out == nullptr || (R > 0 && y == nullptr))
        return PTPC_ERR_NULL;
    if (!aligned(y, 16) || !aligned(out, 16) || ldy % 8 != 0 || ldo % 8 != 0 ||
        !aligned(slots, 4) || !aligned(weights, 4))
        return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    return from_hip(ptpc::launch_combine(static_cast<const uint16_t*>(y), ldy, R, slots, weights, T,
                                         (int32_t)top_k, C, static_cast<uint16_t*>(out), ldo,
                                         as_stream(stream)));
}

const char* ptpc_gemm_block_kernel(int64_t R, int64_t E, int64_t Ci, int64_t Co) {
    if (R < 1 || E < 0 || Co < 1 || R > kMaxRows || check_weight(E, Ci, Co) != PTPC_OK ||
        R * Co > kMaxOutputs)
        return nullptr;
    const ptpc::BlockPlan p = ptpc::block_gemm_plan(R, E, Ci, Co);
    if (E > 0 && ptpc::block_gemm_grid(p, R, E, Co) > ptpc::kMaxGrid) return nullptr;
    return ptpc::block_plan_name(p);
}

}  // extern "C"
