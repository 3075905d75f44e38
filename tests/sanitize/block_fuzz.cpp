// Host half of the block-scaled operators and the experts under AddressSanitizer /
// UBSan.
//
// Built with g++ from block_api.cpp and block_plan.cpp plus the stub launchers
// below, which check what validation must guarantee before anything is enqueued.
// main() calls every entry point over a grid of extents, pitches and pointers with
// negative, zero, misaligned, boundary and extreme values.
#include <cstdint>
#include <cstdio>

#include "block.h"
#include "ptpc.h"

static long g_launches = 0, g_fail = 0;

#define REQUIRE(c)                                                                         \
    do {                                                                                   \
        if (!(c)) {                                                                        \
            std::fprintf(stderr, "%s:%d: requirement failed: %s\n", __FILE__, __LINE__, #c); \
            ++g_fail;                                                                      \
        }                                                                                  \
    } while (0)

static bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

namespace ptpc {

hipError_t launch_quant_act_block(const uint16_t* x, int64_t T, int64_t C, int64_t ldx, bool gate,
                                  const int32_t* count, uint8_t* qx, int64_t ldq, float* sx,
                                  int64_t lds, hipStream_t) {
    ++g_launches;
    REQUIRE(x && qx && sx && al(x, 16) && al(qx, 16) && al(sx, 4) && al(count, 4));
    REQUIRE(T >= 1 && T <= (1 << 24) && C >= 16 && C % 16 == 0 && lds >= T);
    REQUIRE(ldx >= C * (gate ? 2 : 1) && ldx % 8 == 0 && ldx <= (1 << 22));
    REQUIRE(ldq >= C && ldq % 16 == 0 && ldq <= (1 << 22));
    return hipSuccess;
}

hipError_t launch_quant_weight_block(const uint16_t* w, int64_t E, int64_t Ci, int64_t Co,
                                     int64_t ldw, int64_t se, uint8_t* packed, float* sw,
                                     hipStream_t) {
    ++g_launches;
    REQUIRE(w && packed && sw && al(w, 16) && al(packed, 16) && ldw >= Co && ldw % 8 == 0);
    REQUIRE(E >= 1 && E <= kMaxExperts && se >= 0 && se % 8 == 0);
    REQUIRE(Ci >= 16 && Ci % 16 == 0 && Ci <= (1 << 17) && Co >= 16 && Co % 16 == 0);
    REQUIRE(E * scale_blocks(Ci) * scale_blocks(Co) <= (1 << 24));
    return hipSuccess;
}

hipError_t launch_pack_weight_block(const PackArgs& a, hipStream_t) {
    ++g_launches;
    REQUIRE(a.codes && a.scales && a.packed && a.sw && al(a.packed, 16) && al(a.scales, 4));
    REQUIRE((a.sk == 1 || a.so == 1) && a.se >= 0 && a.sk >= 0 && a.so >= 0);
    REQUIRE(a.te >= 0 && a.tk >= 0 && a.to >= 0);
    REQUIRE(a.E * scale_blocks(a.Ci) * scale_blocks(a.Co) <= (1 << 24));
    return hipSuccess;
}

hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t) {
    ++g_launches;
    REQUIRE(a.T >= 1 && a.T <= (1 << 24) && a.T_in >= 0 && a.out && al(a.out, 16));
    REQUIRE(a.Co >= 16 && a.Co % 16 == 0 && a.Ci >= 0 && a.Ci <= (1 << 17));
    REQUIRE(a.ldo >= a.Co && a.ldo % 8 == 0 && 256 * a.ldo * 2 <= (int64_t(1) << 31));
    if (a.Ci > 0) {
        REQUIRE(a.wp && a.sw && al(a.wp, 16) && a.ldq % 16 == 0 && a.ldq >= a.Ci);
        if (a.T_in > 0) REQUIRE(a.qx && a.sx && al(a.qx, 16) && a.lds >= a.T_in);
    }
    if (a.offsets) {
        REQUIRE(a.E >= 1 && a.E <= kMaxExperts && a.top_k >= 1);
        REQUIRE(a.rows ? a.T_in * a.ldq <= (int64_t(1) << 31) : a.T_in == a.T);
    }
    const BlockPlan p = block_gemm_plan(a.T, a.offsets ? a.E : 0, a.Ci, a.Co);
    const int64_t n = block_gemm_grid(p, a.T, a.offsets ? a.E : 0, a.Co);
    REQUIRE(n >= 1 && n <= kMaxGrid && block_plan_name(p) != nullptr);
    REQUIRE(p != BlockPlan::kFew || (!a.offsets && a.T <= kFewRows16));
    return hipSuccess;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t) {
    ++g_launches;
    REQUIRE(a.T >= 0 && a.T * a.K <= (1 << 28) && a.E >= 1 && a.E <= kMaxExperts);
    REQUIRE(a.K >= 1 && a.K <= 64 && a.groups >= 1 && a.groups <= 64 && a.E % a.groups == 0);
    REQUIRE(a.top_groups >= 1 && a.top_groups <= a.groups && a.K <= a.top_groups * (a.E / a.groups));
    REQUIRE(a.first >= 0 && a.local >= 1 && a.first + a.local <= a.E && a.offsets);
    if (a.T > 0) REQUIRE(a.logits && a.ids && a.weights && a.rows && a.slots && a.ldl >= a.E);
    const RoutePlan p = route_plan(a.T);
    REQUIRE(p.chunks >= 1 && p.chunks <= kRouteMaxChunks && p.chunk * p.chunks >= a.T);
    REQUIRE(p.chunks > 1 || p.chunk <= 16);
    REQUIRE(p.chunks == 1 || a.ws != nullptr);
    return hipSuccess;
}

hipError_t launch_combine(const uint16_t* y, int64_t ldy, int64_t R, const int32_t* slots,
                          const float* weights, int64_t T, int32_t K, int64_t C, uint16_t* out,
                          int64_t ldo, hipStream_t) {
    ++g_launches;
    REQUIRE(T >= 1 && K >= 1 && C >= 16 && C % 16 == 0 && slots && weights && out && al(out, 16));
    REQUIRE(R >= 0 && (R == 0 || (y && al(y, 16))) && ldy >= C && ldy % 8 == 0 && ldo % 8 == 0);
    return hipSuccess;
}

}  // namespace ptpc

static void* ptr(uintptr_t v) { return reinterpret_cast<void*>(v); }

int main() {
    const int64_t ext[] = {INT64_MIN, -1, 0, 1, 2, 16, 24, 128, 400, 513, 1 << 12, 1 << 17, 1 << 19,
                           (1 << 22) + 16, 1 << 24, (1 << 24) + 16, int64_t(1) << 28,
                           int64_t(1) << 31, INT64_MAX};
    void* const ptrs[] = {nullptr, ptr(0x10000), ptr(0x10008), ptr(0x10001)};
    long calls = 0, ok = 0;
    auto count = [&](ptpc_status st, long before) {
        ++calls;
        REQUIRE(st >= PTPC_OK && st <= PTPC_ERR_HIP);
        if (st != PTPC_OK) REQUIRE(g_launches == before);
        ok += g_launches != before;
    };
    void* const P = ptr(0x10000);
    float* const F = (float*)P;
    int32_t* const I = (int32_t*)P;
    for (int64_t a : ext)
        for (int64_t b : ext)
            for (int v = 0; v < 16; ++v)
                for (void* p : ptrs) {
                    int64_t T = 48, R = 96, K = 2, E = 8, Ci = 400, Co = 272, ldq = 512, ldx = 1024,
                            lds = 64, ldo = 512, groups = 4, top = 2, gt = 2, first = 0, local = 8,
                            step = 1;
                    void *x = P, *q = P, *s = P, *w = P, *o = P, *i = P;
                    switch (v) {
                        case 0: T = a; Ci = b; x = p; break;
                        case 1: T = a; lds = b; q = p; break;
                        case 2: Ci = a; Co = b; w = p; break;
                        case 3: ldq = a; ldx = b; s = p; break;
                        case 4: Co = a; ldo = b; o = p; break;
                        case 5: E = a; Co = b; i = p; break;
                        case 6: R = a; T = b; K = 1; break;
                        case 7: K = a; T = b; i = p; break;
                        case 8: E = a; Ci = b; local = a; w = p; break;
                        case 9: groups = a; top = b; break;
                        case 10: first = a; local = b; s = p; break;
                        case 11: gt = a; E = b; ldx = 1 << 19; break;
                        case 12: step = a; ldx = b; q = p; break;
                        case 13: R = a; Co = b; ldo = 1 << 22; E = 512; break;
                        case 14: T = a; ldq = b; lds = int64_t(1) << 28; break;
                        default: T = a; K = b; local = 1; lds = int64_t(1) << 28; break;
                    }
                    long n = g_launches;
                    count(ptpc_quant_act_block(x, T, Ci, ldx, v & 1, (int32_t*)(v & 2 ? i : nullptr),
                                               (uint8_t*)q, ldq, (float*)s, lds, nullptr), n);
                    n = g_launches;
                    count(ptpc_quant_weight_block(x, E, Ci, Co, ldx, step, w, (float*)s, nullptr), n);
                    n = g_launches;
                    count(ptpc_pack_weight_block((uint8_t*)q, ldx, step, 1, (float*)s, lds, K, groups, E,
                                                 Ci, Co, w, F, nullptr), n);
                    n = g_launches;
                    count(ptpc_gemm_block((uint8_t*)q, ldq, (float*)s, lds, w, F, T, Ci, Co, o, ldo,
                                          nullptr), n);
                    for (int gather = 0; gather < 2; ++gather) {
                        n = g_launches;
                        count(ptpc_gemm_experts((uint8_t*)q, ldq, (float*)s, lds, w, F, (int32_t*)i,
                                                gather ? I : nullptr, K, E, gather ? T : R, R, Ci, Co,
                                                o, ldo, nullptr), n);
                    }
                    const size_t need = ptpc_route_experts_workspace_bytes(T, local);
                    n = g_launches;
                    count(ptpc_route_experts(x, v & 1, ldx, (float*)(v & 2 ? s : nullptr), T, E, K, v & 4,
                                             groups, top, gt, 1, 1.0f, first, local, (int32_t*)q, F,
                                             (int32_t*)i, I, (int32_t*)o, need ? w : nullptr, need,
                                             nullptr), n);
                    n = g_launches;
                    count(ptpc_combine_experts(x, ldx, R, (int32_t*)i, (float*)s, T, K, Ci, o, ldo,
                                               nullptr), n);
                    ptpc_gemm_block_kernel(T, E, Ci, Co);
                }
    std::printf("%ld calls, %ld launches, %ld failures\n", calls, ok, g_fail);
    return g_fail ? 1 : 0;
}
