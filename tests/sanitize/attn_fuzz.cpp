// Host half of the attention operators under AddressSanitizer / UBSan.
//
// Built with g++ from attn_api.cpp and attn_plan.cpp plus the stub launchers
// below, which check what validation must guarantee before anything is
// enqueued and walk the launch plan of the call.  main() calls every entry
// point over a grid of extents, pitches and pointers with negative, zero,
// misaligned, boundary and extreme values.
#include <cstdint>
#include <cstdio>

#include "attn.h"
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

static void check_cache(const CacheView& c) {
    REQUIRE(c.pages >= 0 && c.kv_heads >= 1 && c.page_shift >= 4 && c.page_shift <= 16);
    REQUIRE(c.D == 64 || c.D == 128);
    if (c.pages > 0) {
        REQUIRE(c.k && c.v && al(c.k, 16) && al(c.v, 16));
        if (c.fp8) REQUIRE(c.dk && c.dv);
    }
}

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t) {
    ++g_launches;
    check_cache(a.cache);
    REQUIRE(a.T >= 1 && a.T <= (1 << 24) && a.q_heads >= 0 && a.k && a.v && a.positions && a.slots);
    REQUIRE(a.T * (a.q_heads + 2 * (int64_t)a.cache.kv_heads) <= kMaxRowHeads);
    REQUIRE(a.rot_dim % 16 == 0 && a.rot_dim <= a.cache.D && (a.rot_dim == 0 || a.n_pos == 0 || a.table));
    REQUIRE(a.ldk >= a.cache.kv_heads * a.cache.D && a.ldk % 8 == 0 && al(a.k, 16));
    if (a.q_heads) REQUIRE(a.q && a.q_out && a.ldq >= a.q_heads * a.cache.D && a.ldqo % 8 == 0);
    return hipSuccess;
}

static void check_attn(const AttnArgs& a) {
    ++g_launches;
    REQUIRE(a.T >= 1 && a.B >= 1 && a.q && a.out && a.cu && a.ldq % 8 == 0 && a.ldo % 8 == 0);
    REQUIRE(a.q_heads % a.kv_heads == 0 && (a.D == 64 || a.D == 128));
}

hipError_t launch_attn_paged(const AttnArgs& a, hipStream_t) {
    check_attn(a);
    check_cache(a.cache);
    REQUIRE(a.kv_lens && a.table_keys >= 0 && (a.table_keys == 0 || a.page_table));
    const PagedPlan p = paged_plan(a.T, a.B, a.max_q, a.max_kv, a.q_heads, a.cache);
    REQUIRE(p.splits >= 1 && p.splits <= kMaxSplits && p.workspace >= 0);
    REQUIRE((p.workspace > 0) == (p.splits > 1));
    REQUIRE(p.workspace == 0 || a.ws != nullptr);
    REQUIRE(p.blocks >= 1 && p.blocks <= kMaxBlocks);
    // the join's grid: a workgroup of 256 threads for four rows
    if (p.splits > 1) REQUIRE(p.items * p.tile_rows / 4 + 1 < (int64_t(1) << 24));
    REQUIRE(p.tile_rows >= 1 && p.row_tiles >= 1 && p.chunk >= 128 && p.chunk % 128 == 0);
    REQUIRE(p.splits == 1 || (int64_t)p.chunk * p.splits >= a.max_kv);
    return hipSuccess;
}

hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t) {
    check_attn(a);
    REQUIRE(a.k && a.v && a.ldk % 8 == 0 && a.ldv % 8 == 0);
    return hipSuccess;
}

}  // namespace ptpc

static void* ptr(uintptr_t v) { return reinterpret_cast<void*>(v); }

int main() {
    const int64_t ext[] = {INT64_MIN, -1, 0, 1, 3, 4, 64, 100, 128, 1 << 12, (1 << 22) + 8, 1 << 24,
                           (1 << 24) + 1, (int64_t(1) << 31) - 1, int64_t(1) << 31, INT64_MAX};
    void* const ptrs[] = {nullptr, ptr(0x10000), ptr(0x10008), ptr(0x10001)};
    long calls = 0, ok = 0;
    auto count = [&](ptpc_status st, long before) {
        ++calls;
        REQUIRE(st >= PTPC_OK && st <= PTPC_ERR_HIP);
        if (st != PTPC_OK) REQUIRE(g_launches == before);
        ok += g_launches != before;
    };
    void* const P = ptr(0x10000);
    for (int64_t a : ext)
        for (int64_t b : ext)
            for (int v = 0; v < 14; ++v)
                for (void* p : ptrs) {
                    ptpc_kv_cache c{P, P, nullptr, nullptr, 4, 2, 16, 128, 0};
                    int64_t T = 3, B = 2, mq = 2, mk = 700, hq = 4, ld = 512, ldt = 8, wid = 8, rot = 64;
                    void *q = P, *o = P, *i = P;
                    switch (v) {
                        case 0: T = a; B = b; q = p; break;
                        case 1: mq = a; mk = b; o = p; break;
                        case 2: hq = a; ld = b; i = p; break;
                        case 3: c.pages = a; c.kv_heads = b; c.k = p; break;
                        case 4: c.page_size = a; c.head_dim = b; c.v = p; break;
                        case 5: c.fp8 = 1; c.dk = (float*)p; c.dv = (float*)P; T = a; mk = b; break;
                        case 6: ldt = a; wid = b; i = p; break;
                        case 7: rot = a; T = b; q = p; break;
                        case 8: T = a; hq = b; ld = 1 << 19; break;
                        case 9: B = a; mk = b; T = 1 << 24; break;
                        case 10: mq = a; hq = b; ld = 1 << 19; B = 1; break;
                        case 11: c.head_dim = 64; hq = a; mk = b; ld = 1 << 19; break;
                        case 12: c.kv_heads = a; hq = b; ld = 1 << 19; break;
                        default: c.page_size = 1 << 16; wid = ldt = a; mk = b; break;
                    }
                    long n = g_launches;
                    count(ptpc_rope_append(q, ld, i, ld, P, ld, (float*)P, 10, rot, v & 1, (int32_t*)P,
                                           (int64_t*)P, T, hq, &c, o, ld, nullptr), n);
                    const size_t need = ptpc_attn_paged_workspace_bytes(T, B, mq, mk, hq, &c);
                    n = g_launches;
                    count(ptpc_attn_paged(q, ld, (int32_t*)i, &c, (int32_t*)P, ldt, wid, (int32_t*)P, T,
                                          B, mq, mk, hq, 0.1f, o, ld, P, need, nullptr), n);
                    n = g_launches;
                    count(ptpc_attn_prompt(q, ld, i, ld, P, ld, (int32_t*)P, T, B, hq, 2, rot == 64 ? 128 : rot, 0.1f,
                                           o, ld, nullptr), n);
                }
    std::printf("%ld calls, %ld launches, %ld failures\n", calls, ok, g_fail);
    return g_fail ? 1 : 0;
}
