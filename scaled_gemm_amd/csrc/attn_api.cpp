// C ABI of the attention operators: argument validation on the host, then
// kernel launches on the caller's stream (contract: include/ptpc.h).
#include "ptpc.h"

#include <hip/hip_runtime.h>

#include <cstdlib>
#include <cstring>

#include "attn.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// PTPC_FAULT=launch in the environment: every call that would launch work
// returns PTPC_ERR_HIP instead (error-path tests, as for the GEMM calls).
bool forced_launch_failure() {
    const char* f = std::getenv("PTPC_FAULT");
    return f != nullptr && std::strcmp(f, "launch") == 0;
}

ptpc_status from_hip(hipError_t e) { return e == hipSuccess ? PTPC_OK : PTPC_ERR_HIP; }

// Rows and sequences of one call, its row pitches and head count: grids and
// per-row indices then stay within 32 bits (rows * heads <= 2^36 are only
// ever formed in 64 bits).
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxPitch = int64_t(1) << 22;
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxPages = (int64_t(1) << 31) - 1;
// Keys of one sequence: key indices, some tiles past the end included, stay in 32 bits.
constexpr int64_t kMaxKeys = int64_t(1) << 30;

bool power_of_two(int64_t n) { return n > 0 && (n & (n - 1)) == 0; }

// The cache's extents; its pointers are checked by check_cache_pointers.
ptpc_status check_cache_shape(const ptpc_kv_cache* c) {
    if (c->pages < 0 || c->kv_heads < 0 || c->page_size < 0 || c->head_dim < 0)
        return PTPC_ERR_SHAPE;
    if (c->pages > kMaxPages || c->kv_heads < 1 || c->kv_heads > kMaxHeads ||
        !power_of_two(c->page_size) || c->page_size < 16 || c->page_size > 65536 ||
        (c->head_dim != 64 && c->head_dim != 128) || (c->fp8 != 0 && c->fp8 != 1))
        return PTPC_ERR_UNSUPPORTED;
    return PTPC_OK;
}

ptpc_status check_cache_pointers(const ptpc_kv_cache* c) {
    if (c->k == nullptr || c->v == nullptr || (c->fp8 && (c->dk == nullptr || c->dv == nullptr)))
        return PTPC_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v) || (c->fp8 && (!aligned16(c->dk) || !aligned16(c->dv))))
        return PTPC_ERR_ALIGN;
    return PTPC_OK;
}

ptpc::CacheView view(const ptpc_kv_cache* c) {
    int shift = 0;
    while ((int64_t(1) << shift) < c->page_size) ++shift;
    return {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->dk, c->dv,
            (int32_t)c->pages, (int32_t)c->kv_heads, shift, (int32_t)c->head_dim, c->fp8 != 0};
}

}  // namespace

extern "C" {

ptpc_status ptpc_rope_append(const void* q, int64_t ldq, const void* k, int64_t ldk,
                             const void* v, int64_t ldv, const float* table, int64_t n_pos,
                             int64_t rot_dim, int interleaved, const int32_t* positions,
                             const int64_t* slots, int64_t T, int64_t q_heads,
                             const ptpc_kv_cache* cache, void* q_out, int64_t ldqo,
                             void* stream) {
    if (cache == nullptr) return PTPC_ERR_NULL;
    ptpc_status st = check_cache_shape(cache);
    if (st != PTPC_OK) return st;
    const int64_t D = cache->head_dim, H = cache->kv_heads;
    if (T < 0 || q_heads < 0 || n_pos < 0 || rot_dim < 0 || rot_dim > D) return PTPC_ERR_SHAPE;
    if (T > kMaxRows || q_heads > kMaxHeads || rot_dim % 16 != 0 || ldq > kMaxPitch ||
        ldk > kMaxPitch || ldv > kMaxPitch || ldqo > kMaxPitch || n_pos > kMaxPages ||
        T * (q_heads + 2 * H) > ptpc::kMaxRowHeads)
        return PTPC_ERR_UNSUPPORTED;
    if (ldk < H * D || ldv < H * D || (q_heads > 0 && (ldq < q_heads * D || ldqo < q_heads * D)))
        return PTPC_ERR_SHAPE;
    if (T == 0) return PTPC_OK;
    if (k == nullptr || v == nullptr || positions == nullptr || slots == nullptr ||
        (q_heads > 0 && (q == nullptr || q_out == nullptr)) ||
        (rot_dim > 0 && n_pos > 0 && table == nullptr))
        return PTPC_ERR_NULL;
    if (cache->pages > 0 && (st = check_cache_pointers(cache)) != PTPC_OK) return st;
    if (!aligned16(k) || !aligned16(v) || ldk % 8 != 0 || ldv % 8 != 0 || !aligned16(table) ||
        !aligned(positions, 4) || !aligned(slots, 8) ||
        (q_heads > 0 && (!aligned16(q) || !aligned16(q_out) || ldq % 8 != 0 || ldqo % 8 != 0)))
        return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    const ptpc::RopeArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                           static_cast<const uint16_t*>(v), ldq, ldk, ldv, table, n_pos,
                           (int32_t)rot_dim, interleaved != 0, positions, slots, T,
                           (int32_t)q_heads, view(cache), static_cast<uint16_t*>(q_out), ldqo};
    return from_hip(ptpc::launch_rope_append(a, reinterpret_cast<hipStream_t>(stream)));
}

// Extents common to both attention calls.
static ptpc_status check_attn(int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D,
                              int64_t ldq, int64_t ldo) {
    if (T < 0 || B < 0 || q_heads < 0 || kv_heads < 0 || D < 0) return PTPC_ERR_SHAPE;
    if (T > kMaxRows || B > kMaxRows || q_heads < 1 || kv_heads < 1 || q_heads > kMaxHeads ||
        q_heads % kv_heads != 0 || (D != 64 && D != 128) || ldq > kMaxPitch || ldo > kMaxPitch ||
        T * q_heads > ptpc::kMaxRowHeads || B * kv_heads > ptpc::kMaxPairs)
        return PTPC_ERR_UNSUPPORTED;
    if (ldq < q_heads * D || ldo < q_heads * D) return PTPC_ERR_SHAPE;
    return PTPC_OK;
}

size_t ptpc_attn_paged_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t max_kv,
                                       int64_t q_heads, const ptpc_kv_cache* cache) {
    if (cache == nullptr || check_cache_shape(cache) != PTPC_OK || T <= 0 || B <= 0 ||
        max_q <= 0 || max_kv <= 0 || max_kv > kMaxKeys ||
        check_attn(T, B, q_heads, cache->kv_heads, cache->head_dim, kMaxPitch, kMaxPitch) !=
            PTPC_OK)
        return 0;
    return ptpc::attn_paged_workspace(T, B, max_q, max_kv, q_heads, view(cache));
}

ptpc_status ptpc_attn_paged(const void* q, int64_t ldq, const int32_t* cu_q,
                            const ptpc_kv_cache* cache, const int32_t* page_table,
                            int64_t ld_table, int64_t table_pages, const int32_t* kv_lens,
                            int64_t T, int64_t B, int64_t max_q, int64_t max_kv,
                            int64_t q_heads, float scale, void* out, int64_t ldo,
                            void* workspace, size_t workspace_bytes, void* stream) {
    if (cache == nullptr) return PTPC_ERR_NULL;
    ptpc_status st = check_cache_shape(cache);
    if (st != PTPC_OK) return st;
    st = check_attn(T, B, q_heads, cache->kv_heads, cache->head_dim, ldq, ldo);
    if (st != PTPC_OK) return st;
    if (max_q < 0 || max_kv < 0 || table_pages < 0 || ld_table < table_pages)
        return PTPC_ERR_SHAPE;
    if (max_kv > kMaxKeys || ld_table > kMaxPages) return PTPC_ERR_UNSUPPORTED;
    if (T == 0 || B == 0) return PTPC_OK;
    if (q == nullptr || cu_q == nullptr || kv_lens == nullptr || out == nullptr ||
        (table_pages > 0 && page_table == nullptr))
        return PTPC_ERR_NULL;
    // a cache without pages holds no keys: every row is zero
    const int64_t keys = cache->pages == 0 ? 0 : table_pages * cache->page_size;
    if (cache->pages > 0 && (st = check_cache_pointers(cache)) != PTPC_OK) return st;
    if (!aligned16(q) || !aligned16(out) || ldq % 8 != 0 || ldo % 8 != 0 || !aligned(cu_q, 4) ||
        !aligned(kv_lens, 4) || !aligned(page_table, 4))
        return PTPC_ERR_ALIGN;
    const size_t need = ptpc_attn_paged_workspace_bytes(T, B, max_q, max_kv, q_heads, cache);
    if (need > 0) {
        if (workspace == nullptr) return PTPC_ERR_NULL;
        if (workspace_bytes < need) return PTPC_ERR_SHAPE;
        if (!aligned16(workspace)) return PTPC_ERR_ALIGN;
    }
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    ptpc::AttnArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.ldq = ldq;
    a.cu = cu_q;
    a.T = T;
    a.B = (int32_t)B;
    a.q_heads = (int32_t)q_heads;
    a.kv_heads = (int32_t)cache->kv_heads;
    a.D = (int32_t)cache->head_dim;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ldo = ldo;
    a.cache = view(cache);
    a.page_table = page_table;
    a.ld_table = ld_table;
    a.table_keys = (int32_t)(keys < kMaxKeys ? keys : kMaxKeys);
    a.kv_lens = kv_lens;
    a.max_q = max_q;
    a.max_kv = max_kv;
    a.ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
    return from_hip(ptpc::launch_attn_paged(a, reinterpret_cast<hipStream_t>(stream)));
}

ptpc_status ptpc_attn_prompt(const void* q, int64_t ldq, const void* k, int64_t ldk,
                             const void* v, int64_t ldv, const int32_t* cu, int64_t T,
                             int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                             float scale, void* out, int64_t ldo, void* stream) {
    ptpc_status st = check_attn(T, B, q_heads, kv_heads, head_dim, ldq, ldo);
    if (st != PTPC_OK) return st;
    if (ldk > kMaxPitch || ldv > kMaxPitch) return PTPC_ERR_UNSUPPORTED;
    if (ldk < kv_heads * head_dim || ldv < kv_heads * head_dim) return PTPC_ERR_SHAPE;
    if (T == 0 || B == 0) return PTPC_OK;
    if (q == nullptr || k == nullptr || v == nullptr || cu == nullptr || out == nullptr)
        return PTPC_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || ldq % 8 != 0 ||
        ldk % 8 != 0 || ldv % 8 != 0 || ldo % 8 != 0 || !aligned(cu, 4))
        return PTPC_ERR_ALIGN;
    if (forced_launch_failure()) return PTPC_ERR_HIP;
    ptpc::AttnArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.ldq = ldq;
    a.cu = cu;
    a.T = T;
    a.B = (int32_t)B;
    a.q_heads = (int32_t)q_heads;
    a.kv_heads = (int32_t)kv_heads;
    a.D = (int32_t)head_dim;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ldo = ldo;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.ldk = ldk;
    a.ldv = ldv;
    return from_hip(ptpc::launch_attn_prompt(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
