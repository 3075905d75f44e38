#include <hip/hip_runtime.h>

#include "attn.h"

namespace ptpc {
hipError_t launch_attn_paged(const AttnArgs& a, hipStream_t s) {
    const PagedPlan p = paged_plan(a.T, a.B, a.max_q, a.max_kv, a.q_heads, a.cache);
    return launch_attn_tiles(a, p, s);
}
}  // namespace ptpc
