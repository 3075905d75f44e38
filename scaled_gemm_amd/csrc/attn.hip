// Attention over a paged cache and over packed prompts.
//
// One wave per (row, query head): it walks the keys the row sees with the
// running maximum and sum of a softmax, a lane holding D/64 channels.
#include <hip/hip_runtime.h>

#include "attn.h"
#include "device_common.h"

namespace ptpc {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Sequence of row t: the last b with cu[b] <= t (B if t is past the end).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int64_t t) {
    int lo = 0, hi = B;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (cu[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
    return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

template <int D, bool PAGED, bool FP8>
__global__ __launch_bounds__(64) void attn_rows_kernel(AttnArgs a) {
    constexpr int C = D / 64;
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y;
    const int hk = h / (a.q_heads / a.kv_heads);
    const int b = find_sequence(a.cu, a.B, t);
    uint16_t* out = a.out + t * a.ldo + (int64_t)h * D + lane * C;
    int64_t seen = 0, base = 0;
    if (b < a.B) {
        base = a.cu[b];
        if (PAGED) {
            int64_t n = a.kv_lens[b];
            n = n < 0 ? 0 : n > a.table_keys ? a.table_keys : n;
            seen = n - (a.cu[b + 1] - t) + 1;
        } else {
            base = base < 0 ? 0 : base;
            seen = t - base + 1;
        }
    }
    float q[C], acc[C], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        q[c] = __uint_as_float((uint32_t)a.q[t * a.ldq + (int64_t)h * D + lane * C + c] << 16);
        acc[c] = 0.0f;
    }
    for (int64_t j = 0; j < seen; ++j) {
        float k[C], v[C], dk = 1.0f, dv = 1.0f;
        if (PAGED) {
            int64_t page = a.page_table[(int64_t)b * a.ld_table + (j >> a.cache.page_shift)];
            page = page < 0 || page >= a.cache.pages ? 0 : page;
            const int64_t row = ((page * a.kv_heads + hk) << a.cache.page_shift) |
                                (j & ((1 << a.cache.page_shift) - 1));
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t e = row * D + lane * C + c;
                if (FP8) {
                    k[c] = e4m3_to_f32(a.cache.k[e]);
                    v[c] = e4m3_to_f32(a.cache.v[e]);
                } else {
                    k[c] = __uint_as_float((uint32_t)((const uint16_t*)a.cache.k)[e] << 16);
                    v[c] = __uint_as_float((uint32_t)((const uint16_t*)a.cache.v)[e] << 16);
                }
            }
            if (FP8) {
                dk = a.cache.dk[row];
                dv = a.cache.dv[row];
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t e = (int64_t)hk * D + lane * C + c;
                k[c] = __uint_as_float((uint32_t)a.k[(base + j) * a.ldk + e] << 16);
                v[c] = __uint_as_float((uint32_t)a.v[(base + j) * a.ldv + e] << 16);
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) dot += q[c] * k[c];
        const float s = wave_sum(dot) * dk * a.scale;
        const float mn = fmaxf(m, s);
        const float shift = mn == -INFINITY ? 0.0f : mn;
        const float r = expf(m - shift), w = expf(s - shift);
        l = l * r + w;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = acc[c] * r + w * dv * v[c];
        m = mn;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const float o = seen > 0 ? acc[c] / l : 0.0f;
        out[c] = (uint16_t)f32x2_to_bf16x2_rne(o, 0.0f);
    }
}

template <bool PAGED, bool FP8>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.T, (unsigned)a.q_heads);
    if (a.D == 128) attn_rows_kernel<128, PAGED, FP8><<<grid, 64, 0, s>>>(a);
    else attn_rows_kernel<64, PAGED, FP8><<<grid, 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t attn_paged_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, const CacheView&) {
    return 0;
}

hipError_t launch_attn_paged(const AttnArgs& a, hipStream_t s) {
    return a.cache.fp8 ? launch<true, true>(a, s) : launch<true, false>(a, s);
}

hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t s) {
    return launch<false, false>(a, s);
}

}  // namespace ptpc
