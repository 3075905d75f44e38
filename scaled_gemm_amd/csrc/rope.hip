// Rotation of new tokens' queries and keys, and appending keys and values to
// the paged cache, in one pass.
//
// A head is D/16 lanes of two 16-byte units (8 bf16 channels each): the two
// units a lane holds are the halves of eight rotated pairs, so the rotation
// needs no exchange between lanes, and an E4M3 head's amax is a butterfly
// over D/16 lanes.  The q_heads + 2 kv_heads
// heads of a token are consecutive lane groups.  Codes are divided by their scale in
// IEEE division: the values are rotated fp32 numbers, not the bf16 ones the
// quantizer's faster division is proven for.
//
// What bounds it: HBM for large batches (8192 tokens, 64 + 8 heads, E4M3 cache, 324 MB:
// 63 us, 5.1 TB/s, at the 5.0 TB/s of a device copy), the launch and four dependent
// loads for small ones (32 tokens: 3.2 us).
#include <hip/hip_runtime.h>

#include "attn.h"
#include "device_common.h"

namespace ptpc {
namespace {

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    x[0] = bf16lo_to_f32(w.x); x[1] = bf16hi_to_f32(w.x);
    x[2] = bf16lo_to_f32(w.y); x[3] = bf16hi_to_f32(w.y);
    x[4] = bf16lo_to_f32(w.z); x[5] = bf16hi_to_f32(w.z);
    x[6] = bf16lo_to_f32(w.w); x[7] = bf16hi_to_f32(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(f32x2_to_bf16x2_rne(x[0], x[1]), f32x2_to_bf16x2_rne(x[2], x[3]),
                      f32x2_to_bf16x2_rne(x[4], x[5]), f32x2_to_bf16x2_rne(x[6], x[7]));
}

// One pair's rotation: every product and sum rounded by itself (contraction
// is off for the whole library).
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
    const float ra = a * c - b * s;
    const float rb = b * c + a * s;
    a = ra;
    b = rb;
}

// Eight fp32 values / scale -> eight E4M3 codes (IEEE division: the values are
// rotated fp32 numbers, not bf16).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    uint32_t lo = 0, hi = 0;
    lo = cvt_e4m3x2<false>(x[0] / scale, x[1] / scale, lo);
    lo = cvt_e4m3x2<true>(x[2] / scale, x[3] / scale, lo);
    hi = cvt_e4m3x2<false>(x[4] / scale, x[5] / scale, hi);
    hi = cvt_e4m3x2<true>(x[6] / scale, x[7] / scale, hi);
    return make_uint2(lo, hi);
}

// NL: lanes per head (D / 16).
template <int NL, bool INTERLEAVED, bool FP8>
__global__ __launch_bounds__(256) void rope_append_kernel(RopeArgs a) {
    constexpr int D = NL * 16;
    const int lane = threadIdx.x % NL;                        // within the head
    const int heads = a.q_heads + 2 * a.cache.kv_heads;
    const int64_t item = (int64_t)blockIdx.x * (256 / NL) + threadIdx.x / NL;
    if (item >= a.T * heads) return;
    const int64_t t = item / heads;
    const int h = (int)(item - t * heads);
    const bool is_q = h < a.q_heads;
    const bool is_v = h >= a.q_heads + a.cache.kv_heads;

    // the lane's units: halves of rotated pairs, or two plain neighbours
    const int rl = a.rot_dim / 16;                            // lanes that rotate
    const bool turns = lane < rl && !is_v;
    int u0 = 2 * lane, u1 = 2 * lane + 1;
    if (!INTERLEAVED && lane < rl) {
        u0 = lane;
        u1 = lane + rl;
    }
    const int hk = is_q ? h : is_v ? h - a.q_heads - a.cache.kv_heads : h - a.q_heads;
    const uint16_t* src = is_q   ? a.q + t * a.ldq + (int64_t)hk * D
                          : is_v ? a.v + t * a.ldv + (int64_t)hk * D
                                 : a.k + t * a.ldk + (int64_t)hk * D;
    const uint4 w0 = *reinterpret_cast<const uint4*>(src + 8 * u0);
    const uint4 w1 = *reinterpret_cast<const uint4*>(src + 8 * u1);
    const int64_t slot = is_q ? -1 : a.slots[t];
    float x[8], y[8];
    unpack8(w0, x);
    unpack8(w1, y);
    if (turns) {
        const int64_t pos = a.positions[t];
        const bool known = pos >= 0 && pos < a.n_pos;
        const float* row = a.table + (known ? pos : 0) * a.rot_dim + 8 * lane;
        float c[8], s[8];
        if (known) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 cc = reinterpret_cast<const float4*>(row)[i];
                const float4 ss = reinterpret_cast<const float4*>(row + a.rot_dim / 2)[i];
                c[4 * i] = cc.x; c[4 * i + 1] = cc.y; c[4 * i + 2] = cc.z; c[4 * i + 3] = cc.w;
                s[4 * i] = ss.x; s[4 * i + 1] = ss.y; s[4 * i + 2] = ss.z; s[4 * i + 3] = ss.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = s[i] = __builtin_nanf("");
        }
        if (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rotate(x[2 * i], x[2 * i + 1], c[i], s[i]);
                rotate(y[2 * i], y[2 * i + 1], c[4 + i], s[4 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) rotate(x[i], y[i], c[i], s[i]);
        }
    }
    if (is_q) {
        uint16_t* dst = a.q_out + t * a.ldqo + (int64_t)hk * D;
        *reinterpret_cast<uint4*>(dst + 8 * u0) = pack8(x);
        *reinterpret_cast<uint4*>(dst + 8 * u1) = pack8(y);
        return;
    }
    float scale = 1.0f;
    if (FP8) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
        for (int g = NL / 2; g >= 1; g >>= 1) m = fmaxf(m, __shfl_xor(m, g, 64));
        // Rotated values go down to the smallest fp32 numbers, where m / 448 keeps few bits or
        // rounds to zero and the quotients pass what a code can hold.  From 32 of the smallest
        // steps on the largest quotient is at most 455, which still rounds to 448; a head of
        // bf16 values is above that bound by itself (2^-133 / 448).
        scale = fmaxf(scale_from_amax(m), 0x1p-144f);
    }
    const int64_t page = slot >> a.cache.page_shift;
    if (slot < 0 || page >= a.cache.pages) return;
    const int64_t row = (((page * a.cache.kv_heads + hk) << a.cache.page_shift) |
                         (slot & ((1 << a.cache.page_shift) - 1)));
    uint8_t* data = is_v ? a.cache.v : a.cache.k;
    if (FP8) {
        uint8_t* dst = data + row * D;
        *reinterpret_cast<uint2*>(dst + 8 * u0) = codes8(x, scale);
        *reinterpret_cast<uint2*>(dst + 8 * u1) = codes8(y, scale);
        if (lane == 0) (is_v ? a.cache.dv : a.cache.dk)[row] = scale;
    } else {
        uint16_t* dst = reinterpret_cast<uint16_t*>(data) + row * D;
        *reinterpret_cast<uint4*>(dst + 8 * u0) = pack8(x);
        *reinterpret_cast<uint4*>(dst + 8 * u1) = pack8(y);
    }
}

template <int NL>
void launch(const RopeArgs& a, hipStream_t s) {
    const int64_t items = a.T * (a.q_heads + 2 * (int64_t)a.cache.kv_heads);
    const dim3 grid((unsigned)((items + 256 / NL - 1) / (256 / NL)));
    if (a.interleaved) {
        if (a.cache.fp8) rope_append_kernel<NL, true, true><<<grid, 256, 0, s>>>(a);
        else rope_append_kernel<NL, true, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.cache.fp8) rope_append_kernel<NL, false, true><<<grid, 256, 0, s>>>(a);
        else rope_append_kernel<NL, false, false><<<grid, 256, 0, s>>>(a);
    }
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t s) {
    if (a.cache.D == 128) launch<8>(a, s);
    else launch<4>(a, s);
    return hipGetLastError();
}

}  // namespace ptpc
