// Device helpers shared by the attention kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "device_common.h"

namespace ptpc {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) i32x2* lds_i32x2;

constexpr float kLog2e = 1.4426950408889634f;

// A row's running maximum is only replaced (and everything summed so far
// rescaled) once a score exceeds it by this much, in powers of two: weights
// then reach 2^8 at most, which fp32 sums and bf16 weights hold as exactly as
// weights up to 1, and after the first few keys almost no tile rescales.
constexpr float kRescaleAt = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// scale * log2(e), made positive (the sign goes into the queries) and nonzero
// (a scale of 0 weighs all keys alike; masked scores are -inf and must stay so).
__device__ __forceinline__ float score_factor(float scale) {
    const float c = fabsf(scale) * kLog2e;
    return c == 0.0f ? 1e-30f : c;
}
__device__ __forceinline__ u32x4 flip_sign(u32x4 q, float scale) {
    const uint32_t s = scale < 0.0f ? 0x80008000u : 0u;
    return u32x4{q.x ^ s, q.y ^ s, q.z ^ s, q.w ^ s};
}

// Maximum / sum over the lanes l, l ^ 32 (two halves of the wave), and over
// l, l ^ 16 too.
__device__ __forceinline__ float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float quarter_max(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Two E4M3 codes (a 16-bit half of w) -> two bf16, exactly.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Nonfinite bf16 halves of a word: all-ones exponent.
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// The word with its nonfinite halves set to zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) |
           ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
}
__device__ __forceinline__ u32x4 finite_part(u32x4 v) {
    return u32x4{finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w)};
}

__device__ __forceinline__ v16f mfma32(u32x4 a, u32x4 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma16(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Four keys of one channel from LDS rows: the 16 lanes of a group each point
// at 8 bytes (4 channels) of rows i/4, and lane i receives channel i's four
// values.  (Lane layout checked on the GPU.)
__device__ __forceinline__ u32x2 read_keys4(const void* at) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at));
}
// Eight keys of one channel of 8-bit rows: lane i of a group points at 8 bytes
// of row i/2 and receives channel i's eight codes.
__device__ __forceinline__ u32x2 read_keys8(const void* at) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2)at));
}
// Workgroup barrier without the fences of __syncthreads() (which would wait
// for every load into LDS in flight); callers wait for what they need first.
__device__ __forceinline__ void attn_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Direct load of 1 KB into LDS: lane i's 16 bytes at byte `off` of the buffer land at
// dst + 16 i (dst the same for the whole wave); bytes past the buffer's end are zero.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t buf, void* dst, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void)dst, 16, off, 0, 0, 0);
}

// The wave's loads (LDS accesses) have all come in.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// What one sequence's rows see.
struct Span {
    int start;      // first row of q
    int n;          // new tokens
    int kv;         // keys
};

__device__ __forceinline__ Span sequence_span(const AttnArgs& a, int b, bool paged) {
    const int T = (int)a.T;
    Span s;
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    s.start = c0 < 0 ? 0 : c0 > T ? T : c0;
    const int end = c1 < s.start ? s.start : c1 > T ? T : c1;
    s.n = end - s.start;
    if (paged) {
        const int kv = a.kv_lens[b];
        s.kv = kv < 0 ? 0 : kv > a.table_keys ? a.table_keys : kv;
    } else {
        s.kv = s.n;
    }
    return s;
}

// Keys seen by row r (token r / G) of a sequence.
__device__ __forceinline__ int visible(const Span& s, int r, int G) {
    const int v = s.kv - s.n + r / G + 1;
    return v < 0 ? 0 : v > s.kv ? s.kv : v;
}

// Row idx's share of keys [lo, hi) when `seen` keys are cut into ranges of
// `chunk` (the last range takes whatever is left), and how many ranges hold any.
__device__ __forceinline__ int active_splits(int seen, int chunk, int splits) {
    const int n = (seen + chunk - 1) / chunk;
    return n < 1 ? 1 : n > splits ? splits : n;
}

}  // namespace ptpc
