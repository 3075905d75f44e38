// Device helpers shared by the attention kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "device_common.h"

namespace ptpc {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
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

// Maximum of three, in one instruction (fmaxf would first quiet the NaNs of each).  A NaN
// comes through: it then compares false wherever a maximum is used, so a row's reference
// stays as it was, and the row is NaN by its sum.  A builtin, not inline asm: it reads MFMA
// results, and only for instructions of its own does the compiler keep the wait states
// between the two.
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
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

// The same for E4M3 codes, whose only nonfinite value is NaN (0x7F, 0xFF): some
// code of the word is, and the word with those set to zero.
__device__ __forceinline__ uint32_t nan_bits4(uint32_t w) {      // 0x80 in each NaN byte
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ bool nan_code4(uint32_t w) { return nan_bits4(w) != 0; }
__device__ __forceinline__ uint32_t number_codes4(uint32_t w) {
    const uint32_t n = nan_bits4(w);
    return w & ~(n | (n - (n >> 7)));
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

// LDS-poison debug build (-DPTPC_LDS_POISON): where a wave starts to refill `kb` KB of LDS, it
// overwrites them with ones first -- NaN as bf16 and as E4M3 -- and waits for those writes.  A
// wave that still read the region, or read it before the fill landed, would see NaN.
__device__ __forceinline__ void poison_refill(uint8_t* at, int kb) {
#ifdef PTPC_LDS_POISON
    for (int i = 0; i < kb; ++i)
        *reinterpret_cast<u32x4*>(at + i * 1024 + (threadIdx.x & 63) * 16) = u32x4{~0u, ~0u, ~0u, ~0u};
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
}

// Buffer over [base + bytes_before, + bytes) for a base and extents that are the same
// for the whole wave (said so explicitly, or the compiler may loop over lanes).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t wave_buffer(const void* base, int64_t bytes_before, int bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base) + (uint64_t)bytes_before;
    const uint64_t lo = (uint32_t)uniform((int)(uint32_t)at), hi = (uint32_t)uniform((int)(uint32_t)(at >> 32));
    return make_rsrc(reinterpret_cast<const void*>(hi << 32 | lo), (uint32_t)uniform(bytes));
}

// 16 bytes at byte `off` of the buffer (zeros past its end).
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t buf, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off, 0, 0));
}

// Waits for all but the wave's last VM loads and LG LDS accesses, through the builtin
// (which the compiler's own counting understands) and fenced on both sides.
template <int VM, int LG>
__device__ __forceinline__ void wait_for() {
    static_assert(VM >= 0 && VM < 64 && LG >= 0 && LG < 16, "counter range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (LG << 8));
    asm volatile("" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads_but() { wait_for<N, 15>(); }
__device__ __forceinline__ void wait_loads() { wait_for<0, 15>(); }
__device__ __forceinline__ void wait_lds() { wait_for<63, 0>(); }

__device__ __forceinline__ float buffer_load4(__amdgpu_buffer_rsrc_t buf, int off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, off, 0, 0));
}

// n cut to 0 .. most, in scalar registers (in one expression it becomes a vector
// instruction, whose destination may wait for a load in flight).
__device__ __forceinline__ int clamp_rows(int n, int most) {
    n = uniform(n < most ? n : most);
    return n < 0 ? 0 : n;
}

// Element i (the same for the whole wave) of an index array, as a scalar load:
// the arrays are not written while a kernel runs, and a vector load's wait would
// drain the fills in flight.
__device__ __forceinline__ int scalar_at(const int32_t* p, int64_t i) {
    typedef const __attribute__((address_space(4))) int32_t* cptr;
    const uint64_t at = reinterpret_cast<uint64_t>(p + i);
    const uint64_t lo = (uint32_t)uniform((int)(uint32_t)at), hi = (uint32_t)uniform((int)(uint32_t)(at >> 32));
    return *(cptr)(hi << 32 | lo);
}

// What one sequence's rows see.
struct Span {
    int start;      // first row of q
    int n;          // new tokens
    int kv;         // keys
};

__device__ __forceinline__ Span sequence_span(const AttnArgs& a, int b, bool paged) {
    const int T = (int)a.T;
    Span s;
    const int c0 = scalar_at(a.cu, b), c1 = scalar_at(a.cu, b + 1);
    s.start = c0 < 0 ? 0 : c0 > T ? T : c0;
    const int end = c1 < s.start ? s.start : c1 > T ? T : c1;
    s.n = end - s.start;
    if (paged) {
        const int kv = scalar_at(a.kv_lens, b);
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

// How many ranges of `chunk` keys hold any of `seen` keys (the last of `splits`
// ranges takes whatever is left).
__device__ __forceinline__ int active_splits(int seen, int chunk, int splits) {
    const int n = (seen + chunk - 1) / chunk;
    return n < 1 ? 1 : n > splits ? splits : n;
}

// The workspace holds, for each (item, range, row of the tile), D fp32 sums, and
// after all of those the row's reference maximum and the sum of its weights.
__device__ __forceinline__ float2* part_stats(const AttnArgs& a, int items, int splits, int tile_rows, int D) {
    return reinterpret_cast<float2*>(a.ws + (int64_t)items * splits * tile_rows * D);
}

// Join of a row's ranges by one wave: lane s takes the statistics of ranges s and
// s + 64, then each lane sums its channels over the ranges.
template <int D>
__device__ __forceinline__ void join_row(const AttnArgs& a, int items, int splits, int tile_rows, int item,
                                         int r, int parts, uint16_t* out) {
    static_assert(kMaxSplits <= 128, "two ranges a lane");
    constexpr int C = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t at = (int64_t)item * splits * tile_rows + r;
    const float2* st = part_stats(a, items, splits, tile_rows, D) + at;
    float2 s0 = make_float2(-INFINITY, 0.0f), s1 = s0;
    if (lane < parts) s0 = st[(int64_t)lane * tile_rows];
    if (lane + 64 < parts) s1 = st[(int64_t)(lane + 64) * tile_rows];
    float m = fmaxf(s0.x, s1.x);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    const float shift = m == -INFINITY ? 0.0f : m;
    const float f0 = exp2_fast(s0.x - shift), f1 = exp2_fast(s1.x - shift);
    float l = s0.y * f0 + s1.y * f1;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) l += __shfl_xor(l, d, 64);
    const float* src = a.ws + at * D + lane * C;
    const int64_t stride = (int64_t)tile_rows * D;
    float o[C] = {};
    for (int s = 0; s < parts; s += 4) {         // four ranges' loads in flight
        float f[4], x[4][C];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at_k = s + k < parts ? s + k : s;
#pragma unroll
            for (int i = 0; i < C; ++i) x[k][i] = src[at_k * stride + i];
            f[k] = s + k < parts ? __shfl(s + k < 64 ? f0 : f1, (s + k) & 63, 64) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < C; ++i) o[i] += s + k < parts ? x[k][i] * f[k] : 0.0f;
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    if constexpr (C == 2)
        *reinterpret_cast<uint32_t*>(out + lane * C) = f32x2_to_bf16x2_rne(o[0] * inv, o[1] * inv);
    else
        out[lane] = (uint16_t)f32x2_to_bf16x2_rne(o[0] * inv, 0.0f);
}

}  // namespace ptpc
