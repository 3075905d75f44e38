// Device helpers shared by the block-scaled GEMM kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block.h"
#include "device_common.h"

namespace ptpc {

typedef __attribute__((address_space(3))) void* lds_void;
constexpr uint32_t kNowhere = 0x80000000u;      // a buffer offset past every descriptor

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One MFMA: D[column][row] of a 16-column slab and a 16-row slab over 128 K
// bytes, nothing added.  Lane l holds output row l % 16 and columns
// 4 * (l / 16) .. +3; as an operand, row or column l % 16 and the K bytes
// 16q .. 16q+15 and 64+16q .. 64+16q+15 with q = l / 16 (any order of K will
// do as long as both operands have it; this one takes whole 1 KB blocks of the
// packed weight in one load).
__device__ __forceinline__ v4f mfma_block(v8i w, v8i x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0,
                                                            0, 0, 0, 0);
}

__device__ __forceinline__ v8i join(v4i lo, v4i hi) {
    return v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// LDS-poison debug build (-DPTPC_LDS_POISON): where a wave refills LDS, it first
// overwrites it with ones -- NaN as E4M3 and as fp32 -- and waits for those writes.
// A wave that still read the region, or read it before the refill landed, would see
// NaN, and so would its results.
template <class T>
__device__ __forceinline__ void poison_refill(void* dst, T ones) {
#ifdef PTPC_LDS_POISON
    reinterpret_cast<T*>(dst)[threadIdx.x & 63] = ones;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#else
    (void)dst, (void)ones;
#endif
}

// Direct loads into LDS: lane i's 16 (4) bytes at byte off + base of the buffer
// land at dst + 16 i (4 i), dst and base the same for the whole wave; past the
// buffer's end they are zero.
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t buf, void* dst, uint32_t off,
                                              int base) {
    poison_refill(dst, v4i{-1, -1, -1, -1});
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void)dst, 16, off, base, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t buf, void* dst, uint32_t off) {
    poison_refill(dst, -1);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void)dst, 4, off, 0, 0, 0);
}

// Four sums as bf16, rounded to nearest even, at byte `off` of the output.
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t ro, v4f v, uint32_t off) {
    typedef int v2i __attribute__((ext_vector_type(2)));
    const v2i b = {(int)f32x2_to_bf16x2_rne(v[0], v[1]), (int)f32x2_to_bf16x2_rne(v[2], v[3])};
    __builtin_amdgcn_raw_buffer_store_b64(b, ro, off, 0, 0);
}

// Bounds of expert e's rows, inside the output whatever the array holds.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int R, int& a, int& b) {
    const int lo = offsets[e], hi = offsets[e + 1];
    a = lo < 0 ? 0 : lo > R ? R : lo;
    b = hi < a ? a : hi > R ? R : hi;
}

// Row tiles of BM rows over the experts, in expert order.  Every lane of a
// wave takes per = ceil(E / 64) consecutive experts; returns the tiles in all.
struct ExpertTiles {
    int before;       // tiles of the lanes below this one
    int total;
};
template <int BM>
__device__ __forceinline__ ExpertTiles count_expert_tiles(const int32_t* offsets, int E, int R) {
    const int lane = threadIdx.x & 63, per = (E + 63) / 64;
    int mine = 0;
    for (int p = 0; p < per; ++p) {
        const int e = lane * per + p;
        int a, b;
        expert_rows(offsets, e < E ? e : E - 1, R, a, b);
        if (e < E) mine += (b - a + BM - 1) / BM;
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d, 64);
        if (lane >= d) sum += o;
    }
    return {sum - mine, uniform(__shfl(sum, 63, 64))};
}
// Expert, first row and end row of tile m (m < total); uniform.
template <int BM>
__device__ __forceinline__ void find_expert_tile(const int32_t* offsets, int E, int R,
                                                 const ExpertTiles& t, int m, int& expert,
                                                 int& row0, int& row_end) {
    const int lane = threadIdx.x & 63, per = (E + 63) / 64;
    int e_found = -1, r0 = 0, r1 = 0, at = t.before;
    for (int p = 0; p < per; ++p) {
        const int e = lane * per + p;
        int a, b;
        expert_rows(offsets, e < E ? e : E - 1, R, a, b);
        const int n = e < E ? (b - a + BM - 1) / BM : 0;
        if (m >= at && m < at + n) {
            e_found = e;
            r0 = a + (m - at) * BM;
            r1 = b;
        }
        at += n;
    }
    const uint64_t who = __ballot(e_found >= 0);
    const int src = who ? (int)__builtin_ctzll(who) : 0;
    expert = uniform(__shfl(e_found, src, 64));
    row0 = uniform(__shfl(r0, src, 64));
    row_end = uniform(__shfl(r1, src, 64));
}

// Order of the tiles: workgroups are dealt round-robin to the 8 XCDs, each with
// its own L2; XCD x takes a contiguous run of the logical order, which walks
// groups of 8 column blocks, every row block of a group before the next group.
constexpr int kXcdCount = 8;
constexpr int kGroupCols = 8;
__device__ __forceinline__ int xcd_order(int b, int n) {
    const int x = b % kXcdCount, per = n / kXcdCount, more = n % kXcdCount;
    return x * per + (x < more ? x : more) + b / kXcdCount;
}
__device__ __forceinline__ void tile_at(int i, int gm, int gn, int& tm, int& tn) {
    const int group = i / (kGroupCols * gm);
    const int first = group * kGroupCols;
    const int width = gn - first < kGroupCols ? gn - first : kGroupCols;
    const int r = i - group * kGroupCols * gm;
    tm = uniform(r / width);
    tn = uniform(first + r % width);
}

}  // namespace ptpc
