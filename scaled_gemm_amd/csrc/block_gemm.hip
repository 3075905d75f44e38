// FP8 x FP8 product with scales on blocks of 128, tiled (gfx950 MFMA).
//
//   out[t,o] = bf16( sum_b (sx[b,t] * sw[o/128, b]) * sum_{k in b} qx[t,k] qw[k,o] )
//
// A block of K is 128 bytes, which is one v_mfma_f32_16x16x128_f8f6f4: every
// MFMA starts from zero and its four results are added to the accumulator with
// one fused multiply-add each.  The weight is the first operand, so the four
// results of a lane belong to one row, and the wave's columns to one weight
// block: the factor is one number per lane and row slab.
#include "block_device.h"

namespace ptpc {
namespace {

// Workgroup barrier without the fences of __syncthreads(): the callers wait
// for exactly what they need first.
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

// Waits for every load and LDS access of the wave.
__device__ __forceinline__ void wait_all() { __builtin_amdgcn_s_waitcnt(7 << 4); }

template <int BM, int BN, int WM, int WN, bool EXPERTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void block_gemm_kernel(BlockGemmArgs g) {
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int MT = WTM / 16, NT = WTN / 16;
    constexpr int A_PER_W = BM / 8 / NW;             // 1 KB loads: 8 rows x 128 B
    constexpr int B_PER_W = BN / 8 / NW;             // 1 KB blocks of the packed weight
    constexpr int S_LOADS = (BM + 63) / 64;          // 256-byte loads of row scales
    static_assert(A_PER_W * NW * 8 == BM && B_PER_W * NW * 8 == BN && S_LOADS <= NW, "tile/waves");
    static_assert(WTN <= 128 && 128 % WTN == 0 && MT % 2 == 0, "one weight block a wave");
    constexpr int D = 4;                             // MFMA results in flight
    __shared__ __attribute__((aligned(1024))) uint8_t a_s0[BM * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t a_s1[BM * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t b_s0[BN * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t b_s1[BN * 128];
    __shared__ __attribute__((aligned(1024))) float s_s0[NW * 64];
    __shared__ __attribute__((aligned(1024))) float s_s1[NW * 64];

    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int l16 = lane & 15, q = lane >> 4;
    const int gn = (int)((g.Co + BN - 1) / BN);
    const int nks = (int)scale_blocks(g.Ci);

    int tm, tn, expert = 0, row0, row_end;
    if constexpr (EXPERTS) {
        const ExpertTiles t = count_expert_tiles<BM>(g.offsets, g.E, (int)g.T);
        if ((int)blockIdx.x >= t.total * gn) return;
        tile_at(xcd_order(blockIdx.x, t.total * gn), t.total, gn, tm, tn);
        find_expert_tile<BM>(g.offsets, g.E, (int)g.T, t, tm, expert, row0, row_end);
        if (expert < 0) return;
    } else {
        const int gm = (int)((g.T + BM - 1) / BM);
        tile_at(xcd_order(blockIdx.x, gm * gn), gm, gn, tm, tn);
        row0 = tm * BM;
        row_end = (int)g.T;
    }
    const int rows = row_end - row0 < BM ? row_end - row0 : BM;
    const int64_t n0 = (int64_t)tn * BN;
    const int64_t Kp = (int64_t)nks * 128;

    // Row r of the tile is row row0 + r of qx, or the one that g.rows names.
    const bool gather = EXPERTS && g.rows != nullptr;
    auto source = [&](int r) -> int {
        if (!gather) return r;
        const int p = g.rows[row0 + r];
        const int t = p < 0 ? -1 : p / g.top_k;
        return t < (int)g.T_in ? t : -1;
    };
    const __amdgpu_buffer_rsrc_t ra =
        gather ? make_rsrc(g.qx, (uint32_t)(g.T_in * g.ldq))
               : make_rsrc(g.qx + (int64_t)row0 * g.ldq, (uint32_t)(rows * g.ldq));
    const int64_t b_cols = g.Co - n0 < BN ? g.Co - n0 : BN;
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(g.wp + (int64_t)expert * g.Co * Kp + n0 * Kp, (uint32_t)(b_cols * Kp));
    const float* const sx0 = g.sx + (gather ? 0 : row0);
    const uint32_t sx_bytes = (uint32_t)((gather ? g.T_in : rows) * 4);

    uint32_t a_off[A_PER_W], b_off[B_PER_W], s_off = kNowhere;
    int a_k[A_PER_W];
#pragma unroll
    for (int p = 0; p < A_PER_W; ++p) {
        const int r = (wave + p * NW) * 8 + (lane >> 3);
        a_k[p] = ((lane & 7) ^ ((r >> 1) & 7)) * 16;     // the chunk of this LDS slot
        a_off[p] = kNowhere;
        if (r < rows) {
            const int t = source(r);
            if (t >= 0) a_off[p] = (uint32_t)(t * g.ldq + a_k[p]);
        }
    }
#pragma unroll
    for (int p = 0; p < B_PER_W; ++p) {
        const int blk = wave + p * NW;                   // (column slab, half of the K block)
        b_off[p] = (uint32_t)(((blk >> 1) * nks * 2 + (blk & 1)) * 1024 + lane * 16);
    }
    if (wave < S_LOADS && wave * 64 + lane < rows) {
        const int t = source(wave * 64 + lane);
        if (t >= 0) s_off = (uint32_t)t * 4;
    }

    // The weight block's scales along K: the wave's columns share one block.
    const int nb = (int)((n0 + wn * WTN) / 128), nblocks = (int)scale_blocks(g.Co);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(
        g.sw + ((int64_t)expert * nblocks + (nb < nblocks ? nb : nblocks - 1)) * nks,
        (uint32_t)(nks * 4));

    // Loads of K block ks into a slot (past the last block: zeros).  Every wave
    // issues the same loads; those without rows to scale load nothing.
    auto fill = [&](int ks, uint8_t* as, uint8_t* bs, float* ss) {
        const int left = (int)g.Ci - ks * 128;
#pragma unroll
        for (int p = 0; p < A_PER_W; ++p)
            load16_to_lds(ra, as + (wave + p * NW) * 1024, a_k[p] < left ? a_off[p] : kNowhere,
                            uniform(ks * 128));
#pragma unroll
        for (int p = 0; p < B_PER_W; ++p)
            load16_to_lds(rb, bs + (wave + p * NW) * 1024, left > 0 ? b_off[p] : kNowhere,
                            uniform(ks * 2048));
        load4_to_lds(make_rsrc(sx0 + (int64_t)ks * g.lds, left > 0 ? sx_bytes : 0),
                       ss + wave * 64, s_off);
    };

    const int a_lo = (wm * WTM + l16) * 128 + ((q ^ ((l16 >> 1) & 7)) << 4);
    const int a_hi = (wm * WTM + l16) * 128 + (((q + 4) ^ ((l16 >> 1) & 7)) << 4);
    const int b_at = wn * WTN * 128 + l16 * 64 + ((q ^ (l16 >> 2)) << 4);
    auto read_a = [&](const uint8_t* as, int i) {
        return join(*reinterpret_cast<const v4i*>(as + a_lo + i * 2048),
                    *reinterpret_cast<const v4i*>(as + a_hi + i * 2048));
    };
    auto read_b = [&](const uint8_t* bs, int j) {
        return join(*reinterpret_cast<const v4i*>(bs + b_at + j * 2048),
                    *reinterpret_cast<const v4i*>(bs + b_at + j * 2048 + 1024));
    };
    auto read_s = [&](const float* ss, int i) { return ss[wm * WTM + i * 16 + l16]; };

    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    v8i fa[2], fb[NT];
    float fs[2];
    auto weight_scale = [&](int ks) {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, 0, uniform(ks * 4), 0));
    };
    float sw_next = weight_scale(0);
    // One K block.  On entry its weight operands and the first row slab's are
    // in registers.  Before the last slab every read of this slot is done and
    // the next block has landed: one barrier, then the slot is refilled with
    // the block after the next and the next block's operands are read.
    auto step = [&](int ks, uint8_t* as, uint8_t* bs, float* ss, const uint8_t* an,
                    const uint8_t* bn, const float* sn) {
        const float swk = sw_next;
        sw_next = weight_scale(ks + 1);
        v4f t[D];
        float s = 0.0f, s_prev = 0.0f;
#pragma unroll
        for (int n = 0; n < MT * NT + D - 1; ++n) {
            const int i = n / NT, j = n % NT;
            if (n < MT * NT) {
                if (j == 0) {
                    if (i == MT - 1) {
                        wait_all();
                        barrier_only();
                        fill(ks + 2, as, bs, ss);
                        fa[(i + 1) & 1] = read_a(an, 0);
                        fs[(i + 1) & 1] = read_s(sn, 0);
                    } else {
                        fa[(i + 1) & 1] = read_a(as, i + 1);
                        fs[(i + 1) & 1] = read_s(ss, i + 1);
                    }
                    s_prev = s;
                    s = fs[i & 1] * swk;
                }
                t[n % D] = mfma_block(fb[j], fa[i & 1]);
                if (i == MT - 1) fb[j] = read_b(bn, j);
            }
            if (n >= D - 1) {
                const int m = n - (D - 1), mi = m / NT, mj = m % NT;
                const float f = (n < MT * NT && mi != i) ? s_prev : s;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[mi][mj][e] = __builtin_fmaf(t[m % D][e], f, acc[mi][mj][e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (nks > 0) {
        fill(0, a_s0, b_s0, s_s0);
        fill(1, a_s1, b_s1, s_s1);
        wait_all();
        barrier_only();
        fa[0] = read_a(a_s0, 0);
        fs[0] = read_s(s_s0, 0);
#pragma unroll
        for (int j = 0; j < NT; ++j) fb[j] = read_b(b_s0, j);
        int ks = 0;
#pragma clang loop unroll(disable)
        for (; ks + 1 < nks; ks += 2) {
            step(ks, a_s0, b_s0, s_s0, a_s1, b_s1, s_s1);
            step(ks + 1, a_s1, b_s1, s_s1, a_s0, b_s0, s_s0);
        }
        if (ks < nks) step(ks, a_s0, b_s0, s_s0, a_s1, b_s1, s_s1);
        wait_all();                                  // no load into LDS outlives the workgroup
    }

    const __amdgpu_buffer_rsrc_t ro =
        make_rsrc(g.out + (int64_t)row0 * g.ldo, (uint32_t)(rows * g.ldo * 2));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = wm * WTM + i * 16 + l16;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t col = n0 + wn * WTN + j * 16 + 4 * q;
            typedef int v2i __attribute__((ext_vector_type(2)));
            const v2i v = {(int)f32x2_to_bf16x2_rne(acc[i][j][0], acc[i][j][1]),
                           (int)f32x2_to_bf16x2_rne(acc[i][j][2], acc[i][j][3])};
            __builtin_amdgcn_raw_buffer_store_b64(
                v, ro, col < g.Co && r < rows ? (uint32_t)((r * g.ldo + col) * 2) : kNowhere, 0, 0);
        }
    }
}

template <int BM, int BN, int WM, int WN>
hipError_t launch(const BlockGemmArgs& a, BlockPlan p, hipStream_t s) {
    const dim3 grid((unsigned)block_gemm_grid(p, a.T, a.offsets ? a.E : 0, a.Co));
    if (a.offsets != nullptr)
        block_gemm_kernel<BM, BN, WM, WN, true><<<grid, WM * WN * 64, 0, s>>>(a);
    else
        block_gemm_kernel<BM, BN, WM, WN, false><<<grid, WM * WN * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s) {
    const BlockPlan p = block_gemm_plan(a.T, a.offsets ? a.E : 1, a.Ci, a.Co);
    switch (p) {
        case BlockPlan::k256x256: return launch<256, 256, 2, 4>(a, p, s);
        case BlockPlan::k128x256: return launch<128, 256, 2, 4>(a, p, s);
        case BlockPlan::k128x128: return launch<128, 128, 2, 2>(a, p, s);
        case BlockPlan::k64x128: return launch<64, 128, 2, 2>(a, p, s);
        default: return launch_block_gemm_few(a, p, s);
    }
}

}  // namespace ptpc
