// FP8 x FP8 product with scales on blocks of 128, tiled (gfx950 MFMA).
//
//   out[t,o] = bf16( sum_b (sx[b,t] * sw[o/128, b]) * sum_{k in b} qx[t,k] qw[k,o] )
//
// A block of K is 128 bytes, which is one v_mfma_f32_16x16x128_f8f6f4: every
// MFMA starts from zero and its four results are added to the accumulator with
// one fused multiply-add each.  The weight is the first operand, so the four
// results of a lane belong to one row, and the wave's columns to one weight
// block: the factor is one number per lane and row slab.  Within an MFMA the
// hardware adds products in groups of 8 neighbours along K, each product cut towards
// zero to a multiple of 2^(m - 13), m the group's largest sum of two operands'
// exponents (measured: with that, torch gives the results bit for bit); it is why a
// few results in a hundred are a bf16 step from a product in 32 bits.  Between blocks
// everything is fp32.
//
// Tiles: six sizes from 32 x 64 (a weight streamed for few rows: more workgroups on
// a CU, less latency) to 256 x 256 (fewest bytes per MFMA), chosen on the host by
// what a K block of each was measured to take.  Operands go from memory straight
// into an LDS ring; results collect in registers.
//
// What bounds it.  Large products: the operand stream into LDS and the clock, which
// power holds at 1.65 to 1.85 GHz, card by card; MFMAs are busy 68% of the cycles, the
// four multiply-adds of each (18 cycles beside its 32) run under the other wave's.
// 8192 x 28672 x 8192 takes 1479 to 1613 us (2.39 to 2.60 PFLOP/s; without the fills
// 18% less, without the multiply-adds 10%), 8192 x 2048 x 16384 247 to 262 us, of which
// the results alone (268 MB) are 55 of HBM time.  Few rows: the weight's stream, one
// token through 8192 x 10240 13.3 us (6.3 TB/s, part of the weight still in the
// memory-side cache), 2048 rows of 128 experts (1408 x 4096) 138 us (5.4 TB/s).  In
// between: a CU takes 34 to 36 bytes a clock into LDS, 333 x 2736 x 4112 10.5 us.
// Prompts over experts also pay for rows that are not there and for a short K (24576
// rows of 64 experts, 2048 x 2816: 186 to 222 us, 1.28 to 1.52 PFLOP/s).
//
// Tried and level or slower: three or four slots of 256 x 256, one workgroup a CU
// that walks the tiles (5 to 9%), two or three MFMA results in flight, wave
// priorities around the MFMAs, non-temporal stores of the results; last tiles of an
// expert cut to quarters instead of halves (1 to 3% on some prompts, level on
// others, for twice the code).
#include <utility>

#include "block_device.h"

namespace ptpc {
namespace {

// Workgroup barrier without the fences of __syncthreads(): the callers wait
// for exactly what they need first.
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

// Waits until at most VM of the wave's loads are in flight, and for its LDS reads.
template <int VM>
__device__ __forceinline__ void wait_loads() {
    static_assert(VM >= 0 && VM < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
}

// LDS: NS slots, each a K block of the tile: BM rows of 128 bytes, BN columns as
// they are packed, and the scales (those of the rows, then, for the wave after
// the ones that load them, those of the weight's blocks).  Distinct objects, so
// that the compiler can tell the slot being filled from the one being read.
template <int BM, int BN, int WM, int WN, int NS, bool EXPERTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void block_gemm_kernel(BlockGemmArgs g) {
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int MT = WTM / 16, NT = WTN / 16;
    constexpr int A_PER_W = BM / 8 / NW;             // 1 KB loads: 8 rows x 128 B
    constexpr int B_PER_W = BN / 8 / NW;             // 1 KB blocks of the packed weight
    constexpr int LOADS = A_PER_W + B_PER_W + 1;
    constexpr int S_LOADS = (BM + 63) / 64;          // 256-byte loads of row scales
    static_assert(A_PER_W * NW * 8 == BM && B_PER_W * NW * 8 == BN && S_LOADS < NW, "tile/waves");
    static_assert(WTN <= 128 && 128 % WTN == 0 && MT % 2 == 0, "one weight block a wave");
    constexpr bool ONE_BARRIER = MT == 2;            // the second slab is the last one
    // Row slabs whose operands are on their way from LDS, and their registers (two of
    // eight slabs: 8192 x 28672 x 8192 1526 -> 1504 us; the others have four or two).
    constexpr int LOOK = MT >= 8 ? 2 : 1, FA = 2 * LOOK;
    // Where a step's barriers stand, in row slabs, and what they let go: see step.
    constexpr int AT_A = ONE_BARRIER ? 1 : MT / 2 - LOOK, AT_END = MT - LOOK;
    constexpr int A1 = ONE_BARRIER ? A_PER_W : A_PER_W / 2, A2 = A_PER_W - A1;
    constexpr int A2_NOW = (A2 + 1) / 2, A2_LATE = A2 - A2_NOW;
    // (a step's refills of the weight fill the slabs up to AT_A2, the rows' those after)
    constexpr int AT_A2 = AT_A > 1 ? AT_A + 2 : 2;
    constexpr int LO = ONE_BARRIER ? MT : MT / 2;    // row slabs of the first part of the rows
    constexpr int A_LO = LO * WM * 2048, A_HI = ONE_BARRIER ? 16 : BM * 128 - A_LO;
    static_assert(ONE_BARRIER || (A_PER_W % 2 == 0 && MT % 4 == 0), "halves of the rows");
    constexpr int D = 4;                             // MFMA results in flight
    __shared__ __attribute__((aligned(1024))) uint8_t a_lo0[A_LO];
    __shared__ __attribute__((aligned(1024))) uint8_t a_hi0[A_HI];
    __shared__ __attribute__((aligned(1024))) uint8_t a_lo1[A_LO];
    __shared__ __attribute__((aligned(1024))) uint8_t a_hi1[A_HI];
    __shared__ __attribute__((aligned(1024))) uint8_t a_lo2[NS > 2 ? A_LO : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t a_hi2[NS > 2 ? A_HI : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t a_lo3[NS > 3 ? A_LO : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t a_hi3[NS > 3 ? A_HI : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b_s0[BN * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t b_s1[BN * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t b_s2[NS > 2 ? BN * 128 : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t b_s3[NS > 3 ? BN * 128 : 16];
    __shared__ __attribute__((aligned(256))) float s_s0[NW * 64];
    __shared__ __attribute__((aligned(256))) float s_s1[NW * 64];
    __shared__ __attribute__((aligned(256))) float s_s2[NS > 2 ? NW * 64 : 4];
    __shared__ __attribute__((aligned(256))) float s_s3[NS > 3 ? NW * 64 : 4];
    uint8_t* const a_slot[4][2] = {{a_lo0, a_hi0}, {a_lo1, a_hi1}, {a_lo2, a_hi2}, {a_lo3, a_hi3}};
    uint8_t* const b_slot[4] = {b_s0, b_s1, b_s2, b_s3};
    float* const s_slot[4] = {s_s0, s_s1, s_s2, s_s3};

    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int l16 = lane & 15, q = lane >> 4;
    const int gn = (int)((g.Co + BN - 1) / BN);
    const int nks = (int)scale_blocks(g.Ci);

    int tm, tn, expert = 0, row0, row_end;
    if constexpr (EXPERTS) {
        const ExpertTiles t = count_expert_tiles<BM>(g.offsets, g.E, (int)g.T);
        // (offsets that make no sense can claim more tiles than the grid was sized for)
        const int most = (int)g.T / BM + (g.E < (int)g.T ? g.E : (int)g.T);
        const int gm = t.total < most ? t.total : most;
        if ((int)blockIdx.x >= gm * gn) return;
        tile_at(xcd_order(blockIdx.x, gm * gn), gm, gn, tm, tn);
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
    const int nblocks = (int)scale_blocks(g.Co);
    const float* const sw0 = g.sw + ((int64_t)expert * nblocks + (int)(n0 / 128)) * nks;
    if (wave < S_LOADS) {
        if (wave * 64 + lane < rows) {
            const int t = source(wave * 64 + lane);
            if (t >= 0) s_off = (uint32_t)t * 4;
        }
    } else if (wave == S_LOADS && lane < (BN + 127) / 128) {
        s_off = (uint32_t)(lane * nks) * 4;
    }
    const int64_t s_step = wave == S_LOADS ? 1 : g.lds;
    const float* const s_base = wave == S_LOADS ? sw0 : sx0;
    const uint32_t s_bytes =
        wave == S_LOADS ? (uint32_t)((nblocks - (int)(n0 / 128)) * nks * 4) : sx_bytes;

    // Loads of K block ks into a slot (past the last block: zeros), one at a
    // time.  Every wave issues the same ones; those without scales load nothing.
    auto fill_a = [&](int ks, int p, uint8_t* const (&as)[2]) {
        const int left = (int)g.Ci - ks * 128;
        uint8_t* const at = p < A1 ? as[0] + (wave + p * NW) * 1024
                                   : as[1] + (wave + (p - A1) * NW) * 1024;
        load16_to_lds(ra, at, a_k[p] < left ? a_off[p] : kNowhere,
                      uniform(ks * 128));
    };
    auto fill_b = [&](int ks, int p, uint8_t* bs) {
        load16_to_lds(rb, bs + (wave + p * NW) * 1024, ks < nks ? b_off[p] : kNowhere,
                      uniform(ks * 2048));
    };
    auto fill_s = [&](int ks, float* ss) {
        // (the weight's scales of block ks start ks entries in: the range shrinks by as much)
        load4_to_lds(make_rsrc(s_base + ks * s_step,
                               ks < nks ? s_bytes - (wave == S_LOADS ? ks * 4 : 0) : 0),
                     ss + wave * 64, s_off);
    };

    const int a_lo = (wm * 16 + l16) * 128 + ((q ^ ((l16 >> 1) & 7)) << 4);
    const int a_hi = (wm * 16 + l16) * 128 + (((q + 4) ^ ((l16 >> 1) & 7)) << 4);
    const int b_at = wn * WTN * 128 + l16 * 64 + ((q ^ (l16 >> 2)) << 4);
    auto read_a = [&](uint8_t* const (&as)[2], int i) {
        const uint8_t* const at = i < LO ? as[0] + i * WM * 2048 : as[1] + (i - LO) * WM * 2048;
        return join(*reinterpret_cast<const v4i*>(at + a_lo), *reinterpret_cast<const v4i*>(at + a_hi));
    };
    auto read_b = [&](const uint8_t* bs, int j) {
        return join(*reinterpret_cast<const v4i*>(bs + b_at + j * 2048),
                    *reinterpret_cast<const v4i*>(bs + b_at + j * 2048 + 1024));
    };
    auto read_s = [&](const float* ss, int i) { return ss[(i * WM + wm) * 16 + l16]; };
    auto read_w = [&](const float* ss) { return ss[S_LOADS * 64 + wn * WTN / 128]; };

    if (nks > 0) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
#pragma unroll
            for (int p = 0; p < B_PER_W; ++p) fill_b(u, p, b_slot[u]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < A1; ++p) fill_a(u, p, a_slot[u]);
            __builtin_amdgcn_sched_barrier(0);
            fill_s(u, s_slot[u]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < A2 - (u == NS - 1 ? A2_LATE : 0); ++p) fill_a(u, A1 + p, a_slot[u]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The tile's product and its results.  SLABS: the wave's row slabs that have rows.
    auto product = [&](auto F) __attribute__((always_inline)) {
        constexpr int SLABS = decltype(F)::value;
        v4f acc[SLABS][NT];
#pragma unroll
        for (int i = 0; i < SLABS; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

        v8i fa[FA], fb[NT];
        float fs[FA], fw;
        // One K block (slot u).  On entry its weight operands and those of the first LOOK
        // row slabs are in registers or on their way.  The slot is let go in parts, each
        // behind one of two barriers at which every wave has read it, and refilled with
        // block ks + NS: the weight (in registers from the step's start) and the first
        // half of the rows from AT_A on, the second half and the scales from AT_END on
        // (and in the next step's first slab).  Likewise a part is waited for where it is
        // read first: the second half of the rows at AT_A, everything else of the next
        // block at AT_END.  So a load has about a step and a half to land.  (The wave's
        // slabs are dealt round the tile's rows, so that the first half of a slot is the
        // first half of every wave's slabs.  With two slabs one barrier does it all.)
        auto step = [&](auto U, int ks) __attribute__((always_inline)) {
            constexpr int u = decltype(U)::value, v = (u + 1) % NS;
            uint8_t* const(&as)[2] = a_slot[u];
            uint8_t* const bs = b_slot[u];
            float* const ss = s_slot[u];
            uint8_t* const(&an)[2] = a_slot[v];
            const uint8_t* const bn = b_slot[v];
            const float* const sn = s_slot[v];
            const float swk = fw;
            v4f t[D];
            float factor[MT];
#pragma unroll
            for (int n = 0; n < MT * NT + D - 1; ++n) {
                const int i = n / NT, j = n % NT;
                if (n < MT * NT) {
                    if (j == 0) {
                        if (!ONE_BARRIER && i == AT_A) {
                            wait_loads<(NS - 1) * LOADS>();
                            barrier_only();
                        }
                        if (i == AT_END) {
                            wait_loads<(NS - 2) * LOADS + (ONE_BARRIER ? 0 : A2 + B_PER_W + A1)>();
                            barrier_only();
                            fill_s(ks + NS, ss);
                            fw = read_w(sn);
                        }
                        if (i >= AT_END) {
                            fa[(i + LOOK) % FA] = read_a(an, i - AT_END);
                            fs[(i + LOOK) % FA] = read_s(sn, i - AT_END);
                        } else if (i + LOOK < SLABS) {
                            fa[(i + LOOK) % FA] = read_a(as, i + LOOK);
                            fs[(i + LOOK) % FA] = read_s(ss, i + LOOK);
                        }
                        factor[i] = fs[i % FA] * swk;
                    }
                    // the refills, about one to a slab: the address unit takes several cycles
                    // for each, and a burst of them would hold up the MFMAs behind it
                    if constexpr (ONE_BARRIER) {
                        if (i == MT - 1) {
#pragma unroll
                            for (int p = j * B_PER_W / NT; p < (j + 1) * B_PER_W / NT; ++p)
                                fill_b(ks + NS, p, bs);
#pragma unroll
                            for (int p = j * A_PER_W / NT; p < (j + 1) * A_PER_W / NT; ++p)
                                fill_a(ks + NS, p, as);
                        }
                    } else {
                        // part p of `parts` loads over the slabs from .. to - 1 is due at MFMA n
                        auto due = [&](int p, int parts, int from, int to) {
                            return n == from * NT + p * (to - from) * NT / parts;
                        };
#pragma unroll
                        for (int p = 0; p < A2_LATE; ++p)
                            if (due(p, A2_LATE, 0, 1))
                                fill_a(ks - 1 + NS, A1 + A2_NOW + p, a_slot[(u + NS - 1) % NS]);
#pragma unroll
                        for (int p = 0; p < B_PER_W; ++p)
                            if (due(p, B_PER_W, AT_A, AT_A2)) fill_b(ks + NS, p, bs);
#pragma unroll
                        for (int p = 0; p < A1; ++p)
                            if (due(p, A1, AT_A2, AT_END)) fill_a(ks + NS, p, as);
#pragma unroll
                        for (int p = 0; p < A2_NOW; ++p)
                            if (due(p, A2_NOW, AT_END, MT)) fill_a(ks + NS, A1 + p, as);
                    }
                    if (i < SLABS) t[n % D] = mfma_block(fb[j], fa[i % FA]);
                    if (i == MT - 1) fb[j] = read_b(bn, j);
                }
                if (n >= D - 1 && n - (D - 1) < SLABS * NT) {
                    const int m = n - (D - 1), mi = m / NT, mj = m % NT;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[mi][mj][e] = __builtin_fmaf(t[m % D][e], factor[mi], acc[mi][mj][e]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        if (nks > 0) {
            wait_loads<(NS - 1) * LOADS + A2 - A2_LATE>();
            barrier_only();
#pragma unroll
            for (int i = 0; i < LOOK; ++i) {
                fa[i] = read_a(a_slot[0], i);
                fs[i] = read_s(s_s0, i);
            }
            fw = read_w(s_s0);
#pragma unroll
            for (int j = 0; j < NT; ++j) fb[j] = read_b(b_s0, j);
            int ks = 0;
#pragma clang loop unroll(disable)
            for (; ks + NS <= nks; ks += NS) {
                [&]<int... Us>(std::integer_sequence<int, Us...>) {
                    (step(std::integral_constant<int, Us>{}, ks + Us), ...);
                }(std::make_integer_sequence<int, NS>{});
            }
            // the blocks left over, fewer than NS
            if (ks < nks) step(std::integral_constant<int, 0>{}, ks);
            if constexpr (NS > 2)
                if (ks + 1 < nks) step(std::integral_constant<int, 1>{}, ks + 1);
            if constexpr (NS > 3)
                if (ks + 2 < nks) step(std::integral_constant<int, 2>{}, ks + 2);
            wait_loads<0>();                             // no load into LDS outlives the workgroup
        }

        const __amdgpu_buffer_rsrc_t ro =
            make_rsrc(g.out + (int64_t)row0 * g.ldo, (uint32_t)(rows * g.ldo * 2));
        auto out_at = [&](int i, int r, int c) {         // row of slab i, column of the wave
            const int row = (i * WM + wm) * 16 + r;
            const int64_t col = n0 + wn * WTN + c;
            return col < g.Co && row < rows ? (uint32_t)((row * g.ldo + col) * 2) : kNowhere;
        };
        if constexpr (NT == 4) {
            // A slab's 16 rows of 64 columns pass through 2 KB of the wave's own LDS (two
            // of them in turn, in the weight's first slot), so that a store writes whole
            // 128-byte rows instead of 32-byte pieces: 8192 tokens of 2048 x 16384 278 ->
            // 247 us.  16-byte chunk c of row r lies at c ^ (r & 7).
            barrier_only();
            uint8_t* const mine = b_s0 + wave * 4096;
#pragma unroll
            for (int i = 0; i < SLABS; ++i) {
                uint8_t* const buf = mine + (i & 1) * 2048;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint2 v = {f32x2_to_bf16x2_rne(acc[i][j][0], acc[i][j][1]),
                                     f32x2_to_bf16x2_rne(acc[i][j][2], acc[i][j][3])};
                    *reinterpret_cast<uint2*>(
                        buf + l16 * 128 + (((2 * j + (q >> 1)) ^ (l16 & 7)) << 4) + (q & 1) * 8) = v;
                }
                __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = h * 8 + (lane >> 3), c = lane & 7;
                    const v4i v =
                        *reinterpret_cast<const v4i*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
                    __builtin_amdgcn_raw_buffer_store_b128(v, ro, out_at(i, r, c * 8), 0, 0);
                }
                __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            }
        } else {
#pragma unroll
            for (int i = 0; i < SLABS; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    store4(ro, acc[i][j], out_at(i, l16, j * 16 + 4 * q));
        }
    };
    // An expert's last tile is half empty half of the time: without the products of
    // its second half then.
    if constexpr (EXPERTS && MT >= 4) {
        if (rows <= BM / 2) {
            product(std::integral_constant<int, MT / 2>{});
            return;
        }
    }
    product(std::integral_constant<int, MT>{});
}

// NS, ENS: slots of the dense kernel and of the experts' (whose many small tiles
// gain more from a further workgroup on the CU than from a further slot).
template <int BM, int BN, int WM, int WN, int NS, int ENS = NS>
hipError_t launch(const BlockGemmArgs& a, BlockPlan p, hipStream_t s) {
    const dim3 grid((unsigned)block_gemm_grid(p, a.T, a.offsets ? a.E : 0, a.Co));
    if (a.offsets != nullptr)
        block_gemm_kernel<BM, BN, WM, WN, ENS, true><<<grid, WM * WN * 64, 0, s>>>(a);
    else
        block_gemm_kernel<BM, BN, WM, WN, NS, false><<<grid, WM * WN * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s) {
    const BlockPlan p = block_gemm_plan(a.T, a.offsets ? a.E : 0, a.Ci, a.Co);
    switch (p) {
        case BlockPlan::k256x256: return launch<256, 256, 2, 4, 2>(a, p, s);
        case BlockPlan::k128x256: return launch<128, 256, 2, 4, 2>(a, p, s);
        case BlockPlan::k128x128: return launch<128, 128, 2, 2, 2>(a, p, s);
        case BlockPlan::k64x128: return launch<64, 128, 2, 2, 3>(a, p, s);
        case BlockPlan::k64x64: return launch<64, 64, 2, 2, 4>(a, p, s);
        case BlockPlan::k32x64: return launch<32, 64, 1, 4, 4, 3>(a, p, s);
        case BlockPlan::kFew: return launch_block_gemm_few(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace ptpc
