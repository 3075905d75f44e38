// Attention of many query rows: prompts, and chunks of new tokens over the
// paged cache.
//
// For each row, one pass over its keys with the running maximum m and sum l of
// the softmax: w_j = 2^(c s_j - m), O = sum w_j v_j, out = O / l, with
// c = |scale| log2 e; when m grows, O and l are rescaled.
//
// The rows of a workgroup are (token, query head) pairs of one sequence and one
// key head, 32 to a wave, so grouped heads share every key and value read; keys
// come in tiles of 64, filled into LDS by direct loads one tile ahead and shared
// by all waves.  Scores are formed transposed, S^T = K Q^T with 32x32x16 MFMAs, so
// that a lane holds 32 keys of ONE row: the softmax needs one exchange between
// the halves of the wave, and its weights are, without any further exchange, the
// B operand of the second product O^T = V^T P^T (the order of keys inside a
// contraction is free, and the transposing LDS read of V follows the order the
// scores come in).  Sums, maxima and scores are fp32; the weights are rounded to
// bf16 because the MFMA takes its operands in one type and V is bf16 (an output's
// error grows from 0.17% to 0.23% in the 2-norm, most of it the bf16 result).
//
// What bounds it: MFMA and vector ALU of a SIMD take about as long (32 MFMAs, 1024
// cycles, and some 180 vector instructions, 32 exponentials among them, for a wave's
// 32 rows and 64 keys), so two waves share a SIMD and take turns.  32 of the 180 are
// copies: the loop ends with two products or, on its last tile, one, and the compiler
// keeps the accumulator of D = 128 in a place of its own for each (16 copies at
// D = 64).  8192 tokens of 64 heads: 1.02 - 1.12 ms over boxes, 980 - 1075 TFLOP/s,
// 72 - 79% of the 1363 TFLOP/s of a large library bf16 GEMM on the same card; MFMAs
// are busy 51% of the cycles at 1.75 GHz (the clock is power-limited), LDS 25% with
// no bank conflicts.  With one barrier a tile instead of two the same prompt took
// 1.12 ms, with both waves of a SIMD in step 1.16 ms.  FP8 caches (codes converted
// once a workgroup, on the way into LDS; scales applied to scores and weights in
// fp32) run at 820 - 860 TFLOP/s: 2048 tokens over 32768 keys, 32 heads, 1.24 - 1.30
// ms.  MFMAs are busy 33% of the cycles there: 320 vector instructions for 32 MFMAs,
// and at D = 128 36 spilled registers (see the loop).
#include <hip/hip_runtime.h>

#include "attn_device.h"

namespace ptpc {
namespace {

enum Source { kPrompt, kPagedBf16, kPagedFp8 };

// LDS swizzles: 16-byte unit u of row r is stored at unit u ^ swz(r).  For keys
// the 16 lanes reading one unit of 16 consecutive rows, for values the 32 lanes
// of a transposing read (4 rows x 64 bytes), then touch every bank once.
template <int D>
__device__ __forceinline__ int swz_k(int r) {
    return D == 128 ? (r & 15) : ((r >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int swz_v(int r) {
    return D == 128 ? ((r & 3) << 2 | ((r >> 2) & 3)) : ((r >> 1) & 1) << 2;
}

// The row tile of a workgroup: tile `idx` when every sequence's rows are cut
// into tiles of BM, a sequence's last tile first (under the causal mask it sees
// the most keys, so the longest work starts first).  Returns the sequence or -1.
template <int BM>
__device__ __forceinline__ int find_tile(const AttnArgs& a, int G, int idx, int& tile) {
    const int lane = threadIdx.x & 63;
    const int T = (int)a.T;
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        int nt = 0;
        if (b0 + lane < a.B) {
            int c0 = a.cu[b0 + lane], c1 = a.cu[b0 + lane + 1];
            c0 = c0 < 0 ? 0 : c0 > T ? T : c0;
            c1 = c1 < c0 ? c0 : c1 > T ? T : c1;
            nt = ((c1 - c0) * G + BM - 1) / BM;
        }
        int incl = nt;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int o = __shfl_up(incl, m, 64);
            if (lane >= m) incl += o;
        }
        const uint64_t hit = __ballot(before + incl > idx);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int end = before + __shfl(incl, l, 64);
            tile = uniform(end - 1 - idx);
            return uniform(b0 + l);
        }
        before += __shfl(incl, 63, 64);
    }
    return -1;
}

template <int D, int NW, Source SRC>
__global__ __launch_bounds__(NW * 64, 2) void attn_tile_kernel(AttnArgs a, int splits, int chunk) {
    constexpr bool PAGED = SRC != kPrompt, FP8 = SRC == kPagedFp8;
    constexpr int BM = NW * 32, BN = 64;
    constexpr int RB = D * 2;                 // bytes of an LDS row
    constexpr int TILE = BN * RB;             // bytes of one K or V tile
    constexpr int NS = D / 16;                // k-steps of the first product
    constexpr int ND = D / 32;                // channel tiles of the second
    constexpr int UNITS = D / 8;
    constexpr int WROWS = BN / NW;            // rows a wave fills of each tile
    constexpr int LPR = 1024 / RB;            // rows of one 1 KB direct load
    constexpr int FILLS = WROWS / LPR;        // direct loads per wave and operand
    constexpr bool PAIRED = NW == 8;          // two waves to a SIMD take turns (see the loop)
    static_assert(WROWS <= 16, "a wave's rows lie in one page");

    // Two slots each, as objects of their own: the compiler then sees that reads of one
    // do not depend on the direct loads in flight into the others.
    __shared__ __attribute__((aligned(1024))) uint8_t k_lds0[TILE], k_lds1[TILE], v_lds0[TILE], v_lds1[TILE];
    __shared__ __attribute__((aligned(16))) float scales[FP8 ? 2 : 1][2][BN];
    __shared__ int odd[2][NW];                // nonfinite values in a wave's rows of V

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int G = a.q_heads / a.kv_heads;
    const int items = (int)gridDim.x / splits;
    const int split = (int)blockIdx.x / items, item = (int)blockIdx.x % items;
    const int hk = item % a.kv_heads;
    int tile = 0;
    const int b = find_tile<BM>(a, G, item / a.kv_heads, tile);
    if (b < 0) return;
    const Span sp = sequence_span(a, b, PAGED);
    const int rows = sp.n * G;
    const int row0 = tile * BM;
    const int row_end = row0 + BM < rows ? row0 + BM : rows;
    const int seen = visible(sp, row_end - 1, G);          // by the tile's last row
    const int parts = PAGED ? active_splits(seen, chunk, splits) : 1;
    if (split >= parts) return;
    const int lo = split * chunk;
    const int hi = split == parts - 1 ? seen : lo + chunk;

    // the lane's row
    const int w0 = row0 + wave * 32;
    const int r = w0 + col;
    const bool valid = r < rows;
    const int vis = visible(sp, r, G);
    const bool works = w0 < rows;
    const int wave_min = works ? visible(sp, w0, G) : 0;
    const int wave_max = works ? visible(sp, w0 + 31 < rows ? w0 + 31 : rows - 1, G) : 0;
    const int tile_min = visible(sp, row0, G);
    const int64_t token = sp.start + r / G;
    const int head = hk * G + r % G;

    u32x4 q[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        q[s] = u32x4{0, 0, 0, 0};
        if (valid)
            q[s] = flip_sign(*reinterpret_cast<const u32x4*>(a.q + token * a.ldq + (int64_t)head * D +
                                                             16 * s + 8 * half), a.scale);
    }
    const float c = score_factor(a.scale);

    // ---- fills -----------------------------------------------------------------
    // Wave w fills rows w * WROWS .. of each tile (one page holds them all).
    const int pitch_k = PAGED ? (FP8 ? D : RB) : (int)(a.ldk * 2);
    const int pitch_v = PAGED ? (FP8 ? D : RB) : (int)(a.ldv * 2);
    int off_k[FILLS], off_v[FILLS];
#pragma unroll
    for (int i = 0; i < FILLS; ++i) {
        const int rr = i * LPR + lane / UNITS, u = lane % UNITS;
        const int tr = wave * WROWS + rr;
        off_k[i] = rr * pitch_k + ((u ^ swz_k<D>(tr)) * 16);
        off_v[i] = rr * pitch_v + ((u ^ swz_v<D>(tr)) * 16);
    }
    // page of the wave's rows of the tile at key k0 (past the sequence's end any page: the
    // entry lies in the table and is cut to the cache)
    auto page_of = [&](int k0) -> int {
        if constexpr (!PAGED) return 0;
        int j = k0 + wave * WROWS;
        j = j < a.table_keys ? j : a.table_keys - 1;
        const int p = scalar_at(a.page_table, (int64_t)b * a.ld_table + (j >> a.cache.page_shift));
        return (uint32_t)p < (uint32_t)a.cache.pages ? p : 0;
    };
    // element row of the wave's first row of a tile, and how many of its rows hold keys
    auto rows_at = [&](int k0, int page, int64_t& first) -> int {
        const int j = k0 + wave * WROWS;
        first = PAGED ? (((int64_t)page * a.kv_heads + hk) << a.cache.page_shift) +
                            (j & ((1 << a.cache.page_shift) - 1))
                      : (int64_t)sp.start + j;
        return clamp_rows(hi - j, WROWS);
    };
    // The operand's LDS slot (s is a compile-time constant after inlining).
#define K_SLOT(s) ((s) == 0 ? k_lds0 : k_lds1)
#define V_SLOT(s) ((s) == 0 ? v_lds0 : v_lds1)
    auto fill = [&](uint8_t* slot, const uint16_t* packed, int64_t ld, const uint8_t* paged, int pitch,
                    const int (&off)[FILLS], int k0, int page) {
        int64_t first;
        const int have = rows_at(k0, page, first);         // rows past the range become zero
        const void* base = PAGED ? paged + first * RB
                                 : reinterpret_cast<const uint8_t*>(packed + first * ld + (int64_t)hk * D);
        const auto buf = wave_buffer(base, 0, have ? (have - 1) * pitch + RB : 0);
#pragma unroll
        for (int i = 0; i < FILLS; ++i) load_to_lds(buf, slot + (wave * WROWS + i * LPR) * RB, off[i]);
    };
    // E4M3: codes through registers, written to LDS as bf16 (each code is converted once
    // per workgroup, exactly); lane -> row lane * 16 / D of the wave's rows, 16 codes.
    constexpr int CPL = WROWS * D / 16 / 64 > 0 ? WROWS * D / 16 / 64 : 1;   // 16-code pieces per lane
    constexpr bool PARTIAL = WROWS * D / 16 < 64;                            // lanes without a piece
    u32x4 ck[CPL], cv[CPL];
    float cs = 0.0f;
    auto fetch = [&](u32x4 (&w)[CPL], const uint8_t* codes, int k0, int page) {
        int64_t first;
        const int have = rows_at(k0, page, first);
        const auto buf = wave_buffer(codes, first * D, have * D);
#pragma unroll
        for (int i = 0; i < CPL; ++i) w[i] = buffer_load16(buf, (i * 64 + lane) * 16);
    };
    auto fetch_scales = [&](int k0, int page) {            // lanes 0 .. : keys' scales, 32 .. : values'
        int64_t first;
        const int have = rows_at(k0, page, first);
        const float sk = buffer_load4(wave_buffer(a.cache.dk, first * 4, have * 4), (lane & 31) * 4);
        const float sv = buffer_load4(wave_buffer(a.cache.dv, first * 4, have * 4), (lane & 31) * 4);
        cs = lane < 32 ? sk : sv;
    };
    auto put = [&](uint8_t* slot, const u32x4 (&w)[CPL], bool keys) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            const int piece = i * 64 + lane;
            const int tr = wave * WROWS + piece / (D / 16), u = (piece % (D / 16)) * 2;
            const int swz = keys ? swz_k<D>(tr) : swz_v<D>(tr);
            const u32x4 x = w[i];
            const u32x4 lo4{e4m3x2_to_bf16x2<false>(x.x), e4m3x2_to_bf16x2<true>(x.x),
                            e4m3x2_to_bf16x2<false>(x.y), e4m3x2_to_bf16x2<true>(x.y)};
            const u32x4 hi4{e4m3x2_to_bf16x2<false>(x.z), e4m3x2_to_bf16x2<true>(x.z),
                            e4m3x2_to_bf16x2<false>(x.w), e4m3x2_to_bf16x2<true>(x.w)};
            if (!PARTIAL || piece < WROWS * D / 16) {
                *reinterpret_cast<u32x4*>(slot + tr * RB + ((u ^ swz) * 16)) = lo4;
                *reinterpret_cast<u32x4*>(slot + tr * RB + (((u + 1) ^ swz) * 16)) = hi4;
            }
        }
    };
    auto put_scales = [&](int slot) {
        if ((lane & 31) < WROWS) scales[slot][lane >> 5][wave * WROWS + (lane & 31)] = cs;
    };
    // The wave's rows of a V tile that some row of the workgroup sees only in part: nonfinite
    // values are set to zero (a masked key's weight is 0, but 0 times them is not), and the
    // keys that hold any are noted as a bit mask in odd[slot][wave].
    auto look = [&](int slot) {
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < FILLS; ++i) {
            u32x4* at = reinterpret_cast<u32x4*>(V_SLOT(slot) + (wave * WROWS + i * LPR) * RB + lane * 16);
            const u32x4 w = *at;
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= nonfinite2(w[e]);
            const uint64_t lanes = __ballot(bad);
            if (lanes) {
                *at = finite_part(w);
#pragma unroll
                for (int rr = 0; rr < LPR; ++rr)
                    if (lanes >> (rr * UNITS) & ((1ull << UNITS) - 1)) mask |= 1u << (i * LPR + rr);
            }
        }
        if (lane == 0) odd[slot][wave] = mask;
    };
    // ---- LDS read addresses -------------------------------------------------------
    int addr_k[NS], addr_v[ND][2];
#pragma unroll
    for (int s = 0; s < NS; ++s)
        addr_k[s] = col * RB + (((2 * s + half) ^ swz_k<D>(col)) * 16);
    const int i16 = lane & 15, grp = (lane >> 4) & 1;
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int kr = 8 * p + 4 * half + i16 / 4;
            const int u = t * 4 + 2 * grp + (i16 % 4) / 2;
            addr_v[t][p] = kr * RB + ((u ^ swz_v<D>(kr)) * 16) + 8 * (i16 & 1);
        }
    auto read_v = [&](int slot, int t, int ks) -> u32x4 {
        const uint8_t* at = V_SLOT(slot) + ks * 16 * RB;
        const u32x2 x = read_keys4(at + addr_v[t][0]), y = read_keys4(at + addr_v[t][1]);
        return u32x4{x.x, x.y, y.x, y.y};
    };

    // ---- the loop over key tiles ----------------------------------------------------
    float m = -INFINITY, l = 0.0f;
    v16f o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[t][e] = 0.0f;

    v16f s[2];                                // scores: register e of s[t] is key
    u32x4 p[4];                               // k0 + 32 t + 8 (e / 4) + 4 half + e % 4 of the lane's row
    auto scores = [&](int slot) {             // S^T = K Q^T
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < NS; ++ks)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const u32x4 kf = *reinterpret_cast<const u32x4*>(K_SLOT(slot) + t * 32 * RB + addr_k[ks]);
                s[t] = mfma32(kf, q[ks], s[t]);
            }
    };
    auto gather = [&](int slot) {             // O^T += V^T P^T
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int t = 0; t < ND; ++t) o[t] = mfma32(read_v(slot, t, ks), p[ks], o[t]);
    };
    // Weights of the tile at k0, the running maximum and sum.
    auto weigh = [&](int k0, int slot) {
        if constexpr (FP8) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 d = *reinterpret_cast<const float4*>(&scales[slot][0][32 * t + 8 * g + 4 * half]);
                    s[t][4 * g] *= d.x; s[t][4 * g + 1] *= d.y; s[t][4 * g + 2] *= d.z; s[t][4 * g + 3] *= d.w;
                }
        }
        const bool masked = k0 + BN > wave_min;
        const int rel = vis - k0 - 4 * half;
        if (masked) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    s[t][e] = 32 * t + 8 * (e / 4) + e % 4 < rel ? s[t][e] : -INFINITY;
        }
        float mx = max3(s[0][0], s[0][1], s[1][0]);
#pragma unroll
        for (int e = 2; e < 16; e += 2) mx = max3(s[0][e], s[0][e + 1], mx);
#pragma unroll
        for (int e = 1; e < 15; e += 2) mx = max3(s[1][e], s[1][e + 1], mx);
        mx = half_max(max3(mx, s[1][15], mx)) * c;
        if (__any(mx > m + kRescaleAt)) {
            const float mn = fmaxf(m, mx);
            const float f = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
            l *= f;
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[t][e] *= f;
            m = mn;
        }
        const float shift = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[t][e] = exp2_fast(__builtin_fmaf(s[t][e], c, -shift));
                l += s[t][e];
            }
            if constexpr (FP8) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 d = *reinterpret_cast<const float4*>(&scales[slot][1][32 * t + 8 * g + 4 * half]);
                    s[t][4 * g] *= d.x; s[t][4 * g + 1] *= d.y; s[t][4 * g + 2] *= d.z; s[t][4 * g + 3] *= d.w;
                }
                if (masked) {          // a masked key's scale may be anything
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        s[t][e] = 32 * t + 8 * (e / 4) + e % 4 < rel ? s[t][e] : 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                p[2 * t + e / 4][e % 4] = f32x2_to_bf16x2_rne(s[t][2 * e], s[t][2 * e + 1]);
        }
    };
    // The nonfinite values that look() took out of a tile, added (as memory holds them) for the
    // rows that see their keys.
    auto add_nonfinite = [&](int k0, int slot) {
        for (int w = 0; w < NW; ++w) {
            for (uint32_t mask = uniform(odd[slot][w]); mask; mask &= mask - 1) {
                const int j = k0 + w * WROWS + __builtin_ctz(mask);
                int64_t at = (int64_t)sp.start + j;
                if constexpr (PAGED) {
                    const int pg = scalar_at(a.page_table, (int64_t)b * a.ld_table + (j >> a.cache.page_shift));
                    at = ((((int64_t)((uint32_t)pg < (uint32_t)a.cache.pages ? pg : 0) * a.kv_heads + hk)
                           << a.cache.page_shift) + (j & ((1 << a.cache.page_shift) - 1)));
                }
                const uint8_t* row = PAGED ? a.cache.v + at * (FP8 ? D : RB)
                                           : reinterpret_cast<const uint8_t*>(a.v + at * a.ldv + (int64_t)hk * D);
                const bool sees = j < vis;
#pragma unroll
                for (int t = 0; t < ND; ++t)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int d = 32 * t + 8 * g + 4 * half;
                        float x[4];
                        if constexpr (FP8) {
                            const uint32_t w4 = nan_bits4(*reinterpret_cast<const uint32_t*>(row + d));
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] = w4 >> (8 * e) & 0x80 ? __builtin_nanf("") : 0.0f;
                        } else {
                            const uint2 w4 = *reinterpret_cast<const uint2*>(row + 2 * d);
                            x[0] = bf16lo_to_f32(w4.x); x[1] = bf16hi_to_f32(w4.x);
                            x[2] = bf16lo_to_f32(w4.y); x[3] = bf16hi_to_f32(w4.y);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (sees && !__builtin_isfinite(x[e])) o[t][4 * g + e] += x[e];
                    }
            }
        }
    };

    // Two phases a tile: MFMAs (the last tile's second product and this tile's first), and
    // the softmax on the vector ALU.  Where a SIMD holds two waves of the workgroup (PAIRED)
    // the second of them runs one phase behind, so one wave's MFMAs run under the other's
    // softmax; a barrier ends each phase.  In MFMA phase i of the first waves everyone starts
    // the fills of keys i + 1 and values i, whose slots were last read the phase before, and
    // waits for them at the end of the next phase.  (In the E4M3 kernels of D = 128 the wait
    // comes sooner: registers are spilled, and two reloads inside the MFMA phase, seven with
    // 128 rows, wait for every load before them, the codes on their way among them.)
    const int tiles = (hi - lo + BN - 1) / BN;
    if (tiles > 0) {
        const int mine = wave_max <= lo ? 0 : wave_max >= hi ? tiles : (wave_max - lo + BN - 1) / BN;
        int page = page_of(lo), page_next = page_of(lo + BN);
        auto start_keys = [&](int i, int pg, int slot) {
            poison_refill(K_SLOT(slot) + wave * WROWS * RB, FILLS);
            if constexpr (FP8) {
                fetch(ck, a.cache.k, lo + i * BN, pg);
                fetch_scales(lo + i * BN, pg);
            } else {
                fill(K_SLOT(slot), a.k, a.ldk, a.cache.k, pitch_k, off_k, lo + i * BN, pg);
            }
        };
        auto start_fills = [&](int i, int slot) {          // keys i + 1, values i; slot = i % 2
            start_keys(i + 1, page_next, slot ^ 1);
            poison_refill(V_SLOT(slot) + wave * WROWS * RB, FILLS);
            if constexpr (FP8) fetch(cv, a.cache.v, lo + i * BN, page);
            else fill(V_SLOT(slot), a.v, a.ldv, a.cache.v, pitch_v, off_v, lo + i * BN, page);
            page = page_next;
            page_next = page_of(lo + (i + 2) * BN);
        };
        auto end_fills = [&](int i, int slot) {
            if constexpr (FP8) {
                put(K_SLOT(slot ^ 1), ck, true);
                put(V_SLOT(slot), cv, false);
                put_scales(slot ^ 1);
            } else {
                wait_loads();
            }
            if (lo + (i + 1) * BN > tile_min) {
                wait_lds();
                look(slot);
            }
            wait_lds();
        };

        start_keys(0, page, 0);
        if constexpr (FP8) {
            put(K_SLOT(0), ck, true);
            put_scales(0);
            wait_lds();
        } else {
            wait_loads();
        }
        attn_barrier();
        start_fills(0, 0);
        // (the loop is compiled once for each kind of wave: with `late` tested inside, the
        // compiler could not tell which fills are in flight and would wait for all)
        auto loop = [&](const bool late) __attribute__((always_inline)) {
            if (late) attn_barrier();
            if (mine > 0) scores(0);
            if (late) end_fills(0, 0);
            auto step = [&](int i, int slot) __attribute__((always_inline)) {
                if constexpr (PAIRED) attn_barrier();
                if (late) start_fills(i + 1, slot ^ 1);
                if (i < mine) weigh(lo + i * BN, slot);
                if (!late) end_fills(i, slot);
                attn_barrier();
                if (!late) start_fills(i + 1, slot ^ 1);
                if (lo + (i + 1) * BN > tile_min && i < mine) {
                    uint32_t any = 0;
#pragma unroll
                    for (int w = 0; w < NW; ++w) any |= odd[slot][w];
                    if (uniform(any)) add_nonfinite(lo + i * BN, slot);
                }
                if (i + 1 < mine) {
                    gather(slot);
                    scores(slot ^ 1);
                    // reads run a few MFMAs ahead of their use
                    constexpr int PV = 4 * ND, QK = 2 * NS;
                    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
                    for (int n = 0; n < PV + QK; ++n) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        if (n < PV - 4) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    }
                } else if (i < mine) {
                    gather(slot);
                }
                if (late) end_fills(i + 1, slot ^ 1);
            };
            for (int i = 0;;) {
                step(i, 0);
                if (++i == tiles) break;
                step(i, 1);
                if (++i == tiles) break;
            }
            if (PAIRED && !late) attn_barrier();
        };
        if (PAIRED && wave >= NW / 2) loop(true);
        else loop(false);
        wait_loads();                        // (fills of zeros past the range)
    }

    // ---- results -----------------------------------------------------------------------
    l = half_sum(l);
    if (!valid) return;
    if (parts == 1) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        uint16_t* dst = a.out + token * a.ldo + (int64_t)head * D + 4 * half;
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<uint2*>(dst + 32 * t + 8 * g) = make_uint2(
                    f32x2_to_bf16x2_rne(o[t][4 * g] * inv, o[t][4 * g + 1] * inv),
                    f32x2_to_bf16x2_rne(o[t][4 * g + 2] * inv, o[t][4 * g + 3] * inv));
    } else {
        const int64_t at = ((int64_t)item * splits + split) * BM + wave * 32 + col;
        float* dst = a.ws + at * D + 4 * half;
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<v4f*>(dst + 32 * t + 8 * g) =
                    v4f{o[t][4 * g], o[t][4 * g + 1], o[t][4 * g + 2], o[t][4 * g + 3]};
        if (half == 0) part_stats(a, items, splits, BM, D)[at] = make_float2(m, l);
    }
}

#undef K_SLOT
#undef V_SLOT

// Join of the ranges of a tile's rows, join_rows of them a workgroup, a quarter of them a wave
// one after another: 32 where that still makes rounds of workgroups (finding the tile takes
// as long as a few rows), else 4.  Four 70B chunks (27000 workgroups of 4 rows): 45 us with 4
// rows, 25 us with 32; 72 rows of 8 sequences (3200): the call takes 31 us with 4, 40 with 32.
template <int D, int BM>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(AttnArgs a, int splits, int chunk, int join_rows) {
    const int per = BM / join_rows;
    const int item = (int)blockIdx.x / per;
    const int first = (int)blockIdx.x % per * join_rows + uniform(threadIdx.x >> 6);
    const int G = a.q_heads / a.kv_heads, hk = item % a.kv_heads;
    int tile = 0;
    const int b = find_tile<BM>(a, G, item / a.kv_heads, tile);
    if (b < 0) return;
    const Span sp = sequence_span(a, b, true);
    const int rows = sp.n * G;
    const int row_end = tile * BM + BM < rows ? tile * BM + BM : rows;
    const int parts = active_splits(visible(sp, row_end - 1, G), chunk, splits);
    if (parts == 1) return;
    for (int rr = first; rr < first + join_rows && tile * BM + rr < rows; rr += 4) {
        const int r = tile * BM + rr;
        join_row<D>(a, (int)gridDim.x / per, splits, BM, item, rr, parts,
                    a.out + (int64_t)(sp.start + r / G) * a.ldo + (int64_t)(hk * G + r % G) * D);
    }
}

template <int D, int NW, Source SRC>
void launch_tiles(const AttnArgs& a, int64_t items, int splits, int chunk, hipStream_t s) {
    attn_tile_kernel<D, NW, SRC><<<(unsigned)(items * splits), NW * 64, 0, s>>>(a, splits, chunk);
    if constexpr (SRC != kPrompt)
        if (splits > 1) {
            const int join_rows = items * (NW * 8) > 8192 ? 32 : 4;
            attn_tile_join_kernel<D, NW * 32><<<(unsigned)(items * (NW * 32 / join_rows)), 256, 0, s>>>(
                a, splits, chunk, join_rows);
        }
}

template <Source SRC>
void dispatch(const AttnArgs& a, int tile_rows, int64_t items, int splits, int chunk, hipStream_t s) {
    if (a.D == 128) {
        if (tile_rows == kLargeTile) launch_tiles<128, 8, SRC>(a, items, splits, chunk, s);
        else launch_tiles<128, 4, SRC>(a, items, splits, chunk, s);
    } else {
        if (tile_rows == kLargeTile) launch_tiles<64, 8, SRC>(a, items, splits, chunk, s);
        else launch_tiles<64, 4, SRC>(a, items, splits, chunk, s);
    }
}

}  // namespace

hipError_t launch_attn_tiles(const AttnArgs& a, const PagedPlan& p, hipStream_t s) {
    if (a.cache.fp8) dispatch<kPagedFp8>(a, p.tile_rows, p.items, p.splits, p.chunk, s);
    else dispatch<kPagedBf16>(a, p.tile_rows, p.items, p.splits, p.chunk, s);
    return hipGetLastError();
}

hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t s) {
    const int64_t G = a.q_heads / a.kv_heads;
    // Tiles of 256 rows read keys and values half as often, tiles of 128 (two workgroups a CU)
    // spread a small batch better: 4099 tokens of 12 prompts, 32 query heads, 49 us with 256
    // rows (2 rounds of the GPU) and 44 us with 128; 8192 tokens, 64 heads (8 rounds) 1070
    // and 1082 us.
    const int tile = a.T * a.q_heads >= 4 * 256 * kLargeTile ? (int)kLargeTile : (int)kSmallTile;
    const int64_t items = (a.T * G / tile + a.B) * a.kv_heads;
    dispatch<kPrompt>(a, tile, items, 1, INT32_MAX / 2, s);
    return hipGetLastError();
}

}  // namespace ptpc
