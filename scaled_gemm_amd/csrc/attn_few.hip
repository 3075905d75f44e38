// Attention of few query rows over the paged cache: single tokens, and a few
// drafted ones.
//
// The rows of a sequence and key head -- new tokens times the heads of the group
// -- are one row tile of up to 16 NT, or a few such tiles side by side, so each
// key and value is read once.  The four waves of a workgroup take blocks of 32
// keys in turn and never wait for one another: a wave loads its keys straight into
// registers, in the order the MFMA takes them, and its values into LDS slots of its
// own, both one block ahead.  Scores are formed transposed with 16x16x32 MFMAs,
// S^T = K Q^T, so a lane holds keys of one row, and its weights are the B operand of
// O^T = V^T P^T as they stand (bf16 weights, fp32 sums, as in the tile kernel).
// The waves' results are joined in LDS, the ranges of a long context by a second
// kernel from fp32 parts in the workspace.
//
// What bounds it: HBM.  96 sequences over up to 32768 keys, 8 key heads, E4M3 (2.46
// GB): 443 us, 5.6 TB/s, against 5.8 TB/s of a read-only torch sum; 32 sequences over
// up to 8192 bf16 keys (0.31 GB): 75 us, 4.1 TB/s, of which 5 us are the join and the
// rest start and end (a workgroup's start, first loads and join take some 6 us).  A
// third workgroup a CU (fewer registers) spilled and was 20 - 60% slower.
#include <hip/hip_runtime.h>

#include "attn_device.h"

namespace ptpc {
namespace {

// Swizzle of the value rows in LDS (16-byte unit u of row r is stored at unit
// u ^ swz(r)): the 32 lanes that a transposing read serves at a time touch every
// bank once -- bf16: 8 rows x 32 bytes, E4M3: 16 rows x 16 bytes.
template <int D, bool FP8>
__device__ __forceinline__ int swz(int r) {
    if (FP8) return D == 128 ? ((r >> 1) & 3) | ((r >> 4) & 1) << 2 : ((r >> 2) & 1) | ((r >> 4) & 1) << 1;
    return D == 128 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
}

template <int D, bool FP8, int NT>
__global__ __launch_bounds__(256, 2) void attn_few_kernel(AttnArgs a, int tile_rows, int row_tiles,
                                                          int splits, int chunk) {
    constexpr int NW = 4;
    constexpr int KB = 32;                     // keys of a block
    constexpr int SB = KB / 16;                // 16-key groups (one page each)
    constexpr int RB = FP8 ? D : 2 * D;        // bytes of a cached row
    constexpr int UNITS = RB / 16;
    constexpr int SLOT = KB * RB;              // a wave's values of a block
    constexpr int RPS = SLOT / (4 * D);        // rows of fp32 sums that fit a slot
    constexpr int LPR = 1024 / RB;             // rows of one direct load
    constexpr int FILLS = 16 / LPR;            // direct loads of one 16-key group
    constexpr int KL = RB / 64;                // 16-byte loads per lane and key group
    constexpr int NS = D / 32;                 // k-steps of the first product
    constexpr int ND = D / 16;                 // channel tiles of the second
    constexpr int LOADS = SB * (KL + FILLS + (FP8 ? 2 : 0));   // of one block
    static_assert(2 * RPS >= 16, "the waves' results reuse their two value slots");

    __shared__ __attribute__((aligned(1024))) uint8_t lds0[NW][SLOT], lds1[NW][SLOT];
    __shared__ float stat[NW][2][16];     // reference maximum and weights' sum

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int G = a.q_heads / a.kv_heads;
    const int items = (int)gridDim.x / splits;
    const int split = (int)blockIdx.x / items, item = (int)blockIdx.x % items;
    // a pair's row tiles lie B * kv_heads apart: on one XCD (its L2) where that is a multiple of 8
    const int pair = item % (a.B * a.kv_heads), hk = pair % a.kv_heads, b = pair / a.kv_heads;
    const int rt = item / (a.B * a.kv_heads);
    // Pages of a block's 16-key groups.  Past the sequence's end this may read entries that
    // mean nothing (but lie in the table, and are cut to the cache), so the first block's
    // need not wait for the sequence's length.
    int pages[SB];
    auto pages_of = [&](int k0) {
#pragma unroll
        for (int t = 0; t < SB; ++t) {
            int j = k0 + 16 * t;
            j = j < a.table_keys ? j : a.table_keys - 1;
            const int p = scalar_at(a.page_table, (int64_t)b * a.ld_table + (j >> a.cache.page_shift));
            pages[t] = (uint32_t)p < (uint32_t)a.cache.pages ? p : 0;
        }
    };
    if (a.table_keys == 0) pages[0] = pages[SB - 1] = 0;
    else pages_of(split * chunk + wave * KB);
    const Span sp = sequence_span(a, b, true);
    const int rows = sp.n * G;
    const float c = score_factor(a.scale);

    // The item's row tile is split over workgroups; should a sequence have more new tokens
    // than the launch was sized for, the item's first workgroup does the further tiles alone.
    for (int row0 = rt * tile_rows; row0 < rows; row0 += row_tiles * tile_rows) {
        const bool first = row0 == rt * tile_rows;
        if (!first && split != 0) break;
        const int row_end = row0 + tile_rows < rows ? row0 + tile_rows : rows;
        const int seen = visible(sp, row_end - 1, G), least = visible(sp, row0, G);
        const int parts = first ? active_splits(seen, chunk, splits) : 1;
        if (split >= parts) break;
        const int lo = split * chunk;
        const int hi = split == parts - 1 ? seen : lo + chunk;

        int vis[NT];
        u32x4 q[NT][NS];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + 16 * n + i16;
            vis[n] = visible(sp, r, G);
            const uint16_t* src = a.q + (int64_t)(sp.start + r / G) * a.ldq + (int64_t)(hk * G + r % G) * D;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                // channels of k-step s in lane group g, as the key loads bring them
                const int d = FP8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
                q[n][s] = u32x4{0, 0, 0, 0};
                if (r < row_end) q[n][s] = flip_sign(*reinterpret_cast<const u32x4*>(src + d), a.scale);
            }
        }

        // ---- loads ---------------------------------------------------------------------
        u32x4 key[2][SB][KL];
        v4f dk[2][FP8 ? SB : 1], dv[2][FP8 ? SB : 1];
        int off_v[FILLS];
#pragma unroll
        for (int i = 0; i < FILLS; ++i) {
            const int r = i * LPR + lane / UNITS;
            off_v[i] = r * RB;
        }
        // rows past the range's end come as zeros (and cost no traffic)
        auto load = [&](int k0, int slot) {
            poison_refill((slot ? lds1 : lds0)[wave], SLOT / 1024);
#pragma unroll
            for (int t = 0; t < SB; ++t) {
                const int j = k0 + 16 * t;
                const int64_t row = (((int64_t)pages[t] * a.kv_heads + hk) << a.cache.page_shift) +
                                    (j & ((1 << a.cache.page_shift) - 1));
                const int have = clamp_rows(hi - j, 16);
                const auto rk = wave_buffer(a.cache.k, row * RB, have * RB);
                const auto rv = wave_buffer(a.cache.v, row * RB, have * RB);
#pragma unroll
                for (int s = 0; s < KL; ++s)
                    key[slot][t][s] = buffer_load16(rk, i16 * RB + 64 * s + 16 * g);
                if constexpr (FP8) {
                    const auto sk = wave_buffer(a.cache.dk, row * 4, have * 4);
                    const auto sv = wave_buffer(a.cache.dv, row * 4, have * 4);
                    dk[slot][t] = __builtin_bit_cast(v4f, buffer_load16(sk, 16 * g));
                    dv[slot][t] = __builtin_bit_cast(v4f, buffer_load16(sv, 16 * g));
                }
#pragma unroll
                for (int i = 0; i < FILLS; ++i) {
                    const int r = 16 * t + i * LPR + lane / UNITS;
                    load_to_lds(rv, (slot ? lds1 : lds0)[wave] + (16 * t + i * LPR) * RB,
                                off_v[i] + ((lane % UNITS) ^ swz<D, FP8>(r)) * 16);
                }
            }
        };

        // ---- one block -------------------------------------------------------------------
        float m[NT], l[NT];
        v4f o[NT][ND];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.0f;
#pragma unroll
            for (int t = 0; t < ND; ++t) o[n][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        auto k_frag = [&](int slot, int t, int s) -> u32x4 {
            if constexpr (!FP8) return key[slot][t][s];
            const u32x4 w = key[slot][t][s / 2];
            const uint32_t x = s % 2 ? w.z : w.x, y = s % 2 ? w.w : w.y;
            return u32x4{e4m3x2_to_bf16x2<false>(x), e4m3x2_to_bf16x2<true>(x),
                         e4m3x2_to_bf16x2<false>(y), e4m3x2_to_bf16x2<true>(y)};
        };
        // keys 32 h + 4 g + (0 .. 3), 32 h + 16 + 4 g + (0 .. 3) of channel 16 t + i16
        auto v_frag = [&](int slot, int h, int t) -> u32x4 {
            const uint8_t* base = (slot ? lds1 : lds0)[wave];
            if constexpr (FP8) {
                const int jj = i16 / 2, r = 32 * h + (jj < 4 ? 4 * g + jj : 12 + 4 * g + jj);
                const u32x2 w = read_keys8(base + r * RB + ((t ^ swz<D, true>(r)) * 16) + 8 * (i16 % 2));
                return u32x4{e4m3x2_to_bf16x2<false>(w.x), e4m3x2_to_bf16x2<true>(w.x),
                             e4m3x2_to_bf16x2<false>(w.y), e4m3x2_to_bf16x2<true>(w.y)};
            }
            const int r = 32 * h + 4 * g + i16 / 4, u = 2 * t + (i16 % 4) / 2;
            const int at = ((u ^ swz<D, false>(r)) * 16) + 8 * (i16 & 1);      // the same for r + 16
            const u32x2 x = read_keys4(base + r * RB + at), y = read_keys4(base + (r + 16) * RB + at);
            return u32x4{x.x, x.y, y.x, y.y};
        };
        // Values that are not finite, of keys that some row of the tile does not see: added
        // for the rows that see them, and set to zero in LDS (0 times them is not 0).
        auto apart = [&](int k0, int slot) {
            uint8_t* base = (slot ? lds1 : lds0)[wave];
            for (int i = 0; i < SB * FILLS; ++i) {
                u32x4* at = reinterpret_cast<u32x4*>(base + i * 1024 + lane * 16);
                const u32x4 w = *at;
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) bad |= FP8 ? nan_code4(w[e]) : nonfinite2(w[e]);
                const uint64_t lanes = __ballot(bad);
                if (lanes == 0) continue;
                for (int rr = 0; rr < LPR; ++rr) {
                    if (!(lanes >> (rr * UNITS) & ((1ull << UNITS) - 1))) continue;
                    const int r = i * LPR + rr;
#pragma unroll
                    for (int t = 0; t < ND; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {          // channel 16 t + 4 g + e
                            const int d = 16 * t + 4 * g + e;
                            const int byte = FP8 ? d : 2 * d;
                            const uint8_t* p = base + r * RB + (((byte / 16) ^ swz<D, FP8>(r)) * 16) + byte % 16;
                            float x;
                            if constexpr (FP8) x = (*p & 0x7F) == 0x7F ? __builtin_nanf("") : 0.0f;
                            else x = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
                            if (!__builtin_isfinite(x)) {
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    if (k0 + r < vis[n]) o[n][t][e] += x;
                            }
                        }
                }
                wait_lds();
                if constexpr (FP8)
                    *at = u32x4{number_codes4(w.x), number_codes4(w.y), number_codes4(w.z),
                                number_codes4(w.w)};
                else
                    *at = finite_part(w);
            }
            wait_lds();
        };

        auto block = [&](int k0, int slot) {
            const bool masked = k0 + KB > least;
            u32x4 p[NT][KB / 32];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                v4f s[SB];
#pragma unroll
                for (int t = 0; t < SB; ++t) {
                    s[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int ks = 0; ks < NS; ++ks) s[t] = mfma16(k_frag(slot, t, ks), q[n][ks], s[t]);
                    if constexpr (FP8) s[t] *= dk[slot][t];
                }
                const int rel = vis[n] - k0 - 4 * g;          // key 16 t + 4 g + e is seen if 16 t + e < rel
                if (masked) {
#pragma unroll
                    for (int t = 0; t < SB; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[t][e] = 16 * t + e < rel ? s[t][e] : -INFINITY;
                }
                float mx = s[0][0];
#pragma unroll
                for (int t = 0; t < SB; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[t][e]);
                mx = quarter_max(mx) * c;
                if (__any(mx > m[n] + kRescaleAt)) {
                    const float mn = fmaxf(m[n], mx);
                    const float f = mn == -INFINITY ? 1.0f : exp2_fast(m[n] - mn);
                    l[n] *= f;
#pragma unroll
                    for (int t = 0; t < ND; ++t) o[n][t] *= f;
                    m[n] = mn;
                }
                const float shift = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
                for (int t = 0; t < SB; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[t][e] = exp2_fast(__builtin_fmaf(s[t][e], c, -shift));
                        l[n] += s[t][e];
                    }
                    if constexpr (FP8) {
                        s[t] *= dv[slot][t];
                        if (masked) {                        // a masked key's scale may be anything
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[t][e] = 16 * t + e < rel ? s[t][e] : 0.0f;
                        }
                    }
                    p[n][t / 2][2 * (t % 2)] = f32x2_to_bf16x2_rne(s[t][0], s[t][1]);
                    p[n][t / 2][2 * (t % 2) + 1] = f32x2_to_bf16x2_rne(s[t][2], s[t][3]);
                }
            }
            if (masked && least < sp.kv) apart(k0, slot);
#pragma unroll
            for (int h = 0; h < KB / 32; ++h)
#pragma unroll
                for (int t = 0; t < ND; ++t) {
                    const u32x4 v = v_frag(slot, h, t);
#pragma unroll
                    for (int n = 0; n < NT; ++n) o[n][t] = mfma16(v, p[n][h], o[n][t]);
                }
        };

        // ---- the wave's blocks: wave, wave + 4, ... -----------------------------------------
        const int blocks = (hi - lo + KB - 1) / KB;
        if (wave < blocks) {
            if (!first) pages_of(wave * KB);
            load(lo + wave * KB, 0);
            pages_of(lo + (wave + NW) * KB);
            auto step = [&](int i, int slot) {
                const int k0 = lo + i * KB;
                // always one block ahead, past the end too: with a branch here the compiler's
                // counting of loads would wait for the next block's keys
                load(k0 + NW * KB, slot ^ 1);
                pages_of(k0 + 2 * NW * KB);
                wait_loads_but<LOADS>();
                block(k0, slot);
                wait_lds();              // this slot's reads are done before it is filled again
            };
            for (int i = wave;;) {
                step(i, 0);
                if ((i += NW) >= blocks) break;
                step(i, 1);
                if ((i += NW) >= blocks) break;
            }
            wait_loads();                // (fills of zeros included) before the slots are reused
        }

        // ---- join of the four waves: 16 rows at a time, through the wave's value slots --------
        auto sums = [&](int w, int r) {          // fp32 sums of row r of the 16 by wave w
            return reinterpret_cast<float*>(r < RPS ? lds0[w] : lds1[w]) + r % RPS * D;
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] = quarter_sum(l[n]);
#pragma unroll
            for (int t = 0; t < ND; ++t)
                *reinterpret_cast<v4f*>(sums(wave, i16) + (((4 * t + g) ^ i16) * 4)) = o[n][t];
            if (g == 0) {
                stat[wave][0][i16] = m[n];
                stat[wave][1][i16] = l[n];
            }
            __syncthreads();
            const int row_n = row0 + 16 * n;
            const int count = row_end - row_n < 16 ? row_end - row_n : 16;
            for (int i = threadIdx.x; i < count * (D / 4); i += 256) {
                const int r = i / (D / 4), u = i % (D / 4);
                float mt = stat[0][0][r];
#pragma unroll
                for (int w = 1; w < NW; ++w) mt = fmaxf(mt, stat[w][0][r]);
                const float shift = mt == -INFINITY ? 0.0f : mt;
                float lt = 0.0f;
                v4f ot{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float f = exp2_fast(stat[w][0][r] - shift);
                    lt += stat[w][1][r] * f;
                    ot += *reinterpret_cast<const v4f*>(sums(w, r) + ((u ^ r) * 4)) * f;
                }
                if (parts == 1) {
                    const float inv = lt > 0.0f || lt != lt ? 1.0f / lt : 0.0f;
                    const int row = row_n + r;
                    uint16_t* dst = a.out + (int64_t)(sp.start + row / G) * a.ldo +
                                    (int64_t)(hk * G + row % G) * D + 4 * u;
                    *reinterpret_cast<uint2*>(dst) = make_uint2(f32x2_to_bf16x2_rne(ot[0] * inv, ot[1] * inv),
                                                                f32x2_to_bf16x2_rne(ot[2] * inv, ot[3] * inv));
                } else {
                    const int64_t at = ((int64_t)item * splits + split) * tile_rows + 16 * n + r;
                    *reinterpret_cast<v4f*>(a.ws + at * D + 4 * u) = ot;
                    if (u == 0) part_stats(a, items, splits, tile_rows, D)[at] = make_float2(mt, lt);
                }
            }
            __syncthreads();             // before the next rows, or the next tile's fills
        }
    }
}

template <int D>
__global__ __launch_bounds__(256) void attn_few_join_kernel(AttnArgs a, int tile_rows, int splits, int chunk,
                                                            int items) {
    const int i = (int)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    const int item = i / tile_rows, r = i % tile_rows;
    if (item >= items) return;
    const int G = a.q_heads / a.kv_heads;
    const int pair = item % (a.B * a.kv_heads), hk = pair % a.kv_heads;
    const Span sp = sequence_span(a, pair / a.kv_heads, true);
    const int rows = sp.n * G, row0 = item / (a.B * a.kv_heads) * tile_rows;
    const int row = row0 + r;
    if (row >= rows) return;
    const int row_end = row0 + tile_rows < rows ? row0 + tile_rows : rows;
    const int parts = active_splits(visible(sp, row_end - 1, G), chunk, splits);
    if (parts == 1) return;
    join_row<D>(a, items, splits, tile_rows, item, r, parts,
                a.out + (int64_t)(sp.start + row / G) * a.ldo + (int64_t)(hk * G + row % G) * D);
}

template <int D, bool FP8, int NT>
void launch(const AttnArgs& a, const PagedPlan& p, hipStream_t s) {
    attn_few_kernel<D, FP8, NT><<<(unsigned)p.blocks, 256, 0, s>>>(a, p.tile_rows, p.row_tiles, p.splits, p.chunk);
    if (p.splits > 1)
        attn_few_join_kernel<D><<<(unsigned)((p.items * p.tile_rows + 3) / 4), 256, 0, s>>>(
            a, p.tile_rows, p.splits, p.chunk, (int)p.items);
}

template <int D, bool FP8>
void launch(const AttnArgs& a, const PagedPlan& p, hipStream_t s) {
    if (p.tile_rows <= 16) launch<D, FP8, 1>(a, p, s);
    else launch<D, FP8, 2>(a, p, s);
}

}  // namespace

hipError_t launch_attn_paged(const AttnArgs& a, hipStream_t s) {
    const PagedPlan p = paged_plan(a.T, a.B, a.max_q, a.max_kv, a.q_heads, a.cache);
    if (!p.few) return launch_attn_tiles(a, p, s);
    if (a.D == 128) {
        if (a.cache.fp8) launch<128, true>(a, p, s);
        else launch<128, false>(a, p, s);
    } else {
        if (a.cache.fp8) launch<64, true>(a, p, s);
        else launch<64, false>(a, p, s);
    }
    return hipGetLastError();
}

}  // namespace ptpc
