// Routing of tokens to experts, the layout of their pairs, and the weighted
// sum of the experts' rows (gfx950).
//
// route_kernel: a wave scores one token at a time, E / 64 experts a lane, in 64
// bits: near-equal scores then fall the same way in every implementation of
// the formula, and no two experts swap places by a rounding.  The k best come
// out in k rounds of a maximum over the wave; of equal scores the lowest index.
//
// The layout is a counting sort that keeps the pairs' order: a workgroup counts the
// pairs of its chunk of tokens, and a pair's row is its expert's offset, the counts
// of earlier chunks and waves, and the equal lanes below it, so that nothing depends
// on the order in which threads run.  Up to 16 tokens one workgroup does all of it;
// otherwise each workgroup leaves its counts in the workspace and a second kernel
// sums them and places the pairs.
//
// What bounds it: for few tokens the launch and a chain of dependent steps (one token
// of 8 experts 4.3 us), E / 64 scores a lane in 64 bits (one of 256 experts in 8 groups
// 7.7), and a CU that all of a step's tokens share (16 of them 11.2, without groups
// 9.8, with k = 1 instead of 8 9.1).  For many, the scores, then every workgroup's sum
// of all chunks' counts: 8192 of 128 experts (k = 8) 16.1 to 17.4 us, 11.0 of them the
// scores and choices, 6.4 the sums and the layout, of 512 experts 49; the logits and
// pairs alone would be read and written in 2 us.  256 chunks at most: with 512, a token a wave, the sums
// read four times as much (24.2 us).
#include "block_device.h"

namespace ptpc {
namespace {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;

// Reductions over the wave without LDS: neighbours, pairs of them, quads and halves
// of a row of 16 lanes by DPP; then rows (the result reaches the last lane).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t old = 0) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_u32(v, dpp<kSwap1>(v));
    v = max_u32(v, dpp<kSwap2>(v));
    v = max_u32(v, dpp<kHalfMirror>(v));
    v = max_u32(v, dpp<kMirror>(v));
    v = max_u32(v, dpp<kRowBcast15>(v));
    v = max_u32(v, dpp<kRowBcast31>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 |
                                          dpp<CTRL>((uint32_t)b));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(
        double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32 |
                    (uint32_t)__builtin_amdgcn_readlane((int)b, lane));
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp64<kSwap1>(v);
    v += dpp64<kSwap2>(v);
    v += dpp64<kHalfMirror>(v);
    v += dpp64<kMirror>(v);
    return read_lane(v, 0) + read_lane(v, 16) + read_lane(v, 32) + read_lane(v, 48);
}
__device__ __forceinline__ double wave_max(double v) {
    v = fmax(v, dpp64<kSwap1>(v));
    v = fmax(v, dpp64<kSwap2>(v));
    v = fmax(v, dpp64<kHalfMirror>(v));
    v = fmax(v, dpp64<kMirror>(v));
    return fmax(fmax(read_lane(v, 0), read_lane(v, 16)), fmax(read_lane(v, 32), read_lane(v, 48)));
}

// A whole number that orders as the value rounded to 32 bits does, at least 1;
// 0: not there.  Rounding keeps an order, so the largest key decides unless several
// have it; only those are compared in 64 bits.
__device__ __forceinline__ uint32_t key_of(double v) {
    const uint32_t b = __float_as_uint((float)v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The lane whose first key is highest; of several the one with the highest value, of
// equal values with the lowest expert.
template <class VALUE>
__device__ __forceinline__ int highest(uint32_t key, int expert, VALUE value) {
    const uint32_t m = wave_max(key);
    uint64_t at = __ballot(key == m);
    if (at & (at - 1)) {
        const bool mine = key == m;
        const double v = mine ? value(expert) : -INFINITY, top = wave_max(v);
        const uint32_t first = wave_max(mine && v == top ? ~(uint32_t)expert : 0u);
        at = __ballot(mine && v == top && ~(uint32_t)expert == first);
    }
    return (int)__builtin_ctzll(at);
}

// 1 / x for x from 1 to infinity: two Newton steps on the hardware's estimate,
// within an ulp.
__device__ __forceinline__ double reciprocal(double x) {
    double r = __builtin_amdgcn_rcp(x);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    return x == INFINITY ? 0.0 : r;
}

// Expert p * 64 + lane is number p of a lane.  lds: [2][PER * 64], scores, and scores
// with bias.
template <int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* lds, int* count,
                                            int* ids_lds) {
    const int lane = threadIdx.x & 63;
    double* const with_bias = lds + PER * 64;
    double value[PER];
    uint32_t key[PER];
    float logit[PER], bias[PER];
    float top = -INFINITY;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int e = p * 64 + lane;
        logit[p] = -INFINITY;
        bias[p] = 0.0f;
        if (e < a.E) {
            const float l =
                a.bf16 ? __uint_as_float(
                             (uint32_t) static_cast<const uint16_t*>(a.logits)[t * a.ldl + e] << 16)
                       : static_cast<const float*>(a.logits)[t * a.ldl + e];
            if (a.bias != nullptr) bias[p] = a.bias[e];
            logit[p] = l != l ? -INFINITY : fminf(l, 0x1.fffffep127f);
        }
        top = fmaxf(top, logit[p]);
    }
    // scores; both kinds need one exponential
    if (!a.sigmoid) {
        const uint32_t k = wave_max(key_of(top));
        top = __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
    }
    double sum = 0.0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const double x = a.sigmoid ? -(double)logit[p] : (double)logit[p] - (double)top;
        const double e = exp(x);
        value[p] = a.sigmoid ? reciprocal(1.0 + e) : top == -INFINITY ? 0.0 : e;
        sum += value[p];
    }
    double over = 1.0;
    if (!a.sigmoid) {
        sum = wave_sum(sum);
        over = sum > 0.0 ? 1.0 / sum : 1.0;
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        value[p] *= over;
        lds[p * 64 + lane] = value[p];
        value[p] += (double)bias[p];
        if (!(value[p] == value[p])) value[p] = -INFINITY;
        with_bias[p * 64 + lane] = value[p];
        key[p] = p * 64 + lane < a.E ? key_of(value[p]) : 0;
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if (a.top_groups < a.groups) {
        const int size = a.E / a.groups;
        // `wide` lanes a group (a power of two), each over some of its experts
        const int wide = 64 >> (32 - __builtin_clz(a.groups - 1));
        const int group = lane / wide;
        double best = -INFINITY, second = -INFINITY;
        if (group < a.groups)
            for (int i = lane % wide; i < size; i += wide) {
                const double c = with_bias[group * size + i];
                second = fmax(second, fmin(best, c));
                best = fmax(best, c);
            }
        for (int d = 1; d < wide; d <<= 1) {
            const double b = __shfl_xor(best, d, 64), c = __shfl_xor(second, d, 64);
            second = fmax(fmax(second, c), fmin(best, b));
            best = fmax(best, b);
        }
        if (a.group_top == 2 && size > 1) best += second;
        if (!(best == best)) best = -INFINITY;
        uint64_t picked = 0;
        uint32_t open = lane % wide == 0 && group < a.groups ? key_of(best) : 0;
        for (int i = 0; i < a.top_groups; ++i) {
            const int l = highest(open, group, [&](int) { return best; });
            picked |= 1ull << (l / wide);
            if (lane == l) open = 0;
        }
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int e = p * 64 + lane;
            if (e < a.E && !((picked >> (e / size)) & 1)) key[p] = 0;
        }
    }
    // Each lane's experts in falling order (stable: the lowest index first), then k
    // times the highest of the lanes' first ones.
    int order[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) order[p] = p * 64 + lane;
#pragma unroll
    for (int n = PER - 1; n > 0; --n)
#pragma unroll
        for (int p = 0; p < n; ++p) {
            bool swap = key[p + 1] > key[p];
            if (key[p + 1] == key[p]) swap = with_bias[order[p + 1]] > with_bias[order[p]];
            const uint32_t k = key[p];
            const int o = order[p];
            key[p] = swap ? key[p + 1] : k;
            key[p + 1] = swap ? k : key[p + 1];
            order[p] = swap ? order[p + 1] : o;
            order[p + 1] = swap ? o : order[p + 1];
        }
    int id = 0;
    for (int k = 0; k < a.K; ++k) {
        const int l = highest(key[0], order[0], [&](int e) { return with_bias[e]; });
        const int e = __builtin_amdgcn_readlane(order[0], l);
        if (lane == k) id = e;
        const bool won = lane == l;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            key[p] = won ? (p + 1 < PER ? key[p + 1 < PER ? p + 1 : p] : 0) : key[p];
            if (p + 1 < PER) order[p] = won ? order[p + 1 < PER ? p + 1 : p] : order[p];
        }
    }
    double w = lane < a.K ? lds[id] : 0.0;
    if (a.renorm) {
        const double all = wave_sum(w);
        w = all > 0.0 ? w / all : 0.0;
    }
    if (lane < a.K) {
        a.ids[t * a.K + lane] = id;
        a.weights[t * a.K + lane] = (float)(w * (double)a.scale);
        if (ids_lds != nullptr) ids_lds[lane] = id;
        const int e = id - a.first;
        if (e >= 0 && e < a.local) atomicAdd(&count[e], 1);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
}

// Exclusive sums of count[0 .. local-1] (in place); the total.
__device__ __forceinline__ int scan_counts(int* count, int local, int* wave_sums) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int mine = tid < local ? count[tid] : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d, 64);
        if (lane >= d) sum += o;
    }
    if (lane == 63) wave_sums[wave] = sum;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
        before += w < wave ? wave_sums[w] : 0;
        total += wave_sums[w];
    }
    if (tid < local) count[tid] = before + sum - mine;
    __syncthreads();
    return total;
}

// Places pairs pair0 .. pair0 + n - 1, a thread each: behind base[e], those of
// expert e in earlier waves, and the lanes below in its own wave, which it finds by
// comparing the expert's bits over the wave.  ids: the pairs' experts, in LDS or in
// memory; base (LDS) moves on; held: [kRouteWaves][local] in LDS.
__device__ __forceinline__ void place_pairs(const RouteArgs& a, int64_t pair0, int64_t n,
                                            const int* ids, int* base, uint16_t* held) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bits = a.local > 1 ? 32 - __builtin_clz(a.local - 1) : 0;
    for (int64_t b = 0; b < n; b += kRouteThreads) {
        const int64_t i = b + threadIdx.x;
        const int waves = (int)(n - b < kRouteThreads ? (n - b + 63) / 64 : kRouteWaves);
        if (wave < waves)
            for (int e = lane; e < a.local; e += 64) held[wave * a.local + e] = 0;
        const int e = i < n ? ids[i] - a.first : -1;
        const bool mine = e >= 0 && e < a.local;
        uint64_t same = __ballot(mine);
        for (int k = 0; k < bits; ++k) {
            const uint64_t with = __ballot((e >> k) & 1);
            same &= (e >> k) & 1 ? with : ~with;
        }
        const int below = (int)__builtin_popcountll(same & ((1ull << lane) - 1));
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (mine && below == 0) held[wave * a.local + e] = (uint16_t)__builtin_popcountll(same);
        __syncthreads();
        if (mine) {
            int at = base[e] + below;
            for (int w = 0; w < wave; ++w) at += held[w * a.local + e];
            a.rows[at] = (int)(pair0 + i);
            a.slots[pair0 + i] = at;
        } else if (i < n) {
            a.slots[pair0 + i] = -1;                     // experts that are not laid out
        }
        if (b + kRouteThreads < n) {
            __syncthreads();
            if ((int)threadIdx.x < a.local)
                for (int w = 0; w < waves; ++w) base[threadIdx.x] += held[w * a.local + threadIdx.x];
            __syncthreads();
        }
    }
}

template <int PER>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, RoutePlan plan) {
    __shared__ double scores[kRouteWaves][2 * PER * 64];
    __shared__ int count[kMaxExperts];
    __shared__ int wave_sums[kRouteWaves];
    __shared__ int ids[kRouteWaves * 64];
    const int wave = uniform(threadIdx.x >> 6);
    const int64_t t0 = blockIdx.x * plan.chunk;
    const int64_t t1 = t0 + plan.chunk < a.T ? t0 + plan.chunk : a.T;
    for (int e = threadIdx.x; e < a.local; e += kRouteThreads) count[e] = 0;
    const int n = (int)(t1 - t0) * a.K;
    __syncthreads();
    for (int64_t t = t0 + wave; t < t1; t += kRouteWaves)
        route_token<PER>(a, t, scores[wave], count,
                         plan.chunks == 1 ? ids + (t - t0) * a.K : nullptr);
    __syncthreads();
    if (plan.chunks > 1) {
        for (int e = threadIdx.x; e < a.local; e += kRouteThreads)
            a.ws[blockIdx.x * (int64_t)a.local + e] = count[e];
        return;
    }
    const int total = scan_counts(count, a.local, wave_sums);
    if ((int)threadIdx.x < a.local) a.offsets[threadIdx.x] = count[threadIdx.x];
    if (threadIdx.x == 0) a.offsets[a.local] = total;
    for (int i = total + (int)threadIdx.x; i < n; i += kRouteThreads) a.rows[i] = -1;
    place_pairs(a, 0, n, ids, count, reinterpret_cast<uint16_t*>(&scores[0][0]));
}

__global__ __launch_bounds__(kRouteThreads) void place_kernel(RouteArgs a, RoutePlan plan) {
    __shared__ int count[kMaxExperts], before[kMaxExperts];
    __shared__ int wave_sums[kRouteWaves];
    __shared__ uint16_t held[kRouteWaves * kMaxExperts];
    const int me = (int)blockIdx.x;
    for (int e = threadIdx.x; e < a.local; e += kRouteThreads) count[e] = before[e] = 0;
    __syncthreads();
    // every chunk's counts: `lanes` threads an expert, each over some of the chunks
    const int lanes = kRouteThreads / a.local < 1 ? 1 : kRouteThreads / a.local;
    const int e = (int)threadIdx.x % a.local, part = (int)threadIdx.x / a.local;
    if (part < lanes) {
        int all = 0, lower = 0;
#pragma unroll 8
        for (int c = part; c < plan.chunks; c += lanes) {
            const int n = a.ws[c * (int64_t)a.local + e];
            all += n;
            lower += c < me ? n : 0;
        }
        atomicAdd(&count[e], all);
        atomicAdd(&before[e], lower);
    }
    __syncthreads();
    const int total = scan_counts(count, a.local, wave_sums);
    if (me == 0) {
        if ((int)threadIdx.x < a.local) a.offsets[threadIdx.x] = count[threadIdx.x];
        if (threadIdx.x == 0) a.offsets[a.local] = total;
    }
    const int64_t t0 = me * plan.chunk;
    const int64_t t1 = t0 + plan.chunk < a.T ? t0 + plan.chunk : a.T;
    // rows past the last pair, each workgroup a share
    for (int64_t i = total + me * (int64_t)kRouteThreads + threadIdx.x; i < a.T * a.K;
         i += plan.chunks * kRouteThreads)
        a.rows[i] = -1;
    if ((int)threadIdx.x < a.local) count[threadIdx.x] += before[threadIdx.x];
    __syncthreads();
    const int64_t pair0 = t0 * a.K;
    place_pairs(a, pair0, (t1 - t0) * a.K, a.ids + pair0, count, held);
}

// out[t] = sum over k of weights[t,k] * y[slots[t,k]], in that order; 8
// channels a thread, KU rows in flight.  A stream: 8191 tokens of 8 x 4096 in 119 to
// 121 us, 5.0 TB/s; 16 tokens in 4.0, the launch and two dependent loads.
template <int KU>
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ y, int64_t ldy,
                                                      int64_t R, const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, int64_t T,
                                                      int K, int vecs, uint16_t* __restrict__ out,
                                                      int64_t ldo) {
    const int64_t n = T * vecs;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += gridDim.x * (int64_t)256) {
        const int64_t t = i / vecs;
        const int c = (int)(i - t * vecs) * 8;
        float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int k0 = 0; k0 < K; k0 += KU) {
            uint4 v[KU];
            float w[KU];
            bool ok[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const bool in = k0 + j < K;
                const int64_t s = in ? slots[t * K + k0 + j] : -1;
                ok[j] = s >= 0 && s < R;
                w[j] = in ? weights[t * K + k0 + j] : 0.0f;
                v[j] = ok[j] ? *reinterpret_cast<const uint4*>(y + s * ldy + c)
                             : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                if (!ok[j]) continue;
                acc[0] = __builtin_fmaf(w[j], bf16lo_to_f32(v[j].x), acc[0]);
                acc[1] = __builtin_fmaf(w[j], bf16hi_to_f32(v[j].x), acc[1]);
                acc[2] = __builtin_fmaf(w[j], bf16lo_to_f32(v[j].y), acc[2]);
                acc[3] = __builtin_fmaf(w[j], bf16hi_to_f32(v[j].y), acc[3]);
                acc[4] = __builtin_fmaf(w[j], bf16lo_to_f32(v[j].z), acc[4]);
                acc[5] = __builtin_fmaf(w[j], bf16hi_to_f32(v[j].z), acc[5]);
                acc[6] = __builtin_fmaf(w[j], bf16lo_to_f32(v[j].w), acc[6]);
                acc[7] = __builtin_fmaf(w[j], bf16hi_to_f32(v[j].w), acc[7]);
            }
        }
        *reinterpret_cast<uint4*>(out + t * ldo + c) =
            make_uint4(f32x2_to_bf16x2_rne(acc[0], acc[1]), f32x2_to_bf16x2_rne(acc[2], acc[3]),
                       f32x2_to_bf16x2_rne(acc[4], acc[5]), f32x2_to_bf16x2_rne(acc[6], acc[7]));
    }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    const RoutePlan p = route_plan(a.T);
    const dim3 grid((unsigned)p.chunks);
    if (a.E <= 64) route_kernel<1><<<grid, kRouteThreads, 0, s>>>(a, p);
    else if (a.E <= 128) route_kernel<2><<<grid, kRouteThreads, 0, s>>>(a, p);
    else if (a.E <= 256) route_kernel<4><<<grid, kRouteThreads, 0, s>>>(a, p);
    else route_kernel<8><<<grid, kRouteThreads, 0, s>>>(a, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.chunks == 1) return e;
    place_kernel<<<grid, kRouteThreads, 0, s>>>(a, p);
    return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* y, int64_t ldy, int64_t R, const int32_t* slots,
                          const float* weights, int64_t T, int32_t K, int64_t C, uint16_t* out,
                          int64_t ldo, hipStream_t s) {
    const int64_t blocks = (T * (C / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22)));
    const int vecs = (int)(C / 8);
    if (K <= 2) combine_kernel<2><<<grid, 256, 0, s>>>(y, ldy, R, slots, weights, T, K, vecs, out, ldo);
    else if (K <= 4) combine_kernel<4><<<grid, 256, 0, s>>>(y, ldy, R, slots, weights, T, K, vecs, out, ldo);
    else combine_kernel<8><<<grid, 256, 0, s>>>(y, ldy, R, slots, weights, T, K, vecs, out, ldo);
    return hipGetLastError();
}

}  // namespace ptpc
