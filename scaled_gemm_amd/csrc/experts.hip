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
// What bounds it: for few tokens the launch and a chain of dependent steps, for
// many the 64-bit scores.
#include "block_device.h"

namespace ptpc {
namespace {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;

// Maximum and sum over the wave without LDS: neighbours, pairs of them, quads and
// halves of a row of 16 lanes by DPP, rows and halves of the wave by lane swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, __uint_as_float(dpp<kSwap1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<kSwap2>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp<kMirror>(__float_as_uint(v))));
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 |
                                          dpp<CTRL>((uint32_t)b));
}
template <class OP>
__device__ __forceinline__ double wave_reduce(double v, OP op) {
    v = op(v, dpp<kSwap1>(v));
    v = op(v, dpp<kSwap2>(v));
    v = op(v, dpp<kHalfMirror>(v));
    v = op(v, dpp<kMirror>(v));
    auto halves = [&](auto lo, auto hi) {
        const double x = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]);
        const double y = __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
        return op(x, y);
    };
    uint64_t b = __builtin_bit_cast(uint64_t, v);
    v = halves(__builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false),
               __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false));
    b = __builtin_bit_cast(uint64_t, v);
    return halves(
        __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false),
        __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false));
}
__device__ __forceinline__ double wave_max(double v) {
    return wave_reduce(v, [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ double wave_sum(double v) {
    return wave_reduce(v, [](double a, double b) { return a + b; });
}

// The lane whose best (the highest of its own; expert number p) is highest of all
// the lanes that have one; of equal ones that of the lowest p, then lane.
// Rounding keeps an order, so the maximum of the values rounded to 32 bits decides
// unless several lanes share it; only then are they compared in 64.
__device__ __forceinline__ int highest(double best, float best32, bool has, int p, int PER) {
    const float m = wave_max(has ? best32 : -INFINITY);
    uint64_t at = __ballot(has && best32 == m);
    if (at & (at - 1)) {
        const double d = wave_max(has ? best : -INFINITY);
        const bool tied = has && best == d;
        for (int i = 0; i < PER; ++i) {
            at = __ballot(tied && p == i);
            if (at) break;
        }
    }
    return at ? (int)__builtin_ctzll(at) : 0;
}

// Expert p * 64 + lane is number p of a lane.  lds: [2][PER * 64], scores and,
// where groups are compared, scores with bias.
template <int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* lds, int* count,
                                            int* ids_lds) {
    const int lane = threadIdx.x & 63;
    double choice[PER];
    float logit[PER], bias[PER];
    uint32_t alive = 0;
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
            alive |= 1u << p;
        }
        top = fmaxf(top, logit[p]);
    }
    // scores; both kinds need one exponential
    if (!a.sigmoid) top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const double x = a.sigmoid ? -(double)logit[p] : (double)logit[p] - (double)top;
        const double e = exp(x);
        choice[p] = a.sigmoid ? 1.0 / (1.0 + e) : top == -INFINITY ? 0.0 : e;
        sum += choice[p];
    }
    double over = 1.0;
    if (!a.sigmoid) {
        sum = wave_sum(sum);
        over = sum > 0.0 ? sum : 1.0;
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        if (!a.sigmoid) choice[p] /= over;
        lds[p * 64 + lane] = choice[p];
        choice[p] += (double)bias[p];
        if (!(choice[p] == choice[p])) choice[p] = -INFINITY;
    }
    if (a.top_groups < a.groups) {
        const int size = a.E / a.groups;
        double* const all = lds + PER * 64;
#pragma unroll
        for (int p = 0; p < PER; ++p) all[p * 64 + lane] = choice[p];
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        // `wide` lanes a group (a power of two), each over some of its experts
        const int wide = 64 >> (32 - __builtin_clz(a.groups - 1));
        const int group = lane / wide;
        double best = -INFINITY, second = -INFINITY;
        if (group < a.groups)
            for (int i = lane % wide; i < size; i += wide) {
                const double c = all[group * size + i];
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
        for (int i = 0; i < a.top_groups; ++i) {
            const bool open = lane % wide == 0 && group < a.groups && !((picked >> group) & 1);
            picked |= 1ull << (highest(best, (float)best, open, 0, 1) / wide);
        }
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int e = p * 64 + lane;
            if (e < a.E && !((picked >> (e / size)) & 1)) alive &= ~(1u << p);
        }
    }
    // the k best: each lane's own best, of which a round takes the highest
    int id = 0;
    for (int k = 0; k < a.K; ++k) {
        double best = -INFINITY;
        int p_best = PER;
#pragma unroll
        for (int p = PER - 1; p >= 0; --p) {
            const bool up = ((alive >> p) & 1) && choice[p] >= best;
            best = up ? choice[p] : best;
            p_best = up ? p : p_best;
        }
        const int l = highest(best, (float)best, p_best < PER, p_best, PER);
        const int p = __builtin_amdgcn_readlane(p_best, l);
        if (lane == l) alive &= ~(1u << p);
        if (lane == k) id = p * 64 + l;
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
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
// channels a thread, KU rows in flight.
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
