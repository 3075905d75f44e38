// Routing of tokens to experts, the layout of their pairs, and the weighted
// sum of the experts' rows (gfx950).
//
// route_kernel: a wave scores one token at a time, E / 64 experts a lane, in 64
// bits: near-equal scores then fall the same way in every implementation of
// the formula, and no two experts swap places by a rounding.  The k best come
// out in k rounds of a maximum over the wave; of equal scores the lowest index.
//
// The layout is a counting sort that keeps the pairs' order: a workgroup holds
// the pairs of its chunk of tokens in LDS and one thread per expert walks
// them, so nothing depends on the order in which threads run.  Up to 64 tokens
// one workgroup does all of it; otherwise each workgroup leaves its counts in
// the workspace and a second kernel sums them and places the pairs.
//
// What bounds it: for few tokens the launch and a chain of dependent steps, for
// many the 64-bit scores.
#include "block_device.h"

namespace ptpc {
namespace {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
// Pairs that a workgroup holds in LDS at a time.
constexpr int kPairBatch = 4096;

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

// The highest of the values that are alive, and the lanes (of number p) that have
// it.  Rounding keeps an order, so the maximum of the values rounded to 32 bits
// decides unless several share it; only then is it taken in 64.
template <int PER>
__device__ __forceinline__ void highest(const double (&v)[PER], uint32_t alive, int& p_found,
                                        int& lane_found) {
    float m = -INFINITY;
#pragma unroll
    for (int p = 0; p < PER; ++p) m = (alive >> p) & 1 ? fmaxf(m, (float)v[p]) : m;
    m = wave_max(m);
    uint64_t at[PER];
    int many = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        at[p] = __ballot(((alive >> p) & 1) && (float)v[p] == m);
        many += (int)__builtin_popcountll(at[p]);
    }
    if (many > 1) {
        double d = -INFINITY;
#pragma unroll
        for (int p = 0; p < PER; ++p) d = (alive >> p) & 1 ? fmax(d, v[p]) : d;
        d = wave_max(d);
#pragma unroll
        for (int p = 0; p < PER; ++p) at[p] = __ballot(((alive >> p) & 1) && v[p] == d);
    }
    p_found = 0;
    lane_found = 0;
    bool open = true;
#pragma unroll
    for (int p = 0; p < PER; ++p)
        if (open && at[p] != 0) {
            open = false;
            p_found = p;
            lane_found = (int)__builtin_ctzll(at[p]);
        }
}

// Expert p * 64 + lane is number p of a lane.
template <int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* choice_lds,
                                            int* count, int* ids_lds) {
    const int lane = threadIdx.x & 63;
    double score[PER], choice[PER];
    uint32_t alive = 0;
    double top = -INFINITY;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int e = p * 64 + lane;
        float l = -INFINITY;
        if (e < a.E) {
            l = a.bf16 ? __uint_as_float(
                             (uint32_t) static_cast<const uint16_t*>(a.logits)[t * a.ldl + e] << 16)
                       : static_cast<const float*>(a.logits)[t * a.ldl + e];
            l = l != l ? -INFINITY : fminf(l, 0x1.fffffep127f);
            alive |= 1u << p;
        }
        score[p] = l;
        top = fmax(top, score[p]);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int p = 0; p < PER; ++p) score[p] = 1.0 / (1.0 + exp(-score[p]));
    } else {
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            score[p] = top == -INFINITY ? 0.0 : exp(score[p] - top);
            sum += score[p];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int p = 0; p < PER; ++p) score[p] = sum > 0.0 ? score[p] / sum : 0.0;
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int e = p * 64 + lane;
        choice[p] = score[p] + (a.bias != nullptr && e < a.E ? (double)a.bias[e] : 0.0);
        if (!(choice[p] == choice[p])) choice[p] = -INFINITY;
    }
    if (a.top_groups < a.groups) {
        const int size = a.E / a.groups;
#pragma unroll
        for (int p = 0; p < PER; ++p)
            if (p * 64 + lane < a.E) choice_lds[p * 64 + lane] = choice[p];
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        // `wide` lanes a group (a power of two), each over some of its experts
        const int wide = 64 >> (a.groups > 1 ? 32 - __builtin_clz(a.groups - 1) : 0);
        const int group = lane / wide;
        double best[1] = {-INFINITY}, second = -INFINITY;
        if (group < a.groups)
            for (int i = lane % wide; i < size; i += wide) {
                const double c = choice_lds[group * size + i];
                second = fmax(second, fmin(best[0], c));
                best[0] = fmax(best[0], c);
            }
        for (int d = 1; d < wide; d <<= 1) {
            const double b = __shfl_xor(best[0], d, 64), c = __shfl_xor(second, d, 64);
            second = fmax(fmax(second, c), fmin(best[0], b));
            best[0] = fmax(best[0], b);
        }
        if (a.group_top == 2 && size > 1) best[0] += second;
        if (!(best[0] == best[0])) best[0] = -INFINITY;
        uint64_t picked = 0;
        for (int i = 0; i < a.top_groups; ++i) {
            int p, l;
            highest<1>(best, lane % wide == 0 && group < a.groups && !((picked >> group) & 1), p, l);
            picked |= 1ull << (l / wide);
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int e = p * 64 + lane;
            if (e < a.E && !((picked >> (e / size)) & 1)) alive &= ~(1u << p);
        }
    }
    // the k best
    int id = 0;
    double weight = 0.0, sum = 0.0;
    for (int k = 0; k < a.K; ++k) {
        int p, l;
        highest<PER>(choice, alive, p, l);
        double mine = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mine = i == p ? score[i] : mine;
        const uint64_t bits = __builtin_bit_cast(uint64_t, mine);
        const double s = __builtin_bit_cast(
            double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(bits >> 32), l) << 32 |
                        (uint32_t)__builtin_amdgcn_readlane((int)bits, l));
        if (lane == l) alive &= ~(1u << p);
        sum += s;
        if (lane == k) {
            id = p * 64 + l;
            weight = s;
        }
    }
    if (lane < a.K) {
        double w = weight;
        if (a.renorm) w = sum > 0.0 ? weight / sum : 0.0;
        a.ids[t * a.K + lane] = id;
        a.weights[t * a.K + lane] = (float)(w * (double)a.scale);
        if (ids_lds != nullptr) ids_lds[lane] = id;
        const int e = id - a.first;
        if (e >= 0 && e < a.local) atomicAdd(&count[e], 1);
    }
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

// Places m pairs from pair0 on, whose experts are in LDS (padded with -1 to a
// multiple of 4): thread e walks them for expert e from position `base` on.
__device__ __forceinline__ int place_pairs(const RouteArgs& a, int64_t pair0, int m, int base,
                                           const int* ids) {
    for (int i = threadIdx.x; i < m; i += kRouteThreads) {
        const int e = ids[i];                            // experts that are not laid out
        if (e < a.first || e >= a.first + a.local) a.slots[pair0 + i] = -1;
    }
    if (threadIdx.x >= (unsigned)a.local) return base;
    const int mine = (int)threadIdx.x + a.first;
#pragma unroll 4
    for (int i = 0; i < m; i += 4) {
        const int4 v = *reinterpret_cast<const int4*>(ids + i);
        const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (w[j] == mine) {
                const int pair = (int)pair0 + i + j;
                a.rows[base] = pair;
                a.slots[pair] = base;
                ++base;
            }
    }
    return base;
}

template <int PER>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, RoutePlan plan) {
    __shared__ double choice[kRouteWaves][PER * 64];
    __shared__ int count[kMaxExperts];
    __shared__ int wave_sums[kRouteWaves];
    __shared__ __attribute__((aligned(16))) int ids[kPairBatch + 4];
    const int wave = uniform(threadIdx.x >> 6);
    const int64_t t0 = blockIdx.x * plan.chunk;
    const int64_t t1 = t0 + plan.chunk < a.T ? t0 + plan.chunk : a.T;
    for (int e = threadIdx.x; e < a.local; e += kRouteThreads) count[e] = 0;
    const int n = (int)(t1 - t0) * a.K;
    if (plan.chunks == 1 && threadIdx.x < 3) ids[n + threadIdx.x] = -1;
    __syncthreads();
    for (int64_t t = t0 + wave; t < t1; t += kRouteWaves)
        route_token<PER>(a, t, choice[wave], count, plan.chunks == 1 ? ids + (t - t0) * a.K : nullptr);
    __syncthreads();
    if (plan.chunks > 1) {
        for (int e = threadIdx.x; e < a.local; e += kRouteThreads)
            a.ws[blockIdx.x * (int64_t)a.local + e] = count[e];
        return;
    }
    const int total = scan_counts(count, a.local, wave_sums);
    const int base = threadIdx.x < (unsigned)a.local ? count[threadIdx.x] : 0;
    if ((int)threadIdx.x < a.local) a.offsets[threadIdx.x] = base;
    if (threadIdx.x == 0) a.offsets[a.local] = total;
    for (int i = total + (int)threadIdx.x; i < n; i += kRouteThreads) a.rows[i] = -1;
    place_pairs(a, 0, n, base, ids);
}

__global__ __launch_bounds__(kRouteThreads) void place_kernel(RouteArgs a, RoutePlan plan) {
    __shared__ int count[kMaxExperts], before[kMaxExperts];
    __shared__ int wave_sums[kRouteWaves];
    __shared__ __attribute__((aligned(16))) int ids[kPairBatch];
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
    int base = threadIdx.x < (unsigned)a.local ? count[threadIdx.x] + before[threadIdx.x] : 0;
    const int64_t pair0 = t0 * a.K, n = (t1 - t0) * a.K;
    for (int64_t b = 0; b < n; b += kPairBatch) {
        const int m = (int)(n - b < kPairBatch ? n - b : kPairBatch);
        __syncthreads();
        for (int i = threadIdx.x; i < (m + 3) / 4 * 4; i += kRouteThreads)
            ids[i] = i < m ? a.ids[pair0 + b + i] : -1;
        __syncthreads();
        base = place_pairs(a, pair0 + b, m, base, ids);
    }
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
