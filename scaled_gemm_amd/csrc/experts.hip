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

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d, 64));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// Expert p * 64 + lane is number p of a lane.
template <int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, double* choice_lds) {
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
        double best = -INFINITY, second = -INFINITY;
        if (lane < a.groups) {
            for (int i = 0; i < size; ++i) {
                const double c = choice_lds[lane * size + i];
                second = fmax(second, fmin(best, c));
                best = fmax(best, c);
            }
            if (a.group_top == 2 && size > 1) best += second;
            if (!(best == best)) best = -INFINITY;
        }
        uint64_t left = a.groups == 64 ? ~0ull : (1ull << a.groups) - 1, picked = 0;
        for (int i = 0; i < a.top_groups; ++i) {
            const double m = wave_max((left >> lane) & 1 ? best : -INFINITY);
            const uint64_t at = __ballot(best == m) & left;
            const uint64_t one = at & (0 - at);
            picked |= one;
            left &= ~one;
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
        double m = -INFINITY;
#pragma unroll
        for (int p = 0; p < PER; ++p) m = (alive >> p) & 1 ? fmax(m, choice[p]) : m;
        m = wave_max(m);
        int found = 0;
        double s = 0.0;
        bool open = true;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const uint64_t at = __ballot(((alive >> p) & 1) && choice[p] == m);
            if (open && at != 0) {
                open = false;
                const int l = (int)__builtin_ctzll(at);
                found = p * 64 + l;
                s = __shfl(score[p], l, 64);
                if (lane == l) alive &= ~(1u << p);
            }
        }
        sum += s;
        if (lane == k) {
            id = found;
            weight = s;
        }
    }
    if (lane < a.K) {
        double w = weight;
        if (a.renorm) w = sum > 0.0 ? weight / sum : 0.0;
        a.ids[t * a.K + lane] = id;
        a.weights[t * a.K + lane] = (float)(w * (double)a.scale);
    }
}

// Counts of the pairs first_pair .. first_pair + n - 1, by expert, into `count`.
__device__ __forceinline__ void count_pairs(const RouteArgs& a, int64_t pair0, int64_t n,
                                            int* count) {
    for (int e = threadIdx.x; e < a.local; e += kRouteThreads) count[e] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kRouteThreads) {
        const int e = a.ids[pair0 + i] - a.first;
        if (e >= 0 && e < a.local) atomicAdd(&count[e], 1);
    }
    __syncthreads();
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

// Places pairs pair0 .. pair0 + n - 1: thread e walks them for expert e from
// position base on.
__device__ __forceinline__ void place_pairs(const RouteArgs& a, int64_t pair0, int64_t n, int base,
                                            int* ids) {
    const int mine = threadIdx.x < (unsigned)a.local ? (int)threadIdx.x + a.first : -1;
    for (int64_t b = 0; b < n; b += kPairBatch) {
        const int m = (int)(n - b < kPairBatch ? n - b : kPairBatch);
        __syncthreads();
        for (int i = threadIdx.x; i < (m + 3) / 4 * 4; i += kRouteThreads) {
            const int e = i < m ? a.ids[pair0 + b + i] : -1;
            ids[i] = e;
            // experts that are not laid out
            if (i < m && (e < a.first || e >= a.first + a.local)) a.slots[pair0 + b + i] = -1;
        }
        __syncthreads();
        if (mine >= 0) {
            for (int i = 0; i < m; i += 4) {
                const int4 v = *reinterpret_cast<const int4*>(ids + i);
                const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (w[j] == mine) {
                        const int pair = (int)(pair0 + b) + i + j;
                        a.rows[base] = pair;
                        a.slots[pair] = base;
                        ++base;
                    }
            }
        }
    }
}

template <int PER>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a, RoutePlan plan) {
    __shared__ double choice[kRouteWaves][PER * 64];
    __shared__ int count[kMaxExperts];
    __shared__ int wave_sums[kRouteWaves];
    __shared__ __attribute__((aligned(16))) int ids[kPairBatch];
    const int wave = uniform(threadIdx.x >> 6);
    const int64_t t0 = blockIdx.x * plan.chunk;
    const int64_t t1 = t0 + plan.chunk < a.T ? t0 + plan.chunk : a.T;
    for (int64_t t = t0 + wave; t < t1; t += kRouteWaves) route_token<PER>(a, t, choice[wave]);
    __syncthreads();                       // the workgroup's ids are in memory
    const int64_t pair0 = t0 * a.K, n = (t1 - t0) * a.K;
    count_pairs(a, pair0, n, count);
    if (plan.chunks > 1) {
        for (int e = threadIdx.x; e < a.local; e += kRouteThreads)
            a.ws[blockIdx.x * (int64_t)a.local + e] = count[e];
        return;
    }
    const int total = scan_counts(count, a.local, wave_sums);
    if ((int)threadIdx.x < a.local) a.offsets[threadIdx.x] = count[threadIdx.x];
    if (threadIdx.x == 0) a.offsets[a.local] = total;
    for (int64_t i = total + (int)threadIdx.x; i < a.T * a.K; i += kRouteThreads) a.rows[i] = -1;
    place_pairs(a, pair0, n, threadIdx.x < (unsigned)a.local ? count[threadIdx.x] : 0, ids);
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
    const int base = threadIdx.x < (unsigned)a.local ? count[threadIdx.x] + before[threadIdx.x] : 0;
    place_pairs(a, t0 * a.K, (t1 - t0) * a.K, base, ids);
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
