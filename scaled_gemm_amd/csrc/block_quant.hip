// Block-scaled FP8 quantization (gfx950): activations with one scale per token
// and 128 channels, weights with one per 128 x 128.
//
// Scale = amax / 448 (1 for an all-zero block); code = OCP E4M3(x / scale),
// round to nearest even.  All are streams: each element is read once.
//
// What bounds it: HBM from a few thousand rows on.  8192 x 8192 are quantized in 36.4
// us (5.6 TB/s), gated in 67.0 (5.0 TB/s; the exponential, reciprocal and quotient of
// an element nearly fill the vector units then), 24577 x 1408 gated in 32.9 to 34.6;
// 32 x 4096 in 2.6, the launch and one load.
#include "block_device.h"

namespace ptpc {
namespace {

typedef float f8[8];

__device__ __forceinline__ void unpack(uint4 w, f8& x) {
    x[0] = bf16lo_to_f32(w.x); x[1] = bf16hi_to_f32(w.x);
    x[2] = bf16lo_to_f32(w.y); x[3] = bf16hi_to_f32(w.y);
    x[4] = bf16lo_to_f32(w.z); x[5] = bf16hi_to_f32(w.z);
    x[6] = bf16lo_to_f32(w.w); x[7] = bf16hi_to_f32(w.w);
}

// silu(g) * u.  exp(-g) is 2^t with t = -g log2(e) in two parts, the second (what
// the product's rounding lost) as 1 + part * ln 2: each step is within an fp32 ulp or
// so, where 2^t alone would be off by |t| of them.  Beyond +-126 nothing changes:
// exp(-g) is lost beside 1, or overflows and gives a zero (gates below -88.72).
// The reciprocal is taken of a quarter of 1 + exp(-g), because the instruction gives
// zero where its result is no normal number: from 2^126 on, gates of -87.4 to -88.7.
// A quarter of g makes up for it, exactly: bf16 goes down to 2^-133, fp32 to 2^-149.
__device__ __forceinline__ float gated(float g, float u) {
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float x = -__builtin_amdgcn_fmed3f(g, -126.0f, 126.0f);
    const float t = x * kLog2e;
    const float low = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(low, kLn2, 1.0f);
    return 0.25f * g * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.25f, 0.25f)) * u;
}

// Sixteen lanes own one row's block of 128 channels, 8 channels (one 16-byte
// load) each; a wave takes 4 * IT rows of one block, so that the scales, which
// lie token after token, leave as one store.
template <bool GATE, int IT>
__global__ __launch_bounds__(256) void quant_act_block_kernel(
    const uint16_t* __restrict__ x, int64_t T, int64_t C, int64_t ldx,
    const int32_t* __restrict__ count, uint8_t* __restrict__ qx, int64_t ldq,
    float* __restrict__ sx, int64_t lds, int kb, int64_t items) {
    const int lane = threadIdx.x & 63, l16 = lane & 15;
    const int wave = uniform(threadIdx.x >> 6);
    if (count != nullptr) {
        const int64_t n = *count;
        T = n < T ? n : T;
    }
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t tile = item / kb;
        const int b = (int)(item - tile * kb);
        const int64_t t0 = (tile * 4 + wave) * (4 * IT);
        if (t0 >= T) continue;
        const int64_t k = b * 128 + l16 * 8;
        uint4 v[IT], u[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int64_t t = t0 + 4 * i + (lane >> 4);
            const bool in = t < T && k < C;
            const uint16_t* row = x + (in ? t * ldx + k : 0);
            v[i] = *reinterpret_cast<const uint4*>(row);
            if (GATE) u[i] = *reinterpret_cast<const uint4*>(row + (in ? C : 0));
            if (!in) v[i] = u[i] = make_uint4(0, 0, 0, 0);
        }
        float mine = 0.0f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int64_t t = t0 + 4 * i + (lane >> 4);
            const bool in = t < T && k < C;
            float scale;
            uint2 code;
            if (GATE) {
                f8 h, w;
                unpack(v[i], h);
                unpack(u[i], w);
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[e] = gated(h[e], w[e]);
                    m = fmaxf(m, fabsf(h[e]));
                }
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
                // Products go down to the smallest fp32 numbers, where m / 448 keeps few bits
                // or none; from 2^-144 on the largest quotient still rounds to 448.
                scale = fmaxf(scale_from_amax(m), 0x1p-144f);
                // (the quotient by Markstein's correction, correctly rounded for any fp32
                // numerator: see divide; a few codes below the smallest aside, which are 0)
                const Divisor dv = make_divisor(scale);
                uint32_t lo = 0, hi = 0;
                lo = cvt_e4m3x2<false>(divide(h[0], dv), divide(h[1], dv), lo);
                lo = cvt_e4m3x2<true>(divide(h[2], dv), divide(h[3], dv), lo);
                hi = cvt_e4m3x2<false>(divide(h[4], dv), divide(h[5], dv), hi);
                hi = cvt_e4m3x2<true>(divide(h[6], dv), divide(h[7], dv), hi);
                code = make_uint2(lo, hi);
            } else {
                us2 m = max2(max2(abs_bits2(v[i].x), abs_bits2(v[i].y)),
                             max2(abs_bits2(v[i].z), abs_bits2(v[i].w)));
                const uint32_t top = group_max_u32<16>(hmax(m));
                scale = scale_from_amax(__uint_as_float(top << 16));
                code = quantize8(v[i], make_divisor(scale));
            }
            if (in) *reinterpret_cast<uint2*>(qx + t * ldq + k) = code;
            if (l16 == i) mine = scale;
        }
        // lane 16 g + i of the wave holds row 4 i + g
        const int64_t t = t0 + 4 * l16 + (lane >> 4);
        if (l16 < IT && t < T) sx[b * lds + t] = mine;
    }
}

// 128 x 128 elements of a weight by one workgroup: codes of column o in LDS (pitch
// 144), 16 K bytes after another with their order changed by the column's slab (so that
// lanes 8 or 16 columns apart write to other banks), leaving as the 1 KB blocks of the
// packed weight.  A thread holds several neighbours of K and turns them 4 x 4 bytes at
// a time, so that they are written 4 or 8 together.  8192 x 10240 is quantized in 41 us
// (byte by byte: 84), packed in 27 (43) whichever of its axes lies together, larger
// ones at 4.3 to 5.8 TB/s.
constexpr int kPitch = 144;
__device__ __forceinline__ uint8_t* tile_at_chunk(uint8_t* tile, int o, int chunk) {
    return tile + o * kPitch + (chunk ^ ((o >> 4) & 7)) * 16;
}
// Bytes [k][o] of w as [o][k].
__device__ __forceinline__ void turn4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400);
    const uint32_t b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400);
    const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
    const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
    w[0] = __builtin_amdgcn_perm(b, a, 0x05040100);
    w[1] = __builtin_amdgcn_perm(b, a, 0x07060302);
    w[2] = __builtin_amdgcn_perm(d, c, 0x05040100);
    w[3] = __builtin_amdgcn_perm(d, c, 0x07060302);
}
__device__ __forceinline__ void store_packed(uint8_t* tile, uint8_t* packed, int64_t Co,
                                             int64_t kb, int64_t nb, int64_t kblocks) {
    // 8 column groups x 2 halves of K = 16 blocks of 64 units
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int i = p * 256 + threadIdx.x, blk = i >> 6, u = i & 63;
        const int o = (blk >> 1) * 16 + (u >> 2), c = (u & 3) ^ ((u >> 4) & 3);
        if (nb * 128 + o < Co)
            *reinterpret_cast<uint4*>(packed + ((nb * 8 + (blk >> 1)) * kblocks * 2 + kb * 2 +
                                                (blk & 1)) * 1024 + u * 16) =
                *reinterpret_cast<const uint4*>(tile_at_chunk(tile, o, (blk & 1) * 4 + c));
    }
}

__global__ __launch_bounds__(256) void quant_weight_block_kernel(
    const uint16_t* __restrict__ w, int64_t Ci, int64_t Co, int64_t ldw, int64_t se,
    uint8_t* __restrict__ packed, float* __restrict__ sw, int kb, int nb, int64_t blocks) {
    __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kPitch];
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t at = blockIdx.y * kWeightGridX + blockIdx.x;
    if (at >= blocks) return;
    const int64_t e = at / ((int64_t)kb * nb);
    const int r = (int)(at - e * kb * nb), n = r / kb, k = r - n * kb;
    const int64_t col = n * 128 + (tid & 15) * 8;
    const uint16_t* src = w + e * se;
    uint4 v[8];
    us2 m = {0, 0};
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t row = k * 128 + (tid >> 4) * 8 + p;
        const bool in = row < Ci && col < Co;
        v[p] = *reinterpret_cast<const uint4*>(src + (in ? row * ldw + col : 0));
        if (!in) v[p] = make_uint4(0, 0, 0, 0);
        m = max2(max2(m, abs_bits2(v[p].x)), max2(abs_bits2(v[p].y), abs_bits2(v[p].z)));
        m = max2(m, abs_bits2(v[p].w));
    }
    const uint32_t wave = wave_max_u32(hmax(m));
    if ((tid & 63) == 0) red[tid >> 6] = wave;
    __syncthreads();
    uint32_t top = red[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) top = top > red[i] ? top : red[i];
    const float scale = scale_from_amax(__uint_as_float(top << 16));
    const Divisor dv = make_divisor(scale);
    uint32_t c[2][2][4];                                 // [half of the columns][of K][byte row]
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const uint2 q = quantize8(v[p], dv);
        c[0][p >> 2][p & 3] = q.x;
        c[1][p >> 2][p & 3] = q.y;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        turn4(c[h][0]);
        turn4(c[h][1]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2*>(
                tile_at_chunk(tile, (tid & 15) * 8 + h * 4 + j, tid >> 5) + ((tid >> 4) & 1) * 8) =
                make_uint2(c[h][0][j], c[h][1][j]);
    }
    __syncthreads();
    store_packed(tile, packed + e * Co * kb * 128, Co, k, n, kb);
    if (tid == 0) sw[(e * nb + n) * kb + k] = scale;
}

__global__ __launch_bounds__(256) void pack_weight_block_kernel(PackArgs a, int kb, int nb,
                                                                int64_t blocks) {
    __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kPitch];
    const int tid = threadIdx.x;
    const int64_t block = blockIdx.y * kWeightGridX + blockIdx.x;
    if (block >= blocks) return;
    const int64_t e = block / ((int64_t)kb * nb);
    const int r = (int)(block - e * kb * nb), n = r / kb, k = r - n * kb;
    const uint8_t* src = a.codes + e * a.se;
    // 16 bytes at a time along the axis that is contiguous, if they are aligned
    const bool along_o = a.so == 1;
    const int64_t wide = along_o ? a.sk : a.so;
    const bool vec = (along_o || a.sk == 1) &&
                     ((reinterpret_cast<uintptr_t>(src) | (uintptr_t)wide) & 15) == 0;
    uint32_t w[4][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int outer = (tid >> 3) * 4 + p, inner = (tid & 7) * 16;
        const int ko = along_o ? outer : inner, oo = along_o ? inner : outer;
        const int64_t row = k * 128 + ko, col = n * 128 + oo;
        const bool in = row < a.Ci && col < a.Co;
        const uint8_t* at = src + (in ? row * a.sk + col * a.so : 0);
        w[p][0] = w[p][1] = w[p][2] = w[p][3] = 0;
        if (in && vec) {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            w[p][0] = v.x; w[p][1] = v.y; w[p][2] = v.z; w[p][3] = v.w;
        } else if (in) {
            const int64_t step = along_o ? 1 : a.sk;
#pragma unroll
            for (int j = 0; j < 16; ++j) w[p][j >> 2] |= (uint32_t)at[j * step] << (8 * (j & 3));
        }
        if (!along_o)
            *reinterpret_cast<uint4*>(tile_at_chunk(tile, oo, tid & 7)) =
                make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
    if (along_o) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t t[4] = {w[0][g], w[1][g], w[2][g], w[3][g]};
            turn4(t);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t*>(
                    tile_at_chunk(tile, (tid & 7) * 16 + g * 4 + j, tid >> 5) +
                    ((tid >> 3) & 3) * 4) = t[j];
        }
    }
    __syncthreads();
    store_packed(tile, a.packed + e * a.Co * kb * 128, a.Co, k, n, kb);
    if (tid == 0) a.sw[(e * nb + n) * kb + k] = a.scales[e * a.te + k * a.tk + n * a.to];
}

}  // namespace

hipError_t launch_quant_act_block(const uint16_t* x, int64_t T, int64_t C, int64_t ldx, bool gate,
                                  const int32_t* count, uint8_t* qx, int64_t ldq, float* sx,
                                  int64_t lds, hipStream_t s) {
    const int kb = (int)scale_blocks(C);
    // Few rows: one row per 16 lanes, for as many workgroups as there are; from
    // two rounds of the GPU on, four.
    const bool many = T * kb >= (int64_t)64 * 2048;
    const int64_t items = (T + (many ? 64 : 16) - 1) / (many ? 64 : 16) * kb;
    const dim3 grid((unsigned)(items < (1 << 22) ? items : (1 << 22)));
#define PTPC_LAUNCH(G, I) \
    quant_act_block_kernel<G, I><<<grid, 256, 0, s>>>(x, T, C, ldx, count, qx, ldq, sx, lds, kb, items)
    if (gate) {
        if (many) PTPC_LAUNCH(true, 4); else PTPC_LAUNCH(true, 1);
    } else {
        if (many) PTPC_LAUNCH(false, 4); else PTPC_LAUNCH(false, 1);
    }
#undef PTPC_LAUNCH
    return hipGetLastError();
}

hipError_t launch_quant_weight_block(const uint16_t* w, int64_t E, int64_t Ci, int64_t Co,
                                     int64_t ldw, int64_t se, uint8_t* packed, float* sw,
                                     hipStream_t s) {
    const int kb = (int)scale_blocks(Ci), nb = (int)scale_blocks(Co);
    const int64_t blocks = E * kb * nb;
    quant_weight_block_kernel<<<weight_grid(blocks), 256, 0, s>>>(w, Ci, Co, ldw, se, packed, sw, kb,
                                                                  nb, blocks);
    return hipGetLastError();
}

hipError_t launch_pack_weight_block(const PackArgs& a, hipStream_t s) {
    const int kb = (int)scale_blocks(a.Ci), nb = (int)scale_blocks(a.Co);
    const int64_t blocks = a.E * kb * nb;
    pack_weight_block_kernel<<<weight_grid(blocks), 256, 0, s>>>(a, kb, nb, blocks);
    return hipGetLastError();
}

}  // namespace ptpc
