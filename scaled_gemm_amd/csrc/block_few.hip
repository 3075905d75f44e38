// The block-scaled FP8 product for up to 16 rows of one weight (gfx950 MFMA).
//
// A stream of the weight.  Where tiles of 64 columns are too few for the GPU's
// CUs (long K, few columns), a workgroup owns 16 columns, its eight waves deal
// the K blocks among themselves (wave w takes blocks w, w + 8, ...) and load both
// operands straight into registers, DEPTH blocks ahead, so that no wave waits for
// another before the end.  There the waves' sums meet in LDS and are added in wave
// order.
//
// What bounds it: the loads' latency; one token through 8192 x 2048 takes 8.9 us
// (the 32x64 tiles: 12.9), through 16384 x 4096 16.9 us (31.0; the weight alone
// would take 13.7 at 4.9 TB/s).
#include "block_device.h"

namespace ptpc {
namespace {

constexpr int NW = 8, DEPTH = 6;

__global__ __launch_bounds__(NW * 64, 2) void block_few_kernel(BlockGemmArgs g) {
    __shared__ v4f red[NW][64];
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = uniform(threadIdx.x >> 6);
    const int nks = (int)scale_blocks(g.Ci);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t Kp = (int64_t)nks * 128;

    const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.qx, (uint32_t)(g.T * g.ldq));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.wp + n0 * Kp, (uint32_t)(16 * Kp));
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(g.sw + n0 / 128 * nks, (uint32_t)(nks * 4));
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(g.out, (uint32_t)(g.T * g.ldo * 2));
    const uint32_t a_off = l16 < g.T ? (uint32_t)(l16 * g.ldq + 16 * q) : kNowhere;
    const uint32_t s_off = l16 < g.T ? (uint32_t)l16 * 4 : kNowhere;
    // Column l % 16 of a 1 KB block: chunk q of its 64 bytes, in the packing's order.
    const uint32_t b_off = (uint32_t)(l16 * 64 + ((q ^ (l16 >> 2)) << 4));

    v4i fw[DEPTH][2], fx[DEPTH][2];
    float sx[DEPTH], sw[DEPTH];
    auto load = [&](int d, int ks) {
        const int left = (int)g.Ci - ks * 128;           // <= 0 past the last block
        const int kc = uniform(left > 0 ? ks : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fw[d][h] = __builtin_amdgcn_raw_buffer_load_b128(
                rb, left > 0 ? b_off + h * 1024 : kNowhere, kc * 2048, 0);
            fx[d][h] = __builtin_amdgcn_raw_buffer_load_b128(
                ra, 64 * h + 16 * q < left ? a_off + 64 * h : kNowhere, kc * 128, 0);
        }
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(g.sx + (int64_t)kc * g.lds, left > 0 ? (uint32_t)(g.T * 4) : 0);
        sx[d] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, s_off, 0, 0));
        sw[d] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(rw, left > 0 ? 0 : kNowhere, kc * 4, 0));
    };

    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(d, wave + NW * d);
#pragma clang loop unroll(disable)
    for (int k0 = wave; k0 < nks; k0 += NW * DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const float s = sx[d] * sw[d];
            const v4f t = mfma_block(join(fw[d][0], fw[d][1]), join(fx[d][0], fx[d][1]));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(t[e], s, acc[e]);
            load(d, k0 + NW * (d + DEPTH));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    v4f v = red[0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        const v4f o = red[w][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    store4(ro, v, l16 < g.T ? (uint32_t)((l16 * g.ldo + n0 + 4 * q) * 2) : kNowhere);
}

}  // namespace

hipError_t launch_block_gemm_few(const BlockGemmArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)block_gemm_grid(BlockPlan::kFew, a.T, 0, a.Co));
    block_few_kernel<<<grid, NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace ptpc
