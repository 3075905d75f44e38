// The block-scaled FP8 product for few rows of each weight (gfx950 MFMA).
//
// Up to 64 rows a weight the product is a stream of the weight.  A workgroup
// owns 16 * NT columns and 16 * MT rows; its waves deal the K blocks among
// themselves (wave w takes blocks w, w + NW, ...) and load both operands
// straight into registers, DEPTH blocks ahead, so that no wave ever waits for
// another before the end.  There the waves' sums meet in LDS and are added in
// wave order.
#include "block_device.h"

namespace ptpc {
namespace {

template <int MT, int NT, int NW, int DEPTH, bool EXPERTS>
__global__ __launch_bounds__(NW * 64, 2) void block_few_kernel(BlockGemmArgs g) {
    constexpr int BM = 16 * MT, BN = 16 * NT;
    static_assert(128 % BN == 0, "one weight block a workgroup");
    __shared__ v4f red[NW][MT * NT][64];
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int gn = (int)((g.Co + BN - 1) / BN);
    const int nks = (int)scale_blocks(g.Ci);

    int tm, tn, expert = 0, row0, row_end;
    if constexpr (EXPERTS) {
        const ExpertTiles t = count_expert_tiles<BM>(g.offsets, g.E, (int)g.T);
        if ((int)blockIdx.x >= t.total * gn) return;
        const int i = xcd_order(blockIdx.x, t.total * gn);
        tm = uniform(i / gn);
        tn = uniform(i - tm * gn);
        find_expert_tile<BM>(g.offsets, g.E, (int)g.T, t, tm, expert, row0, row_end);
        if (expert < 0) return;
    } else {
        tm = uniform(blockIdx.x / gn);
        tn = uniform(blockIdx.x - tm * gn);
        row0 = tm * BM;
        row_end = (int)g.T;
    }
    const int rows = row_end - row0 < BM ? row_end - row0 : BM;
    const int64_t n0 = (int64_t)tn * BN;
    const int64_t Kp = (int64_t)nks * 128;
    const bool gather = EXPERTS && g.rows != nullptr;

    const __amdgpu_buffer_rsrc_t ra =
        gather ? make_rsrc(g.qx, (uint32_t)(g.T_in * g.ldq))
               : make_rsrc(g.qx + (int64_t)row0 * g.ldq, (uint32_t)(rows * g.ldq));
    const int64_t b_cols = g.Co - n0 < BN ? g.Co - n0 : BN;
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(g.wp + (int64_t)expert * g.Co * Kp + n0 * Kp, (uint32_t)(b_cols * Kp));
    const float* const sx0 = g.sx + (gather ? 0 : row0);
    const uint32_t sx_bytes = (uint32_t)((gather ? g.T_in : rows) * 4);
    const int nblocks = (int)scale_blocks(g.Co);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(
        g.sw + ((int64_t)expert * nblocks + (int)(n0 / 128)) * nks, (uint32_t)(nks * 4));

    uint32_t a_off[MT], s_off[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = i * 16 + l16;
        int t = r < rows ? r : -1;
        if (gather && t >= 0) {
            const int p = g.rows[row0 + r];
            t = p < 0 ? -1 : p / g.top_k;
            if (t >= (int)g.T_in) t = -1;
        }
        a_off[i] = t >= 0 ? (uint32_t)(t * g.ldq + 16 * q) : kNowhere;
        s_off[i] = t >= 0 ? (uint32_t)t * 4 : kNowhere;
    }
    // Column l % 16 of a 1 KB block: chunk q of its 64 bytes, in the packing's order.
    const uint32_t b_off = (uint32_t)(l16 * 64 + ((q ^ (l16 >> 2)) << 4));

    v4i fw[DEPTH][NT][2], fx[DEPTH][MT][2];
    float sx[DEPTH][MT], sw[DEPTH];
    auto load = [&](int d, int ks) {
        const int left = (int)g.Ci - ks * 128;           // <= 0 past the last block
        const int kc = uniform(left > 0 ? ks : 0);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                fw[d][j][h] = __builtin_amdgcn_raw_buffer_load_b128(
                    rb, left > 0 ? b_off + (uint32_t)(j * nks * 2048 + h * 1024) : kNowhere,
                    kc * 2048, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                fx[d][i][h] = __builtin_amdgcn_raw_buffer_load_b128(
                    ra, 64 * h + 16 * q < left ? a_off[i] + 64 * h : kNowhere, kc * 128, 0);
            const __amdgpu_buffer_rsrc_t rs =
                make_rsrc(sx0 + (int64_t)kc * g.lds, left > 0 ? sx_bytes : 0);
            sx[d][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, s_off[i], 0, 0));
        }
        sw[d] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, 0, kc * 4, 0));
    };

    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(d, wave + NW * d);
    for (int k0 = wave; k0 < nks; k0 += NW * DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float f = sx[d][i] * sw[d];
                const v8i x = join(fx[d][i][0], fx[d][i][1]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const v4f t = mfma_block(join(fw[d][j][0], fw[d][j][1]), x);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = __builtin_fmaf(t[e], f, acc[i][j][e]);
                }
            }
            load(d, k0 + NW * (d + DEPTH));
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    // (row slab, column slab) tiles, dealt to the waves
    const __amdgpu_buffer_rsrc_t ro =
        make_rsrc(g.out + (int64_t)row0 * g.ldo, (uint32_t)(rows * g.ldo * 2));
#pragma unroll
    for (int n0w = 0; n0w < MT * NT; n0w += NW) {
        const int n = n0w + wave;
        if (n >= MT * NT) break;
        v4f v = red[0][n][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            const v4f o = red[w][n][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += o[e];
        }
        const int r = (n / NT) * 16 + l16;
        const int64_t col = n0 + (n % NT) * 16 + 4 * q;
        typedef int v2i __attribute__((ext_vector_type(2)));
        const v2i b = {(int)f32x2_to_bf16x2_rne(v[0], v[1]), (int)f32x2_to_bf16x2_rne(v[2], v[3])};
        __builtin_amdgcn_raw_buffer_store_b64(
            b, ro, col < g.Co && r < rows ? (uint32_t)((r * g.ldo + col) * 2) : kNowhere, 0, 0);
    }
}

template <int MT, int NT, int NW, int DEPTH>
hipError_t launch(const BlockGemmArgs& a, BlockPlan p, hipStream_t s) {
    const dim3 grid((unsigned)block_gemm_grid(p, a.T, a.offsets ? a.E : 0, a.Co));
    if (a.offsets != nullptr)
        block_few_kernel<MT, NT, NW, DEPTH, true><<<grid, NW * 64, 0, s>>>(a);
    else
        block_few_kernel<MT, NT, NW, DEPTH, false><<<grid, NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_gemm_few(const BlockGemmArgs& a, BlockPlan p, hipStream_t s) {
    switch (p) {
        case BlockPlan::kFew64: return launch<4, 2, 8, 2>(a, p, s);
        case BlockPlan::kFew32: return launch<2, 2, 8, 3>(a, p, s);
        default: return launch<1, 2, 8, 4>(a, p, s);
    }
}

}  // namespace ptpc
