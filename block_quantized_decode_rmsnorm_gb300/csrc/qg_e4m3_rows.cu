// The block-scaled e4m3 product for up to 16 activation rows: the weights are read
// once, straight into the fragments of mma.sync m16n8k32.
//
//   y[m][n] = sum_b (d_x[m][b] d_w[n/128][b]) S_b[m][n],  S_b = sum of x w over block b
//
// A warp takes 16 weight rows (the M side of the MMA) and 8 activation rows (its
// N side) over one block of 128 per step: four MMAs into a zeroed accumulator
// give S_b, which one product and one FMA per value bring into the sum.  The
// order of the values inside a block does not matter to S_b as long as both
// operands agree, so lane 4g+c loads bytes 16c..16c+15 of each half of its rows'
// block (two 64-byte pieces per row and instruction, whole sectors) and the eight
// words serve as the MMAs' register pairs as they are.  Eight warps split the
// blocks of k; their sums meet in shared memory in warp order.
//
// Gate|up: 16 gate and the 16 matching up rows per CTA, eight CTAs of a cluster
// hold the 128 outputs of one block of h, and exchange their largest magnitudes
// through distributed shared memory before each writes its 16 codes per row.
#include "qg_e4m3.cuh"

namespace qg {

constexpr int RW = 8;           // warps per CTA
constexpr int RR = 16;          // weight rows per CTA (and half, for gate|up)
constexpr int UP_CLUSTER = EB / RR;

struct RowsArgs {
    const uint8_t *w;
    const float *wd;
    int64_t n;         // output columns
    int64_t up_row;    // gate|up: first up row
    int64_t up_block;  // and its first row of scales
    int k, kb;
    const uint8_t *x;
    const float *xd;
    int64_t m;
    const void *residual;
    void *y;
    int y_bf16;
    uint8_t *hq;
    float *hd;
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// NT: groups of 8 activation rows; m <= 8 NT.
template <int NT, bool UP>
__global__ void __launch_bounds__(RW * 32, NT == 1 ? 3 : 2) rows_e4m3_kernel(const RowsArgs p)
{
    constexpr int RT = UP ? 2 : 1;  // weight tiles per CTA
    constexpr int U = UP ? 1 : 2;   // blocks of k in flight per warp
    __shared__ float red[RW][RT][NT * 8 * RR];
    __shared__ float top[NT * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * RR;

    // this lane's two rows of each tile: columns 0 ..  of row n0 + g (+ 8)
    const uint8_t *wr[RT][2];
    const float *wd[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        wd[t] = p.wd + ((t ? p.up_block : 0) + n0 / EB) * p.kb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = n0 + g + 8 * h;
            wr[t][h] = row < p.n ? p.w + ((t ? p.up_row : 0) + row) * p.k : nullptr;
        }
    }
    pdl_wait();
    pdl_trigger();

    const uint8_t *xr[NT];
    const float *xd[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t row = 8 * j + g;
        xr[j] = row < p.m ? p.x + row * p.k : nullptr;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r2 = 8 * j + 2 * c + h;
            xd[j][h] = r2 < p.m ? p.xd + r2 * p.kb : nullptr;
        }
    }
    float acc[RT][NT][4];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][j][i] = 0.0f;

    for (int b0 = warp; b0 < p.kb; b0 += RW * U) {
        uint4 wv[U][RT][2][2], xv[U][NT][2];
        float sw[U][RT], sx[U][NT][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * RW;
            const bool in = b < p.kb;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int col = b * EB + 64 * q + 16 * c;
                const bool ok = in && col < p.k;
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        wv[u][t][h][q] = ok && wr[t][h] ? ld_stream_16B(wr[t][h] + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    xv[u][j][q] = ok && xr[j] ? ld_16B(xr[j] + col) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) sw[u][t] = in ? wd[t][b] : 0.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) sx[u][j][h] = in && xd[j][h] ? xd[j][h][b] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u * RW >= p.kb) break;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 a = wv[u][t][0][q], a8 = wv[u][t][1][q], x = xv[u][j][q];
                        mma_e4m3(d, a.x, a8.x, a.y, a8.y, x.x, x.y);
                        mma_e4m3(d, a.z, a8.z, a.w, a8.w, x.z, x.w);
                    }
                    const float s0 = sx[u][j][0] * sw[u][t], s1 = sx[u][j][1] * sw[u][t];
                    acc[t][j][0] = fmaf(d[0], s0, acc[t][j][0]);
                    acc[t][j][1] = fmaf(d[1], s1, acc[t][j][1]);
                    acc[t][j][2] = fmaf(d[2], s0, acc[t][j][2]);
                    acc[t][j][3] = fmaf(d[3], s1, acc[t][j][3]);
                }
        }
    }
    // [activation row][weight row]: d[0], d[1] are row g of activations 2c, 2c + 1, d[2], d[3] row g + 8
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[warp][t][(8 * j + 2 * c + (i & 1)) * RR + g + 8 * (i >> 1)] = acc[t][j][i];
    __syncthreads();

    const int o = threadIdx.x;  // output: activation row o / 16, weight row o % 16
    const int64_t row = o / RR, col = n0 + o % RR;
    const bool mine = o < NT * 8 * RR, live = mine && row < p.m && col < p.n;
    float v[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        v[t] = mine ? red[0][t][o] : 0.0f;
#pragma unroll
        for (int w = 1; w < RW; ++w) v[t] += mine ? red[w][t][o] : 0.0f;
    }
    if constexpr (UP) {
        const float h = silu_mul_e(v[0], v[RT - 1]);
        float a = live ? fmaxf(fabsf(h), 0.0f) : 0.0f;
#pragma unroll
        for (int s = RR / 2; s >= 1; s >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
        if (mine && o % RR == 0) top[o / RR] = a;
        cluster_sync();
        if (mine) {
            a = 0.0f;
#pragma unroll
            for (int r = 0; r < UP_CLUSTER; ++r) a = fmaxf(a, ld_cluster_f32(&top[o / RR], r));
        }
        a = e4m3_floor(a);
        if (live) {
            p.hq[row * p.n + col] = static_cast<uint8_t>(e4m3_pack2(h * __fdiv_rn(448.0f, a), 0.0f));
            if (col % EB == 0) p.hd[row * e4m3_blocks(p.n) + col / EB] = __fdiv_rn(a, 448.0f);
        }
        cluster_sync();  // the others have read this CTA's maxima
    } else if (live) {
        const int64_t at = row * p.n + col;
        if (p.y_bf16) {
            const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(p.residual);
            const float out = res ? v[0] + __bfloat162float(res[at]) : v[0];
            static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(out);
        } else {
            const float *res = static_cast<const float *>(p.residual);
            static_cast<float *>(p.y)[at] = res ? v[0] + res[at] : v[0];
        }
    }
}

cudaError_t launch_rows_e4m3(const uint8_t *w, const float *wd, int64_t n, int64_t k, const uint8_t *x, const float *xd,
                             int64_t m, const void *residual, void *y, int y_dtype, cudaStream_t s)
{
    RowsArgs p = {};
    p.w = w;
    p.wd = wd;
    p.n = n;
    p.k = static_cast<int>(k);
    p.kb = static_cast<int>(e4m3_blocks(k));
    p.x = x;
    p.xd = xd;
    p.m = m;
    p.residual = residual;
    p.y = y;
    p.y_bf16 = y_dtype == QG_BF16;
    const unsigned gx = static_cast<unsigned>((n + RR - 1) / RR);
    if (m <= 8) return launch_pdl(rows_e4m3_kernel<1, false>, dim3(gx), dim3(RW * 32), 0, s, p);
    return launch_pdl(rows_e4m3_kernel<2, false>, dim3(gx), dim3(RW * 32), 0, s, p);
}

cudaError_t launch_rows_up_e4m3(const uint8_t *w, const float *wd, int64_t ffn, int64_t k, const uint8_t *x,
                                const float *xd, int64_t m, uint8_t *hq, float *hd, cudaStream_t s)
{
    RowsArgs p = {};
    p.w = w;
    p.wd = wd;
    p.n = ffn;
    p.up_row = ffn;
    p.up_block = e4m3_blocks(ffn);
    p.k = static_cast<int>(k);
    p.kb = static_cast<int>(e4m3_blocks(k));
    p.x = x;
    p.xd = xd;
    p.m = m;
    p.hq = hq;
    p.hd = hd;
    const unsigned gx = static_cast<unsigned>(e4m3_blocks(ffn) * UP_CLUSTER);
    if (m <= 8) return launch_pdl_cluster(rows_e4m3_kernel<1, true>, dim3(gx), dim3(RW * 32), 0, s, UP_CLUSTER, p);
    return launch_pdl_cluster(rows_e4m3_kernel<2, true>, dim3(gx), dim3(RW * 32), 0, s, UP_CLUSTER, p);
}

}  // namespace qg
