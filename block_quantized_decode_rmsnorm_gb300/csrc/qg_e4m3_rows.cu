// The block-scaled e4m3 product for up to 8 activation rows: the weights are read
// once, in the order in which mma.sync m16n8k32 takes them.
//
//   y[m][n] = sum_b (d_x[m][b] d_w[n/128][b]) S_b[m][n],  S_b = sum of x w over block b
//
// A warp takes 16 weight rows (the M side of the MMA) and 8 activation rows (its
// N side) over one block of 128 per step: four MMAs into a zeroed accumulator
// give S_b, which one product and one FMA per value bring into the sum.  The
// order of the values inside a block does not matter to S_b as long as both
// operands agree, so lane 4g+c takes bytes 16c..16c+15 of each half of its rows'
// block (two 64-byte pieces per row and instruction, whole sectors) and the eight
// words serve as the MMAs' register pairs as they are.  The warps of a CTA split
// the blocks of k; their sums meet in shared memory in warp order.
//
// What bounds it is the bytes in flight: a lane copies its own pieces of the next
// blocks to shared memory by cp.async (no barrier: nobody else reads them), without
// registers, from before the previous kernel has ended on.  A CTA has eight warps, so
// that few rows still fill the SMs' queues (1x1024x3584 with a residual: 2.6 us; four CTAs
// of a cluster sharing k took 1.2 more); where it then takes more than one wave, gate|up has
// four warps per CTA and four CTAs an SM (1x9216x2560: 10.4 us, 13.8 with eight warps;
// 1x2048x4096: 7.8 us, 5.9 with eight).
//
// Gate|up: 16 gate and the 16 matching up rows per CTA, eight CTAs of a cluster
// hold the 128 outputs of one block of h, and exchange their largest magnitudes
// through distributed shared memory before each writes its 16 codes per row.
//
// Times in this file are of graph replays over operands that rotate through 400 MB.
#include <algorithm>

#include "qg_e4m3.cuh"

namespace qg {

constexpr int RR = 16;          // weight rows per CTA (and half, for gate|up)
constexpr int UP_CLUSTER = EB / RR;
constexpr int R_TILE = RR * EB; // bytes of one tile's block

struct RowsArgs {
    const uint8_t *w;
    const float *wd;
    int64_t n;         // output columns
    int64_t tiles;     // of 16 weight rows
    int64_t up_row;    // gate|up: first up row
    int64_t up_block;  // and its first row of scales
    int k, kb;
    int ahead;         // bytes of a row, from behind the ring's first blocks on, to bring to L2
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

// What a CTA does: ONE tile of the product; a WALK over several, the next one's weights on
// their way while a tile ends (in the others nothing is kept of a next tile); one tile of
// gate and one of up, with eight warps or, NARROW, with half of them, so that twice the CTAs
// find room.
enum class Form { ONE, WALK, UP, UP_NARROW };

template <Form FORM>
struct RowsLayout {
    static constexpr bool UP = FORM == Form::UP || FORM == Form::UP_NARROW;
    static constexpr bool WALK = FORM == Form::WALK, NARROW = FORM == Form::UP_NARROW;
    static constexpr int W = NARROW ? 4 : 8;  // warps per CTA
    static constexpr int T = UP ? 2 : 1;      // weight tiles per CTA
    static constexpr int D = NARROW ? 2 : UP ? 3 : 6;  // blocks on their way per warp
    static constexpr int F = 3;            // steps whose activations are
    static constexpr int RING = W * D * T * R_TILE;  // 96 KB, or 32
    static constexpr int CTAS = NARROW ? 4 : 2;      // per SM
};

template <Form FORM>
__global__ void __launch_bounds__(RowsLayout<FORM>::W * 32, RowsLayout<FORM>::CTAS) rows_e4m3_kernel(const RowsArgs p)
{
    using L = RowsLayout<FORM>;
    constexpr bool UP = L::UP, WALK = L::WALK;
    constexpr int RW = L::W, RT = L::T, D = L::D, F = L::F;
    extern __shared__ __align__(16) uint8_t ring_raw[];  // [warp][slot][tile][row half][block half][lane] of 16 bytes
    __shared__ float red[WALK ? 2 : 1][RW][RT][8 * RR];  // [tile parity][warp]: one barrier a tile
    __shared__ float top[8];  // gate|up: the rows' largest magnitudes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int steps = (p.kb + RW - 1) / RW;  // of a tile: warp w takes blocks w, w + RW, ...
    const int slots = WALK ? D : min(D, steps);
    uint8_t *ring = ring_raw + static_cast<size_t>(warp) * slots * RT * R_TILE + lane * 16;

    // The next step's weights into its slot, tile after tile: zeros where there are
    // none; one group per step, empty past the last.
    int64_t s_tile = blockIdx.x;
    int s_step = 0, s_slot = 0;
    const uint8_t *wr[RT][2];  // this lane's rows of s_tile: columns 0 .. of row g (+ 8), or null
    auto rows = [&]() {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t row = s_tile * RR + g + 8 * h;
                wr[t][h] = row < p.n ? p.w + ((t ? p.up_row : 0) + row) * p.k : nullptr;
            }
    };
    rows();
    auto stage = [&]() {
        const int b = warp + RW * s_step;
        if ((!WALK || s_tile < p.tiles) && b < p.kb) {
            uint8_t *slot = ring + s_slot * RT * R_TILE;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int col = b * EB + 64 * q + 16 * c;
                        uint8_t *to = slot + ((t * 2 + h) * 2 + q) * 512;
                        if (wr[t][h] && col < p.k)
                            cp_async_16(smem_addr(to), wr[t][h] + col);
                        else
                            *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
                    }
        }
        cp_async_commit();
        ++s_step;
        if (WALK && s_step == steps) {
            s_step = 0;
            s_tile += gridDim.x;
            rows();
        }
        if (++s_slot == D) s_slot = 0;
    };
#pragma unroll
    for (int i = 0; i < D; ++i) stage();
    // what comes behind the ring's blocks into L2 meanwhile, a piece per row
    if (!L::NARROW && !WALK && p.ahead > 0 && threadIdx.x < RT * RR) {
        const int64_t row = static_cast<int64_t>(blockIdx.x) * RR + threadIdx.x % RR;
        if (row < p.n)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.w + ((threadIdx.x / RR ? p.up_row : 0) + row) * p.k + D * RW * EB),
                         "r"(p.ahead)
                         : "memory");
    }
    pdl_wait();
    pdl_trigger();

    const uint8_t *xr = g < p.m ? p.x + g * p.k : nullptr;
    const float *xd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) xd[h] = 2 * c + h < p.m ? p.xd + (2 * c + h) * p.kb : nullptr;

    // the activations and scales of the next F steps, in registers
    uint4 xn[F][2];
    float fw[F][RT], fx[F][2];
    int64_t f_tile = blockIdx.x;
    int f_step = 0;
    auto fetch = [&](int u) {
        const int b = warp + RW * f_step;
        const bool in = (!WALK || f_tile < p.tiles) && b < p.kb;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int col = b * EB + 64 * q + 16 * c;
            xn[u][q] = in && xr && col < p.k ? ld_16B(xr + col) : make_uint4(0, 0, 0, 0);
            fx[u][q] = in && xd[q] ? xd[q][b] : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
            fw[u][t] = in ? p.wd[((t ? p.up_block : 0) + f_tile * RR / EB) * p.kb + b] : 0.0f;
        ++f_step;
        if (WALK && f_step == steps) f_step = 0, f_tile += gridDim.x;
    };
#pragma unroll
    for (int u = 0; u < F; ++u) fetch(u);

    float acc[RT][4] = {};
    int64_t tile = blockIdx.x;
    int step = 0, slot_no = 0, parity = 0;
    // The residual of this thread's output of a tile (activation row threadIdx.x / 16,
    // weight row threadIdx.x % 16), loaded while the tile's blocks are (7.3 us at
    // 8x2560x9216 and 0.7 more without, 11.5 and 0.8 at 8x18432x2560, 2.6 and 0.1 at
    // 1x1024x3584; it costs 0.5 of 15.5 at 1x65536x1024 without a residual).
    float res = 0.0f;
    auto residual = [&]() {
        if (UP || !p.residual) return;
        const int row = threadIdx.x / RR;
        const int64_t col = tile * RR + threadIdx.x % RR, at = row * p.n + col;
        if (row >= p.m || col >= p.n) return;
        res = p.y_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.residual)[at])
                       : static_cast<const float *>(p.residual)[at];
    };
    residual();
    // the tile's sums of all warps, in warp order, and what becomes of them
    auto finish = [&]() {
        // [activation row][weight row]: values 0 and 1 are row g of activations 2c, 2c + 1, the others row g + 8
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[parity][warp][t][(2 * c + (e & 1)) * RR + g + 8 * (e >> 1)] = acc[t][e];
        __syncthreads();

        // a thread per output: activation row o / 16, weight row o % 16
        const int o = threadIdx.x, row = o / RR;
        const int64_t col = tile * RR + o % RR;
        const bool mine = o < 8 * RR, live = mine && row < p.m && col < p.n;
        float v[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            v[t] = mine ? red[parity][0][t][o] : 0.0f;
#pragma unroll
            for (int w = 1; w < RW; ++w) v[t] += mine ? red[parity][w][t][o] : 0.0f;
        }
        if constexpr (UP) {
            const float h = silu_mul_e(v[0], v[RT - 1]);
            float a = live ? fmaxf(fabsf(h), 0.0f) : 0.0f;
#pragma unroll
            for (int s = RR / 2; s >= 1; s >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
            if (mine && o % RR == 0) top[row] = a;
            cluster_sync();
            if (live) {
#pragma unroll
                for (int r = 0; r < UP_CLUSTER; ++r) a = fmaxf(a, ld_cluster_f32(&top[row], r));
                a = e4m3_floor(a);
                p.hq[row * p.n + col] = static_cast<uint8_t>(e4m3_pack2(h * __fdiv_rn(448.0f, a), 0.0f));
                if (col % EB == 0) p.hd[row * e4m3_blocks(p.n) + col / EB] = __fdiv_rn(a, 448.0f);
            }
            cluster_sync();  // the others have read this CTA's maxima
        } else if (live) {
            const int64_t at = row * p.n + col;
            const float out = p.residual ? v[0] + res : v[0];
            if (p.y_bf16)
                static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(out);
            else
                static_cast<float *>(p.y)[at] = out;
        }
    };
    bool more = true;
#pragma unroll 1
    while (more) {
#pragma unroll
        for (int u = 0; u < F; ++u) {
            cp_async_wait<D - 1>();
            if (warp + RW * step < p.kb) {
                const uint8_t *slot = ring + slot_no * RT * R_TILE;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(slot + (t * 4 + q) * 512);
                        const uint4 a8 = *reinterpret_cast<const uint4 *>(slot + (t * 4 + 2 + q) * 512);
                        mma_e4m3(d, a.x, a8.x, a.y, a8.y, xn[u][q].x, xn[u][q].y);
                        mma_e4m3(d, a.z, a8.z, a.w, a8.w, xn[u][q].z, xn[u][q].w);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(d[e], fx[u][e & 1] * fw[u][t], acc[t][e]);
                }
            }
            if (++step == steps) {
                if (!WALK) {
                    more = false;
                    break;
                }
                finish();
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][e] = 0.0f;
                step = 0;
                tile += gridDim.x;
                parity ^= 1;
                if (tile >= p.tiles) {
                    more = false;
                    break;
                }
                residual();
            }
            if (++slot_no == D) slot_no = 0;
            stage();  // into the slot just read
            fetch(u);
        }
    }
    if (!WALK) finish();
}

// At most three CTAs of eight warps on two SMs (of the four that find room).
static bool few(int64_t tiles) { return 4 * tiles <= 3 * RowsLayout<Form::ONE>::CTAS * static_cast<int64_t>(num_sms()); }
static_assert(RowsLayout<Form::ONE>::CTAS == RowsLayout<Form::UP>::CTAS, "few");

template <Form FORM>
static cudaError_t launch_rows(int64_t ctas, RowsArgs p, cudaStream_t s)
{
    using L = RowsLayout<FORM>;
    const int need = (p.kb + L::W - 1) / L::W;
    constexpr int ring = L::D * L::W * EB;  // columns in flight
    // Where the next kernel's CTAs find room beside these, a second ring's columns go to L2
    // before the wait (7x2560x9216 bf16: 7.9 -> 7.2 us, 1x2560x12288: 9.1 -> 8.3, gate|up
    // 1x512x9216: 8.9 -> 8.6); with two CTAs an SM it is no gain (1x4096x14336: 11.2 us, 1.0
    // more with all columns).
    if (few(p.tiles)) p.ahead = std::max(0, std::min(p.k - ring, ring));
    const int bytes = L::W * (L::WALK || need > L::D ? L::D : need) * L::T * R_TILE;
    const auto kernel = rows_e4m3_kernel<FORM>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), L::RING); e != cudaSuccess) return e;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(ctas)), dim3(L::W * 32), static_cast<size_t>(bytes), s,
                              L::UP ? UP_CLUSTER : 1, p);
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
    p.tiles = (n + RR - 1) / RR;
    // More tiles than CTAs find room: as many each (1x65536x1024: 15.5 us against 22.3 with
    // a CTA to each, 8x18432x2560 11.5 and 12.8; one each, 1x1024x3584: 2.6 us against 2.9 by
    // the kernel that walks, 7x2560x9216 7.2 and 8.4).
    const int64_t room = RowsLayout<Form::ONE>::CTAS * static_cast<int64_t>(num_sms());
    if (p.tiles <= room) return launch_rows<Form::ONE>(p.tiles, p, s);
    const int64_t each = (p.tiles + room - 1) / room;
    return launch_rows<Form::WALK>((p.tiles + each - 1) / each, p, s);
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
    p.tiles = e4m3_blocks(ffn) * UP_CLUSTER;
    // Eight warps a CTA up to there: 1x512x2560 3.4 us and 4.9 with four, 8x3584x2560 6.4 and
    // 7.0, 8x3584x1024 4.3 and 4.2; 8x4608x2560 8.9 and 7.8.
    if (few(p.tiles)) return launch_rows<Form::UP>(p.tiles, p, s);
    return launch_rows<Form::UP_NARROW>(p.tiles, p, s);
}

}  // namespace qg
