// The block-scaled e4m3 product on tcgen05, for more rows than the few-row kernel
// takes.
//
//   y[m][n] = sum_b (d_x[m][b] d_w[n/128][b]) S_b[m][n],  S_b = sum of x w over block b
//
// A tile is 128 activation rows (TMEM lanes) by BN weight rows (TMEM columns).  Per
// block of 128, one thread copies the 128-byte wide slabs of both operands by TMA
// (128-byte swizzle), one thread issues four tcgen05.mma kind::f8f6f4 (K = 32) into
// one of two to four TMEM buffers, and the epilogue warps bring the block sum into f32
// registers: a warp takes a quarter of the lanes and 64 columns, a thread one
// activation row of them.  Those lie in one block of weight rows, so the factor
// d_x d_w is one register and a value costs half a packed FMA.  One more warp reads
// the scales ahead, four blocks at a time, into shared memory.
//
// Gate|up: 128 gate rows and the 128 matching up rows make the 256 columns; a warp
// takes 32 of each, so that SiLU(g) * u stays in its registers, and the four warps of
// a quarter exchange their rows' largest magnitudes before the codes are written.
//
// Two forms.  tiles_e4m3_kernel walks the tiles with one CTA per SM.  Where there
// are too few tiles for the SMs, split_e4m3_kernel puts a cluster on each tile: its
// CTAs take consecutive parts of k, leave their sums in shared memory, and each adds
// up (in rank order, through distributed shared memory) and finishes a share of the
// rows.
//
// Every barrier wait is bounded by the global timer; a stalled pipeline aborts instead
// of hanging: the CTA waits (bounded) for the copies and MMAs that it has issued, and the
// tiles that it has left become NaN outputs or codes (a cluster's tile as a whole).
//
// Times in this file are of graph replays over operands that rotate through 400 MB.
// Gate|up 8192x9216x2560 305 us (2.53 PFLOP/s; 333 under the power cap that sets in after a
// second), product 4096x2560x9216 with the residual 79 us (87).  Both are bound by the
// hand-over of the two TMEM buffers, all that TMEM holds at N = 256: an MMA's 512 cycles, the
// 365 to 390 of reading its sums (whatever the loads' width) and some 700 between the two
// make about 800 a block.  Behind that comes the operands' way from L2 (227 and 73 us
// alone).  100x2727x3600 takes 8.7 us, bound by its chain of latencies.
#include <algorithm>
#include <cuda.h>
#include <type_traits>

#include "qg_e4m3.cuh"
#include "qg_tc.cuh"

namespace qg {

constexpr int TM = 128;    // activation rows per tile
constexpr int T_CW = 64;   // tile columns per epilogue warp
constexpr int T_XP = 9;    // row stride (floats) of a warp's 32 x 8 transpose buffer
constexpr int T_SB = 4;    // blocks of k per buffer of scales
constexpr int T_STAGES = 8;  // stages at most
constexpr int T_SPLIT = 6;   // CTAs sharing a tile at most

template <int BN>
struct TileLayout {
    static constexpr int CG = BN / T_CW;  // column groups
    static constexpr int EW = 4 * CG;     // epilogue warps: four lane quarters x column groups
    static constexpr int TMA_WARP = EW, MMA_WARP = EW + 1, SCALE_WARP = EW + 2;
    static constexpr int THREADS = (EW + 3) * 32;
    static constexpr int W = BN * EB;          // a stage: the weights' slab, then the activations'
    static constexpr int STAGE = W + TM * EB;
    static constexpr int FIT = 196608 / STAGE;
    static constexpr int STAGES = FIT < T_STAGES ? FIT : T_STAGES;
    // TMEM buffers: narrow tiles' blocks take less time than it takes from an MMA's issue
    // to its buffer's release, so they have four on their way (two CTAs an SM share TMEM
    // where BN is 64).  Never more than the stages, or a phase could be missed.
    static constexpr int BUFS = BN <= 128 ? 4 : 2;
    static constexpr int TMEM = BN == 192 ? 512 : BUFS * BN;  // columns allocated: a power of two
    static constexpr int BYTES = STAGES * STAGE + 1024;     // + alignment of the base
    static constexpr int ANY_BYTES = BYTES + EW * 32 * T_XP * 4;  // + the transpose buffers
    static constexpr int SPLIT_CTAS = BN == 64 ? 2 : 1;     // per SM, of the split kernel
    static constexpr int SPLIT_ROOM = (SPLIT_CTAS == 2 ? 100 : 210) * 1024;  // shared memory of its stages at most
    static constexpr int LD = BN + 4;                       // row stride (floats) of a split tile's sums
    static_assert(ANY_BYTES <= 220 * 1024 && STAGES >= BUFS, "shared memory");
};

struct TileArgs {
    const float *wd, *xd;
    int64_t m, n;        // n: output columns
    int64_t up_row, up_block;
    int kb;
    int m_tiles, tiles;
    int box_m;           // activation rows per copy
    int split;           // CTAs per tile, and of each the stages and their bytes
    int stages, stage;
    const void *residual;
    void *y;
    int y_bf16;
    uint8_t *hq;
    float *hd;
    static constexpr uint64_t limit_ns = kCopyWaitLimitNs;  // of a barrier wait
};

// With a stall made on purpose (qg_debug_stalled_e4m3): CTA `cta` issues the copies of its
// block number `block` late, and waits are shorter.  A type of its own, and kernels of its
// own: the limit as a value and the comparison per block cost the others 1 %.
struct StalledArgs : TileArgs {
    int64_t cta, block;
    static constexpr uint64_t limit_ns = 5000000, hold_ns = 50000000;
};
template <class P>
constexpr bool kStalls = std::is_same<P, StalledArgs>::value;

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(
                     d_tmem),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Barriers, and the factors d_x d_w of T_SB blocks of k at a time, in two buffers: per
// activation row two, as a tile's columns lie in at most two blocks of weight rows
// (gate|up: the gate's and the up's).
struct TileShared {
    uint64_t full[T_STAGES], done[T_STAGES], tempty[4], sfull[2], sempty[2];
    float2 f[2][T_SB][TM];
    uint32_t tmem;
    int abort_flag;
    uint32_t issued[2];  // the walk: blocks that the copy warp and the MMA warp have issued, at the end
};

// First column (in the tile) of half i (32 columns) of column group cg.
template <bool UP>
__device__ __forceinline__ constexpr int half_col(int cg, int i)
{
    return UP ? 128 * i + 32 * cg : T_CW * cg + 32 * i;
}

template <int BN>
__device__ __forceinline__ void tile_setup(TileShared &b, int warp)
{
    using L = TileLayout<BN>;
    if (threadIdx.x == 0) {
        b.abort_flag = 0;
        for (int i = 0; i < T_STAGES; ++i) {
            mbar_init(&b.full[i], 1);  // the copy thread's expect_tx
            mbar_init(&b.done[i], 1);  // the MMA thread's commit
        }
        for (int i = 0; i < L::BUFS; ++i) mbar_init(&b.tempty[i], L::EW);  // one arrival per epilogue warp
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.sfull[i], 1);       // the scale warp
            mbar_init(&b.sempty[i], L::EW);  // one arrival per epilogue warp
        }
    }
    if (warp == L::MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&b.tmem)),
                     "r"(L::TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// tc_wait for barriers that have mostly completed by the time they are asked for: one
// plain try first, 13 cycles against the 103 of tc_wait's way in (its suspended try and
// what surrounds it), five times per block.
template <class P>
__device__ __forceinline__ bool stage_wait(uint64_t *bar, uint32_t parity, TileShared &b)
{
    return mbar_try_wait(bar, parity) || tc_wait(bar, parity, &b.abort_flag, P::limit_ns);
}

// One lane of a converged warp.  The tensor core's and the copy engine's
// instructions take uniform registers: behind elect.sync the compiler knows that one
// lane is left, behind a lane's number it does not, and an MMA then took 148 cycles
// to issue, whatever its size (104 here, and 128 of the tensor core's for N = 256).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(p));
    return p != 0;
}

// done[s] completes when the MMAs that read stage s have: the stage may be filled
// again, and the block's sums may be read.  (One commit for both: a second one per
// block cost the issuing thread as much as an MMA.)  The copy warp is never more than
// the stages' number of blocks ahead of the MMAs, nor the MMAs more than the buffers'
// number, which is no larger, ahead of the epilogue: a phase's parity says which one
// it is.

// Number and bytes of the stages: the layout's, or what a split tile's launch chose.
template <int BN, bool SPLIT>
__device__ __forceinline__ uint32_t stages_of(const TileArgs &p)
{
    return SPLIT ? p.stages : TileLayout<BN>::STAGES;
}
template <int BN, bool SPLIT>
__device__ __forceinline__ uint32_t stage_bytes(const TileArgs &p)
{
    return SPLIT ? p.stage : TileLayout<BN>::STAGE;
}

template <int BN, bool UP>
__device__ __forceinline__ void copy_weights(const CUtensorMap &tw, const TileArgs &p, TileShared &b, uint8_t *st,
                                             uint32_t s, int n0, int kb)
{
    mbar_expect_tx(&b.full[s], (p.box_m + BN) * EB);
    tma_load_2d(st, &tw, kb * EB, n0, &b.full[s]);
    if constexpr (UP) tma_load_2d(st + 128 * EB, &tw, kb * EB, static_cast<int>(p.up_row + n0), &b.full[s]);
}

// Copies of blocks [kb0, kb1) of one tile; `it` counts blocks over all tiles.  A split
// tile's first weights go out before the wait for the previous kernel, which makes the
// activations.
template <int BN, bool UP, bool SPLIT, class P>
__device__ __forceinline__ bool tile_copies(const CUtensorMap &tx, const CUtensorMap &tw, const P &p,
                                            TileShared &b, uint8_t *smem, int m0, int n0, int kb0, int kb1,
                                            uint32_t &it)
{
    using L = TileLayout<BN>;
    const uint32_t S = stages_of<BN, SPLIT>(p), bytes = stage_bytes<BN, SPLIT>(p);
    int early = kb0;  // weights of the blocks before this one are on their way
    if constexpr (SPLIT) {
        early = min(kb1, kb0 + static_cast<int>(S));
        if (elect_one())
            for (int kb = kb0; kb < early; ++kb) copy_weights<BN, UP>(tw, p, b, smem + (kb - kb0) * bytes, kb - kb0, n0, kb);
        __syncwarp();
        pdl_wait();
    }
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % S, use = it / S;
        if (!__all_sync(0xffffffffu, stage_wait<P>(&b.done[s], (use & 1) ^ 1, b))) return false;
        if constexpr (kStalls<P>)
            if (p.cta == blockIdx.x && p.block == it)
                for (const uint64_t t0 = global_ns(); global_ns() - t0 < P::hold_ns;) __nanosleep(1000);
        if (elect_one()) {
            uint8_t *st = smem + s * bytes;
            if (kb >= early) copy_weights<BN, UP>(tw, p, b, st, s, n0, kb);
            tma_load_2d(st + L::W, &tx, kb * EB, m0, &b.full[s]);
        }
        __syncwarp();
    }
    return true;
}

// The MMAs of one tile's blocks, each into its own TMEM buffer.
template <int BN, bool SPLIT, class P>
__device__ __forceinline__ bool tile_mmas(const P &p, TileShared &b, uint32_t tmem, uint64_t desc0, int blocks,
                                          uint32_t &it)
{
    using L = TileLayout<BN>;
    const uint32_t S = stages_of<BN, SPLIT>(p), step = stage_bytes<BN, SPLIT>(p) >> 4;
    // D f32, A and B e4m3, both K-major
    constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(TM >> 4) << 24);
    for (int i = 0; i < blocks; ++i, ++it) {
        const uint32_t s = it % S, use = it / S, t = it % L::BUFS, tuse = it / L::BUFS;
        const bool ok = stage_wait<P>(&b.full[s], use & 1, b) && stage_wait<P>(&b.tempty[t], (tuse & 1) ^ 1, b);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc_fence_after();
        if (elect_one()) {
            const uint64_t w = desc0 + s * step, a = w + (L::W >> 4);  // the address field, in 16 bytes
#pragma unroll
            for (int k = 0; k < EB / 32; ++k) umma_f8(tmem + t * BN, a + 2 * k, w + 2 * k, idesc, k != 0);
            umma_commit(&b.done[s]);
        }
        __syncwarp();
    }
    return true;
}

// The scale warp: the factors of blocks [kb0, kb1) of one tile, T_SB at a time, the
// next scales on their way while the last factors are waited for.  `c` counts buffers.
template <int BN, bool UP, class P>
__device__ __forceinline__ bool tile_scales(const P &p, TileShared &b, int lane, int m0, int n0, int kb0,
                                            int kb1, uint32_t &c)
{
    const float *xr[TM / 32];
#pragma unroll
    for (int i = 0; i < TM / 32; ++i) xr[i] = p.xd + min(static_cast<int64_t>(m0 + 32 * i + lane), p.m - 1) * p.kb;
    const int64_t b0 = n0 / EB, b1 = UP ? p.up_block + b0 : min(b0 + 1, (p.n - 1) / EB);
    const float *w0 = p.wd + b0 * p.kb, *w1 = p.wd + b1 * p.kb;
    const bool vec = (p.kb % 4 == 0) && (kb0 % 4 == 0) && (reinterpret_cast<uintptr_t>(p.xd) & 15) == 0;
    for (int kb = kb0; kb < kb1; kb += T_SB, ++c) {
        float x[TM / 32][T_SB], wa[T_SB], wb[T_SB];
#pragma unroll
        for (int i = 0; i < TM / 32; ++i) {
            if (vec) {
                const float4 v = *reinterpret_cast<const float4 *>(xr[i] + kb);  // kb % 4 == 0 and so is the row's length
                x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
            } else {
#pragma unroll
                for (int o = 0; o < T_SB; ++o) x[i][o] = kb + o < kb1 ? xr[i][kb + o] : 0.0f;
            }
        }
#pragma unroll
        for (int o = 0; o < T_SB; ++o) {
            wa[o] = kb + o < kb1 ? w0[kb + o] : 0.0f;
            wb[o] = kb + o < kb1 ? w1[kb + o] : 0.0f;
        }
        const uint32_t t = c & 1, use = c >> 1;
        if (!__all_sync(0xffffffffu, stage_wait<P>(&b.sempty[t], (use & 1) ^ 1, b))) return false;
#pragma unroll
        for (int i = 0; i < TM / 32; ++i)
#pragma unroll
            for (int o = 0; o < T_SB; ++o) b.f[t][o][32 * i + lane] = make_float2(x[i][o] * wa[o], x[i][o] * wb[o]);
        __syncwarp();
        if (elect_one()) mbar_arrive(&b.sfull[t]);
    }
    return true;
}

// The sums of blocks [kb0, kb1) of one tile in registers: two halves of 32 columns of
// this thread's row, in adjacent pairs.  `it` counts blocks, `c` buffers of scales.
template <int BN, bool UP, bool SPLIT, class P>
__device__ __forceinline__ bool tile_sums(const P &p, TileShared &b, uint32_t tmem, int q, int cg, int lane,
                                          int n0, int kb0, int kb1, uint32_t &it, uint32_t &c,
                                          uint64_t (&acc)[2][16])
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0;
    const int second = UP ? 0 : (n0 + T_CW * cg) / EB - n0 / EB;  // this warp's columns lie in the second block
    for (int kb = kb0; kb < kb1; kb += T_SB, ++c) {
        const uint32_t sb = c & 1, suse = c >> 1;
        if (!__all_sync(0xffffffffu, stage_wait<P>(&b.sfull[sb], suse & 1, b))) return false;
#pragma unroll 1
        for (int o = 0; o < T_SB; ++o) {
            if (kb + o >= kb1) break;
            float f0, f1;
            if constexpr (UP) {
                const float2 f = b.f[sb][o][32 * q + lane];
                f0 = f.x, f1 = f.y;
            } else {
                f0 = f1 = reinterpret_cast<const float *>(&b.f[sb][o][32 * q + lane])[second];
            }
            if (o == T_SB - 1 || kb + o + 1 == kb1) {  // the buffer's last: every lane has read it
                __syncwarp();
                if (elect_one()) mbar_arrive(&b.sempty[sb]);
            }
            const uint32_t t = it % TileLayout<BN>::BUFS, s = it % stages_of<BN, SPLIT>(p),
                           use = it / stages_of<BN, SPLIT>(p);
            // tcgen05.ld is warp-collective: the whole warp proceeds or stops
            if (!__all_sync(0xffffffffu, stage_wait<P>(&b.done[s], use & 1, b))) return false;
            tc_fence_after();
            const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + t * BN;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t v[8];
                tmem_ld_8(ta + half_col<UP>(cg, i >> 2) + 8 * (i & 3), v);
                tmem_ld_wait_regs8(v);
                if (i == 7) {
                    tc_fence_before();
                    __syncwarp();
                    if (elect_one()) mbar_arrive(&b.tempty[t]);
                }
                const float f = i >> 2 ? f1 : f0;
                const uint64_t ff = pack2(f, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint64_t &sum = acc[i >> 2][4 * (i & 3) + j];
                    sum = fma2(pack2u(v[2 * j], v[2 * j + 1]), ff, sum);
                }
            }
            ++it;
        }
    }
    return true;
}

// After every role's last block, and all threads behind a __syncthreads: without an abort
// the MMA warp has waited for every copy and the epilogue for every MMA.  After one, waits
// (bounded) for whatever this warp has issued (`issued` blocks, of the copy and of the MMA
// warp), whichever role gave up: for the last copy into each stage (earlier ones were waited
// for before a stage was filled again), and for the last commit, which covers those before.
// False after an abort: shared memory and TMEM may be used again, the sums are not to be.
// (The split kernel passes its count on in a register, the walk through shared memory:
// registers there are all taken, and 512x2560x9216 took 1.1 us more.)
template <int BN, bool SPLIT, class P>
__device__ __forceinline__ bool tile_drain(const P &p, TileShared &b, int warp, uint32_t issued)
{
    using L = TileLayout<BN>;
    if (*static_cast<volatile int *>(&b.abort_flag) == 0) return true;
    const uint32_t S = stages_of<BN, SPLIT>(p);
    if (warp == L::TMA_WARP)
        for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j)
            mbar_wait_bounded(&b.full[j % S], (j / S) & 1, kCopyWaitLimitNs);
    if (warp == L::MMA_WARP && issued > 0)
        mbar_wait_bounded(&b.done[(issued - 1) % S], ((issued - 1) / S) & 1, kCopyWaitLimitNs);
    __syncthreads();
    return false;
}

// silu_mul_e of two values, the products and FMAs packed.
__device__ __forceinline__ uint64_t silu_mul2(uint64_t g2, uint64_t u2)
{
    const float2 g = unpack2(g2);
    const uint64_t x = pack2(fminf(fmaxf(g.x, -kSiluRange), kSiluRange), fminf(fmaxf(g.y, -kSiluRange), kSiluRange));
    const uint64_t c = pack2(kSiluC, kSiluC);
    const uint64_t hi = mul2(x, pack2(-kLog2e, -kLog2e));
    const uint64_t rest = fma2(x, pack2(kLog2eRest, kLog2eRest), fma2(x, pack2(kLog2e, kLog2e), hi));
    const float2 h = unpack2(hi);
    uint64_t e = pack2(ex2_approx(h.x), ex2_approx(h.y));
    e = fma2(e, mul2(rest, pack2(-kLn2, -kLn2)), e);
    const float2 d = unpack2(fma2(e, c, c));
    return mul2(mul2(mul2(g2, c), pack2(rcp_approx(d.x), rcp_approx(d.y))), u2);
}

__device__ __forceinline__ float load_y(const void *p, int64_t at, int bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at]) : static_cast<const float *>(p)[at];
}

// ---------------------------------------------------------------------------
// one CTA per SM over all tiles
// ---------------------------------------------------------------------------
__device__ __forceinline__ void st_32B(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Read once, so past L1 (1500x3000x2560 with an f32 residual: 20.0 us, 5 more through L1).
__device__ __forceinline__ void ld_32B(const void *p, uint32_t (&v)[8])
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p)
                 : "memory");
}

// What becomes of a tile's sums: SiLU and codes; y of either type in whole 32-byte
// sectors; any y without and with a residual.  Each has a kernel of its own: in a common
// one the registers of one form's stores are taken from every form's main loop (98 us for
// 4096x2560x9216 with a residual, where the bf16 kernel takes 79).
enum class Out { UP, BF16, F32, ANY, ANY_ADD };

// 32 columns from c0 of this thread's row of y, 32 bytes (a whole sector) per store,
// the residual's loads of two pieces before their stores (all four f32 pieces at once cost
// 96 bytes of spills, and 1 us more at 1500x3000x2560); every row of
// y starts on 32 bytes and n is a multiple of those 8 or 16 columns.
template <Out OUT>
__device__ __forceinline__ void store_row(const TileArgs &p, const uint64_t (&acc)[16], int64_t row, int c0)
{
    constexpr int BYTES = OUT == Out::BF16 ? 2 : 4, PER = 32 / BYTES, G = 32 / PER;  // columns per 32 bytes, pieces
    const int64_t at = (row * p.n + c0) * BYTES;
    const uint8_t *res = static_cast<const uint8_t *>(p.residual) + at;
    uint8_t *y = static_cast<uint8_t *>(p.y) + at;
    const int groups = min(static_cast<int>(p.n - c0), 32) / PER;  // of this row, none or fewer at the edge
#pragma unroll
    for (int g0 = 0; g0 < G; g0 += 2) {
        uint32_t e[2][8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (p.residual && g0 + g < groups) {
                ld_32B(res + 32 * (g0 + g), e[g]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) e[g][j] = 0;
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (g0 + g >= groups) break;
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (OUT == Out::BF16) {
                    const float2 v = unpack2(acc[8 * g + j]);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x + __uint_as_float(e[g][j] << 16),
                                                                   v.y + __uint_as_float(e[g][j] & 0xffff0000u));
                    o[j] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    const float2 v = unpack2(acc[4 * (g0 + g) + j / 2]);
                    o[j] = __float_as_uint((j & 1 ? v.y : v.x) + __uint_as_float(e[g][j]));
                }
            }
            st_32B(y + 32 * (g0 + g), o);
        }
    }
}

// The same for any n and either type: eight columns of the warp's 32 rows at a time
// through its transpose buffer, so that eight lanes write neighbouring values.  Of a lane's
// eight rows four residuals are loaded ahead: 4096x2561x1024, bf16, takes 38 us, 34
// more with one, 10 more with two and 6 more with eight (1 KB of spills).
template <bool ADD>
__device__ __forceinline__ void store_any(const TileArgs &p, const uint64_t (&acc)[16], float *xp, int64_t r0, int64_t c0,
                                          int lane)
{
    constexpr int AHEAD = ADD ? 4 : 1;  // rows whose residual a lane has loaded before it stores the first
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = unpack2(acc[4 * g + j]);
            xp[lane * T_XP + 2 * j] = v.x;
            xp[lane * T_XP + 2 * j + 1] = v.y;
        }
        __syncwarp();
        const int64_t col = c0 + 8 * g + (lane & 7);
        if (col >= p.n) continue;
#pragma unroll 1
        for (int i0 = lane >> 3; i0 < 32; i0 += 4 * AHEAD) {
            const int rows = static_cast<int>(min(p.m - r0, int64_t(32))) - i0;
            if (rows <= 0) break;
            const int64_t at = (r0 + i0) * p.n + col;
            float e[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                e[i] = ADD && 4 * i < rows ? load_y(p.residual, at + 4 * i * p.n, p.y_bf16) : 0.0f;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (4 * i >= rows) break;
                const float v = xp[(i0 + 4 * i) * T_XP + (lane & 7)];
                const float o = ADD ? v + e[i] : v;
                if (p.y_bf16)
                    static_cast<__nv_bfloat16 *>(p.y)[at + 4 * i * p.n] = __float2bfloat16_rn(o);
                else
                    static_cast<float *>(p.y)[at + 4 * i * p.n] = o;
            }
        }
    }
}

template <int BN, Out OUT, class P>
__global__ void __launch_bounds__(TileLayout<BN>::THREADS, 1)
    tiles_e4m3_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const P p)
{
    using L = TileLayout<BN>;
    constexpr bool UP = OUT == Out::UP;
    constexpr int BO = UP ? 128 : BN;  // output columns per tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) TileShared b;
    __shared__ float top[2][4][TM];  // [tile parity][column group][row]
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    tile_setup<BN>(b, warp);
    pdl_trigger();
    pdl_wait();  // the activations come from the previous kernel

    const uint32_t tmem = __shfl_sync(0xffffffffu, b.tmem, 0);
    const uint64_t desc0 = umma_desc_sw128(smem_addr(smem));
    uint32_t it = 0, c = 0;
    bool ok = true;
    if (warp == L::TMA_WARP) {
        for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x)
            ok = tile_copies<BN, UP, false>(tx, tw, p, b, smem, (tile % p.m_tiles) * TM, (tile / p.m_tiles) * BO, 0,
                                            p.kb, it);
        b.issued[0] = it;
    } else if (warp == L::MMA_WARP) {
        for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x)
            ok = tile_mmas<BN, false>(p, b, tmem, desc0, p.kb, it);
        b.issued[1] = it;
    } else if (warp == L::SCALE_WARP) {
        for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x)
            ok = tile_scales<BN, UP>(p, b, lane, (tile % p.m_tiles) * TM, (tile / p.m_tiles) * BO, 0, p.kb, c);
    } else {
        const int q = warp & 3, cg = warp >> 2;
        float *xp = reinterpret_cast<float *>(smem + L::STAGES * L::STAGE) + warp * 32 * T_XP;
        uint32_t parity = 0;
        for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, parity ^= 1) {
            uint64_t acc[2][16];
            ok = ok && tile_sums<BN, UP, false>(p, b, tmem, q, cg, lane, tile / p.m_tiles * BO, 0, p.kb, it, c, acc);
            if (!ok) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = pack2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
            }
            const int m0 = tile % p.m_tiles * TM, n0 = tile / p.m_tiles * BO;
            const int64_t row = m0 + 32 * q + lane;
            if constexpr (UP) {
                // 32 values of h, in place of the gate's sums
                const int c0 = n0 + 32 * cg;
                const int cols = static_cast<int>(min(p.n - c0, int64_t(32)));  // 32, 16 or none
                float half[2] = {0.0f, 0.0f};  // the largest of each 16 columns
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    acc[0][j] = silu_mul2(acc[0][j], acc[1][j]);
                    const float2 h = unpack2(acc[0][j]);
                    half[j >> 3] = fmaxf(half[j >> 3], fmaxf(fabsf(h.x), fabsf(h.y)));
                }
                float a = fmaxf(cols > 0 ? half[0] : 0.0f, cols > 16 ? half[1] : 0.0f);
                top[parity][cg][32 * q + lane] = a;
                asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) a = fmaxf(a, top[parity][i][32 * q + lane]);
                a = e4m3_floor(a);
                const float f = __fdiv_rn(448.0f, a);
                if (row < p.m) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // 16 codes each
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 h0 = unpack2(acc[0][8 * i + 2 * j]), h1 = unpack2(acc[0][8 * i + 2 * j + 1]);
                            w[j] = e4m3_pack4(h0.x * f, h0.y * f, h1.x * f, h1.y * f);
                        }
                        if (16 * i < cols)
                            *reinterpret_cast<uint4 *>(p.hq + row * p.n + c0 + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (cg == 0)
                        p.hd[row * e4m3_blocks(p.n) + n0 / EB] = __fdiv_rn(a, 448.0f);
                }
            } else if constexpr (OUT != Out::ANY && OUT != Out::ANY_ADD) {
                if (row < p.m) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) store_row<OUT>(p, acc[i], row, n0 + half_col<UP>(cg, i));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) store_any<OUT == Out::ANY_ADD>(p, acc[i], xp, m0 + 32 * q, n0 + half_col<UP>(cg, i), lane);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tile_drain<BN, false>(p, b, warp, b.issued[warp == L::MMA_WARP]);  // before the CTA's shared memory and TMEM go away
    if (warp == L::MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::TMEM) : "memory");
    }
}

// ---------------------------------------------------------------------------
// one cluster per tile, its CTAs sharing k
// ---------------------------------------------------------------------------
__device__ __forceinline__ float4 ld_cluster_f32x4(const float *local, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

// Four neighbouring sums of the tile over the cluster's CTAs: every load first (one
// takes about 0.3 us), then the additions in rank order.
__device__ __forceinline__ float4 cluster_sum4(const float *at, int split)
{
    float4 e[T_SPLIT];
#pragma unroll
    for (int r = 0; r < T_SPLIT; ++r)
        if (r < split) e[r] = ld_cluster_f32x4(at, r);
    float4 v = e[0];
#pragma unroll
    for (int r = 1; r < T_SPLIT; ++r)
        if (r < split) v = make_float4(v.x + e[r].x, v.y + e[r].y, v.z + e[r].z, v.w + e[r].w);
    return v;
}

// Four neighbouring residual values from `at` on, column c of n; zeros past the row's
// end and where there is no residual.  whole: n is a multiple of four.
__device__ __forceinline__ float4 residual4(const TileArgs &p, int64_t at, int64_t c, bool whole)
{
    float4 e = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!p.residual) return e;
    if (whole)
        return p.y_bf16 ? Vec4<__nv_bfloat16>::widen(*reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.residual) + at))
                        : *reinterpret_cast<const float4 *>(static_cast<const float *>(p.residual) + at);
    e.x = load_y(p.residual, at, p.y_bf16);
    if (c + 1 < p.n) e.y = load_y(p.residual, at + 1, p.y_bf16);
    if (c + 2 < p.n) e.z = load_y(p.residual, at + 2, p.y_bf16);
    if (c + 3 < p.n) e.w = load_y(p.residual, at + 3, p.y_bf16);
    return e;
}

// NaN outputs, or NaN codes and the floor's scales, for a whole tile.
template <bool UP>
__device__ __forceinline__ void nan_tile(const TileArgs &p, int m0, int rows, int n0, int width)
{
    const int cols = static_cast<int>(min(p.n - n0, static_cast<int64_t>(width)));
    for (int i = threadIdx.x; i < rows * cols; i += blockDim.x) {
        const int64_t row = m0 + i / cols, at = row * p.n + n0 + i % cols;
        if constexpr (UP) {
            p.hq[at] = 0x7f;
            if (i % cols == 0) p.hd[row * e4m3_blocks(p.n) + n0 / EB] = __fdiv_rn(e4m3_floor(0.0f), 448.0f);
        } else if (p.y_bf16) {
            static_cast<__nv_bfloat16 *>(p.y)[at] = __ushort_as_bfloat16(0x7fff);
        } else {
            static_cast<float *>(p.y)[at] = __int_as_float(0x7fc00000);
        }
    }
}

template <int BN, bool UP, class P>
__global__ void __launch_bounds__(TileLayout<BN>::THREADS, TileLayout<BN>::SPLIT_CTAS)
    split_e4m3_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const P p)
{
    using L = TileLayout<BN>;
    constexpr int BO = UP ? 128 : BN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) TileShared b;
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int tile = blockIdx.x / p.split;
    const int m0 = tile % p.m_tiles * TM, n0 = tile / p.m_tiles * BO;
    const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * p.kb / p.split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.kb / p.split);
    tile_setup<BN>(b, warp);
    pdl_trigger();

    const int q = warp & 3, cg = warp >> 2;
    const uint32_t tmem = __shfl_sync(0xffffffffu, b.tmem, 0);
    const uint64_t desc0 = umma_desc_sw128(smem_addr(smem));
    uint32_t it = 0, c = 0;
    uint64_t acc[2][16];
    if (warp == L::TMA_WARP) {
        // (the first use of a stage waits for nothing: early weights' blocks are always copied)
        tile_copies<BN, UP, true>(tx, tw, p, b, smem, m0, n0, kb0, kb1, it);
    } else if (warp == L::MMA_WARP) {
        pdl_wait();
        tile_mmas<BN, true>(p, b, tmem, desc0, kb1 - kb0, it);
    } else if (warp == L::SCALE_WARP) {
        pdl_wait();
        tile_scales<BN, UP>(p, b, lane, m0, n0, kb0, kb1, c);
    } else {
        pdl_wait();
        tile_sums<BN, UP, true>(p, b, tmem, q, cg, lane, n0, kb0, kb1, it, c, acc);
    }
    tc_fence_before();
    __syncthreads();
    const bool whole = tile_drain<BN, true>(p, b, warp, it);  // copies landed, MMAs done: the stages are free
    if (warp == L::MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::TMEM) : "memory");
    }
    float *sums = reinterpret_cast<float *>(smem);  // [128][LD]
    const int rows = static_cast<int>(min(p.m - m0, static_cast<int64_t>(TM)));
    if (warp < L::EW && 32 * q + lane < rows) {
        float *r = sums + (32 * q + lane) * L::LD;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float2 v0 = unpack2(acc[i][j]), v1 = unpack2(acc[i][j + 1]);
                *reinterpret_cast<float4 *>(r + half_col<UP>(cg, i) + 2 * j) = make_float4(v0.x, v0.y, v1.x, v1.y);
            }
    }
    cluster_sync();

    // this CTA's share of the rows
    const int per = (rows + p.split - 1) / p.split;
    const int r_end = min(rows, (rank + 1) * per);
    if constexpr (UP) {
        // a warp per row: four columns of both halves per lane, the row's block of h in the warp
        for (int r = rank * per + warp; r < r_end; r += L::THREADS / 32) {
            const float4 g = cluster_sum4(sums + r * L::LD + 4 * lane, p.split);
            const float4 u = cluster_sum4(sums + r * L::LD + 128 + 4 * lane, p.split);
            const bool live = n0 + 4 * lane < p.n;
            float4 h = make_float4(silu_mul_e(g.x, u.x), silu_mul_e(g.y, u.y), silu_mul_e(g.z, u.z), silu_mul_e(g.w, u.w));
            const float a = e4m3_floor(warp_max_nonneg(live ? max_abs4(h) : 0.0f));
            const float f = __fdiv_rn(448.0f, a);
            const int64_t row = m0 + r;
            if (live)
                *reinterpret_cast<uint32_t *>(p.hq + row * p.n + n0 + 4 * lane) =
                    e4m3_pack4(h.x * f, h.y * f, h.z * f, h.w * f);
            if (lane == 0) p.hd[row * e4m3_blocks(p.n) + n0 / EB] = __fdiv_rn(a, 448.0f);
        }
    } else {
        constexpr int G = BN / 4;  // groups of four columns
        const int items = (r_end - rank * per) * G;
        const bool fours = (p.n & 3) == 0;
        for (int i = threadIdx.x; i < items; i += L::THREADS) {
            const int r = rank * per + i / G, c = 4 * (i % G);
            if (n0 + c >= p.n) continue;
            const int64_t at = static_cast<int64_t>(m0 + r) * p.n + n0 + c;
            const float4 e = residual4(p, at, n0 + c, fours);  // its load beside the sums' (100x2727x3600 f32: 9.3 us, 1.0 more behind them)
            const float4 s = cluster_sum4(sums + r * L::LD + c, p.split);
            const float4 o = p.residual ? make_float4(s.x + e.x, s.y + e.y, s.z + e.z, s.w + e.w) : s;
            if (fours) {
                if (p.y_bf16)
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.y) + at) = Vec4<__nv_bfloat16>::narrow(o);
                else
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + at) = o;
            } else {
                const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (n0 + c + j >= p.n) break;
                    if (p.y_bf16)
                        static_cast<__nv_bfloat16 *>(p.y)[at + j] = __float2bfloat16_rn(v[j]);
                    else
                        static_cast<float *>(p.y)[at + j] = v[j];
                }
            }
        }
    }
    cluster_sync();  // the others have read this CTA's sums, and written what they made of them
    if (!whole) nan_tile<UP>(p, m0, rows, n0, BO);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static cudaError_t e4m3_map(EncodeTiledFn enc, CUtensorMap *map, const uint8_t *base, int64_t rows, int64_t k, int box)
{
    const cuuint64_t dim[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(k)};
    const cuuint32_t size[2] = {EB, static_cast<cuuint32_t>(box)};
    const cuuint32_t estride[2] = {1, 1};
    if (enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dim, stride, size, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

// The operands' maps and the tile counts of BN-wide tiles.
template <int BN, bool UP>
static cudaError_t tile_maps(const uint8_t *w, int64_t w_rows, int64_t k, const uint8_t *x, TileArgs &p,
                             CUtensorMap &tx, CUtensorMap &tw)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    constexpr int BO = UP ? 128 : BN;
    p.box_m = static_cast<int>(p.m >= TM ? TM : (p.m + 7) / 8 * 8);
    const int64_t m_tiles = (p.m + TM - 1) / TM, tiles = m_tiles * ((p.n + BO - 1) / BO);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;  // an output of 2^45 values and more
    p.m_tiles = static_cast<int>(m_tiles);
    p.tiles = static_cast<int>(tiles);
    if (cudaError_t e = e4m3_map(enc, &tx, x, p.m, k, p.box_m); e != cudaSuccess) return e;
    return e4m3_map(enc, &tw, w, w_rows, k, UP ? 128 : BN);
}

template <int BN, Out OUT, class P>
static cudaError_t launch_tiles(const uint8_t *w, int64_t w_rows, int64_t k, const uint8_t *x, P p, cudaStream_t s)
{
    using L = TileLayout<BN>;
    constexpr bool UP = OUT == Out::UP;
    CUtensorMap tx, tw;
    if (cudaError_t e = tile_maps<BN, UP>(w, w_rows, k, x, p, tx, tw); e != cudaSuccess) return e;
    constexpr int bytes = OUT == Out::ANY || OUT == Out::ANY_ADD ? L::ANY_BYTES : L::BYTES;
    const auto kernel = tiles_e4m3_kernel<BN, OUT, P>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), bytes); e != cudaSuccess) return e;
    const int64_t grid = p.tiles < num_sms() ? p.tiles : num_sms();
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(L::THREADS), static_cast<size_t>(bytes), s, tx, tw, p);
}

template <int BN>
static cudaError_t launch_tiles_out(const uint8_t *w, int64_t n, int64_t k, const uint8_t *x, const TileArgs &p,
                                    cudaStream_t s)
{
    // every row of y (and of the residual) starts on 32 bytes
    const bool rows32 = n % (p.y_bf16 ? 16 : 8) == 0 && reinterpret_cast<uintptr_t>(p.y) % 32 == 0 &&
                        reinterpret_cast<uintptr_t>(p.residual) % 32 == 0;
    if (!rows32)
        return p.residual ? launch_tiles<BN, Out::ANY_ADD>(w, n, k, x, p, s) : launch_tiles<BN, Out::ANY>(w, n, k, x, p, s);
    return p.y_bf16 ? launch_tiles<BN, Out::BF16>(w, n, k, x, p, s) : launch_tiles<BN, Out::F32>(w, n, k, x, p, s);
}

template <int BN, bool UP, class P>
static cudaError_t launch_split(const uint8_t *w, int64_t w_rows, int64_t k, const uint8_t *x, P p, int split,
                                cudaStream_t s)
{
    using L = TileLayout<BN>;
    CUtensorMap tx, tw;
    p.split = split;
    if (cudaError_t e = tile_maps<BN, UP>(w, w_rows, k, x, p, tx, tw); e != cudaSuccess) return e;
    // Stages for the blocks that a CTA has, as far as they fit: two at least where it has
    // as many.  The MMA reads 128 rows of activations whatever the copies bring: room for
    // them behind the last stage (their sums are not looked at).
    p.stage = L::W + p.box_m * EB;
    const int blocks = (p.kb + split - 1) / split, pad = (TM - p.box_m) * EB;
    p.stages = std::min({blocks, T_STAGES, (L::SPLIT_ROOM - pad) / p.stage});
    const int rows = static_cast<int>(std::min<int64_t>(p.m, TM));
    const int bytes = std::max(p.stages * p.stage + pad, rows * L::LD * 4) + 1024;
    const auto kernel = split_e4m3_kernel<BN, UP, P>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), L::SPLIT_ROOM + 1024); e != cudaSuccess) return e;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(p.tiles * split)), dim3(L::THREADS),
                              static_cast<size_t>(bytes), s, static_cast<unsigned>(split), tx, tw, p);
}

// How many clusters of `split` CTAs the device holds at once (asked once per device).
// A cluster stays inside one processing cluster of the chip, of 18 to 20 SMs: 46
// clusters of 6 CTAs at two an SM, but 30 of 7.  A grid one cluster too large takes
// twice as long (17x2560x9216: 9.5 us with 6 a tile, 6 more with 7).
// The query is made for one CTA an SM, which is all that it counts for a kernel of
// this kind.
template <int BN, bool UP>
static int clusters_at_once(int split)
{
    using L = TileLayout<BN>;
    static std::mutex mu;
    static int cache[64][T_SPLIT + 1] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int &n = cache[dev][split];
    if (n == 0) {
        cudaLaunchAttribute attr = {};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim = {static_cast<unsigned>(split), 1, 1};
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(split);
        cfg.blockDim = dim3(L::THREADS);
        cfg.dynamicSmemBytes = L::SPLIT_ROOM + 1024;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int one = 0;
        const auto kernel = split_e4m3_kernel<BN, UP, TileArgs>;
        if (opt_in_smem(reinterpret_cast<const void *>(kernel), L::SPLIT_ROOM + 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&one, kernel, &cfg) != cudaSuccess || one <= 0) {
            cudaGetLastError();
            one = 1;
        }
        n = one * L::SPLIT_CTAS;
    }
    return n;
}

// CTAs per tile: the most that find room at once with four blocks of k each, below
// which the cluster's own cost is no longer earned (gate|up 16x3584x1024: 5.6 us with
// 2 CTAs of 4 blocks, 0.7 more with 5 CTAs).
template <int BN, bool UP>
static int split_of(int64_t tiles, int64_t kb)
{
    for (int split = T_SPLIT; split > 1; --split)
        if (4 * split <= kb && tiles <= clusters_at_once<BN, UP>(split)) return split;
    return 1;
}

static TileArgs product_args(const float *wd, int64_t n, int64_t k, const float *xd, int64_t m, const void *residual,
                             void *y, int y_dtype)
{
    TileArgs p = {};
    p.wd = wd;
    p.xd = xd;
    p.m = m;
    p.n = n;
    p.kb = static_cast<int>(e4m3_blocks(k));
    p.residual = residual;
    p.y = y;
    p.y_bf16 = y_dtype == QG_BF16;
    return p;
}

static TileArgs up_args(const float *wd, int64_t ffn, int64_t k, const float *xd, int64_t m, uint8_t *hq, float *hd)
{
    TileArgs p = {};
    p.wd = wd;
    p.xd = xd;
    p.m = m;
    p.n = ffn;
    p.up_row = ffn;
    p.up_block = e4m3_blocks(ffn);
    p.kb = static_cast<int>(e4m3_blocks(k));
    p.hq = hq;
    p.hd = hd;
    return p;
}

static int product_split(const TileArgs &p) { return split_of<64, false>((p.m + TM - 1) / TM * ((p.n + 63) / 64), p.kb); }
static int up_split(const TileArgs &p) { return split_of<256, true>((p.m + TM - 1) / TM * e4m3_blocks(p.n), p.kb); }

cudaError_t launch_tiles_e4m3(const uint8_t *w, const float *wd, int64_t n, int64_t k, const uint8_t *x,
                              const float *xd, int64_t m, const void *residual, void *y, int y_dtype, cudaStream_t s)
{
    const TileArgs p = product_args(wd, n, k, xd, m, residual, y, y_dtype);
    const int64_t sms = num_sms(), mt = (m + TM - 1) / TM;
    // Too few tiles for the SMs: 64 columns wide, and a cluster to each.  Where a cluster of
    // two does not find room the walk over wider tiles is as fast or faster (512x2560x9216:
    // 22.8 us, 7.5 more with one CTA to each tile of 64).
    if (const int split = product_split(p); split > 1) return launch_split<64, false>(w, n, k, x, p, split, s);
    // the tile width whose busiest SM covers the fewest columns
    int best = 256;
    int64_t cost = INT64_MAX;
    for (int bn : {256, 192, 128}) {
        const int64_t c = (mt * ((n + bn - 1) / bn) + sms - 1) / sms * bn;
        if (c < cost) cost = c, best = bn;
    }
    if (best == 256) return launch_tiles_out<256>(w, n, k, x, p, s);
    if (best == 192) return launch_tiles_out<192>(w, n, k, x, p, s);
    return launch_tiles_out<128>(w, n, k, x, p, s);
}

cudaError_t launch_tiles_up_e4m3(const uint8_t *w, const float *wd, int64_t ffn, int64_t k, const uint8_t *x,
                                 const float *xd, int64_t m, uint8_t *hq, float *hd, cudaStream_t s)
{
    const TileArgs p = up_args(wd, ffn, k, xd, m, hq, hd);
    if (const int split = up_split(p); split > 1) return launch_split<256, true>(w, 2 * ffn, k, x, p, split, s);
    return launch_tiles<256, Out::UP>(w, 2 * ffn, k, x, p, s);
}

cudaError_t launch_stalled_e4m3(const uint8_t *w, const float *wd, int64_t n, int64_t k, const uint8_t *x, const float *xd,
                                int64_t m, void *out, float *out_d, int64_t cta, int64_t block, cudaStream_t s)
{
    StalledArgs p = {};
    if (out_d) {
        static_cast<TileArgs &>(p) = up_args(wd, n, k, xd, m, static_cast<uint8_t *>(out), out_d);
        p.cta = cta, p.block = block;
        if (const int split = up_split(p); split > 1) return launch_split<256, true>(w, 2 * n, k, x, p, split, s);
        return launch_tiles<256, Out::UP>(w, 2 * n, k, x, p, s);
    }
    static_cast<TileArgs &>(p) = product_args(wd, n, k, xd, m, nullptr, out, QG_F32);
    p.cta = cta, p.block = block;
    if (const int split = product_split(p); split > 1) return launch_split<64, false>(w, n, k, x, p, split, s);
    return launch_tiles<128, Out::ANY>(w, n, k, x, p, s);
}

}  // namespace qg
