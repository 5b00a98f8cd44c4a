// Attention of one new token per sequence over the paged, block-quantized cache.
//
//   o = sum_t p_t V_t / sum_t p_t,  p_t = e^(scale q . K_t),  one pass with a running maximum
//
// The cache is read once, whatever the number of query heads that share a cache head (up
// to 16), so HBM bounds it: 2 (D + D/16) bytes a token and head (Q8_0).  What has to
// fit under that bound is the work on each byte - its code made a binary16 operand, two
// matrix products, the softmax - so both products run on mma.sync m16n8k16 with the codes
// as exact f16 integers (or e4m3 values), scales applied outside in f32:
//
//   S = Q K^T   16 rows x 8 tokens.  q's row, scaled by a power of two, is split into two
//               f16 parts (22 bits); rows 0-7 of the tile are eight heads' high parts, rows
//               8-15 their low parts, so the split costs no instruction.  Per block of a
//               scale the sums are exact up to the tensor core's additions, then
//               s += d_K * (high + low).
//   O^T = V^T P^T   16 dims x 8 heads.  S's accumulators are P^T's operand as they lie in
//               the registers.  V's scale belongs to the summed index, so it goes into the
//               weight: p_t d_V,t.  The running maximum is taken over s_t + log2 d_V,t, less
//               14: the largest weight is about 2^14 whatever the scales are, and f16
//               holds 11 bits of every weight down to 2^-28 of it.  For f32 outputs the weight
//               is split into two f16 parts like q; for bf16 outputs its one rounding (2^-11,
//               of either sign from token to token) is under the output's own (2^-8).
//
// A warp takes TOK tokens a step and copies its own steps to shared memory by cp.async,
// STAGES - 1 of them ahead: no barrier, nothing shared between warps.  The rows there are
// padded so that a step's fragment loads (8 bytes of eight tokens' keys, 4 bytes of values
// of four tokens at a time) touch every bank once.
//
// Work is split evenly whatever the lengths are: the units (a step of each of the CTA's
// warps) of all sequences and heads lie in one line, and each CTA takes a stretch of it.
// A CTA finds its place by a scan over the lengths.  A head that lies inside one stretch
// is finished there; the parts of the others go to the workspace, and the CTA that brings
// the last of them (a counter per head that starts in a CTA) joins them in order.
#pragma once

#include <cfloat>

#include "qg_kv.cuh"

namespace qg {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = 32 * AT_WARPS;
constexpr int AT_CTAS_MAX = 4;  // per SM

struct AttnArgs {
    KvPlanes c;
    const void *q;
    int64_t q_row, q_head;
    int q_bf16, group, q_heads, chunks;  // chunks: of 8 NT query heads to a cache head
    int page_shift;                      // log2 of the page size, or -1
    int64_t batch;
    const int32_t *pages, *lengths;
    int64_t max_pages, window;
    float scale;
    void *out;
    int out_bf16;
    float *lse;
    int *counters;   // one per CTA, zero between calls
    float *records;  // two per CTA
};

template <bool E4M3, int D, int NT>
struct AttnShape {
    static constexpr int NB = kv_blocks(E4M3, D);
    static constexpr int SB = E4M3 ? 4 : 2;  // bytes of a scale
    static constexpr int CH = D <= 128 ? 2 : 1;                        // tiles of 16 tokens to a step
    static constexpr int TOK = KV_TILE * CH;
    static constexpr int STAGES = D <= 128 ? 2 : 3;
    static constexpr int KS = D % 64 == 32 ? D : D + 32;  // padded rows of keys: 32 or 96 bytes past a multiple of 128
    static constexpr int VS = D + 16;                     // and of values: 16 bytes past a multiple of 32
    static constexpr int SCALES = KV_TILE * NB * SB;      // bytes of a tile's scales
    static constexpr int TILE = KV_TILE * (KS + VS) + 2 * SCALES;
    static constexpr int STAGE = CH * TILE;
    static constexpr int HEADS = 8 * NT;
    static constexpr int OROW = D + 4;  // floats of a head's row when warps meet
    static constexpr int RING = AT_WARPS * STAGES * STAGE;
    static constexpr int QF = HEADS * D * 4;  // bytes of q's fragments
    static constexpr int MEET = AT_WARPS * HEADS * OROW * 4;
    static constexpr int SMEM = RING + QF + MEET + AT_WARPS * HEADS * 8 + HEADS * 4;
    static constexpr int CTAS = 227 * 1024 / (SMEM + 1024) < AT_CTAS_MAX ? 227 * 1024 / (SMEM + 1024) : AT_CTAS_MAX;
    static constexpr int RECORD = HEADS * (D + 2);  // floats
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two codes, in bytes 0 and 1 of w (HI: 2 and 3), as an f16 pair.  Q8_0: w holds code + 128,
// which placed in the mantissa of 1024 gives 1152 + code; exact.
template <bool E4M3, bool HI>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w)
{
    if constexpr (E4M3) {
        uint32_t r;
        const uint16_t h = static_cast<uint16_t>(HI ? w >> 16 : w);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
        return r;
    } else {
        const uint32_t m = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&m), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <bool E4M3>
__device__ __forceinline__ uint32_t code_bits(uint32_t w)
{
    return E4M3 ? w : w ^ 0x80808080u;
}

// The NB scales of two neighbouring tokens at p (4-byte aligned at least), as f32: [token][block].
template <bool E4M3, int NB>
__device__ __forceinline__ void two_scales(const uint8_t *p, float (&d)[2][NB])
{
    constexpr int WORDS = E4M3 ? 2 * NB : NB;
    uint32_t w[WORDS];
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else if constexpr (WORDS % 2 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS / 2; ++i) {
            const uint2 v = reinterpret_cast<const uint2 *>(p)[i];
            w[2 * i] = v.x, w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
        if constexpr (E4M3) {
            d[i / NB][i % NB] = __uint_as_float(w[i]);
        } else {
            d[i / NB][i % NB] = h2f(static_cast<uint16_t>(i % 2 ? w[i / 2] >> 16 : w[i / 2]));
        }
    }
}

__device__ __forceinline__ void cp_async_16_if(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One sequence's tokens in steps of TOK: the first and the end of what it sees.
struct Seen {
    int first, n;
};
__device__ __forceinline__ Seen seen_of(const AttnArgs &a, int64_t b)
{
    const int64_t held = a.max_pages * a.c.page;  // < 2^31
    const int n = static_cast<int>(min(static_cast<int64_t>(max(a.lengths[b], 0)), held));
    return {a.window > 0 && a.window < n ? n - static_cast<int>(a.window) : 0, n};
}

template <bool E4M3, int D, int NT, bool SPLIT>
struct Attn {
    using S = AttnShape<E4M3, D, NT>;
    static constexpr int NB = S::NB, CH = S::CH, TOK = S::TOK, DG = D / 32;

    static __device__ __forceinline__ int steps(Seen s) { return s.n > s.first ? (s.n + TOK - 1) / TOK - s.first / TOK : 0; }
    static __device__ __forceinline__ int units(Seen s) { return (steps(s) + AT_WARPS - 1) / AT_WARPS; }

    // A place in the line of units: sequence, item (a cache head and a chunk of its query heads), unit.
    struct Place {
        int64_t b, left;  // left: units of the CTA's stretch from here on
        Seen seen;
        int units, item, unit;
        __device__ __forceinline__ void next(const AttnArgs &a)
        {
            --left;
            if (++unit < units) return;
            unit = 0;
            next_item(a);
        }
        __device__ __forceinline__ void next_item(const AttnArgs &a)
        {
            if (++item < a.c.heads * a.chunks) return;
            item = 0;
            if (left <= 0) return;
            do {  // there is a further sequence with units while any of the stretch is left
                seen = seen_of(a, ++b);
                units = Attn::units(seen);
            } while (units == 0 && b + 1 < a.batch);
            if (units == 0) left = 0;
        }
    };

    // The tokens of this warp's step in a unit, [at, at + TOK), and their pages.
    struct Step {
        int at;
        bool any;
        int page[CH], off[CH];  // page number (loaded), first row in it
        __device__ __forceinline__ void find(const AttnArgs &a, const Place &p, int warp)
        {
            const int step = p.seen.first / TOK + p.unit * AT_WARPS + warp;
            at = step * TOK;
            any = p.left > 0 && step - p.seen.first / TOK < steps(p.seen);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int t = at + i * KV_TILE;
                const int col = a.page_shift >= 0 ? t >> a.page_shift : static_cast<int>(static_cast<uint32_t>(t) / static_cast<uint32_t>(a.c.page));
                off[i] = t - col * a.c.page;
                page[i] = any && t < p.seen.n && t + KV_TILE > p.seen.first ? a.pages[p.b * a.max_pages + col] : 0;
            }
        }
    };

    // Start the copies of a step into a stage.  Rows outside the tokens seen are zeros (their
    // codes may be NaN's); their scales come as they are and are passed over where they are
    // used.  Bit i of the answer: tile i lies on a page outside the cache (nothing is copied).
    static __device__ __forceinline__ uint32_t copy(const AttnArgs &a, const Place &p, const Step &s, uint32_t stage, int lane)
    {
        uint32_t bad = 0;
        const int h = a.chunks == 1 ? p.item : p.item / a.chunks;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int t = s.at + i * KV_TILE;
            if (t >= p.seen.n || t + KV_TILE <= p.seen.first) {
                // no token of it is seen: zeros, without a page to read from
                const uint32_t dst = stage + i * S::TILE;
                for (int x = lane; x < S::TILE / 16; x += 32)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst + x * 16), "r"(0) : "memory");
                continue;
            }
            if (s.page[i] < 0 || s.page[i] >= a.c.n_pages) {
                bad |= 1u << i;
                continue;
            }
            const int64_t row = (static_cast<int64_t>(s.page[i]) * a.c.heads + h) * a.c.page + s.off[i];
            const uint8_t *k = a.c.kq + row * D + lane * 16, *v = a.c.vq + row * D + lane * 16;
            const uint32_t dk = stage + i * S::TILE, dv = dk + KV_TILE * S::KS, ds = dv + KV_TILE * S::VS;
            const bool whole = t >= p.seen.first && t + KV_TILE <= p.seen.n;
            if (whole) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const int u = lane + 32 * j, r = u / (D / 16), c = u % (D / 16);
                    cp_async_16(dk + r * S::KS + c * 16, k + j * 512);
                    cp_async_16(dv + r * S::VS + c * 16, v + j * 512);
                }
            } else {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const int u = lane + 32 * j, r = u / (D / 16), c = u % (D / 16);
                    const bool there = t + r >= p.seen.first && t + r < p.seen.n;
                    cp_async_16_if(dk + r * S::KS + c * 16, k + j * 512, there);
                    cp_async_16_if(dv + r * S::VS + c * 16, v + j * 512, there);
                }
            }
            const int x = lane & 15;  // the tile's scales: keys' by lanes 0-15, values' by 16-31
            if (x < S::SCALES / 16) {
                const uint8_t *src = static_cast<const uint8_t *>(lane < 16 ? a.c.kd : a.c.vd) + row * NB * S::SB;
                cp_async_16(ds + (lane < 16 ? 0 : S::SCALES) + x * 16, src + x * 16);
            }
        }
        return bad;
    }

    float o[NT][2 * DG][4];  // O^T: tile of 16 dims, its accumulators
    float m[NT], l[NT];      // of head lane / 4 of each tile: the running reference, this lane's part of the sum

    __device__ __forceinline__ void reset()
    {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            m[i] = -FLT_MAX;
            l[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2 * DG; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
        }
    }

    // One step: `st` its stage, `qf` q's fragments, c the factor of each tile's scores (log2 units).
    __device__ __forceinline__ void step(const uint8_t *st, const uint4 *qf, const float (&c)[NT], int at, Seen seen,
                                         uint32_t bad, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        // ---- scores
        float s[NT][2 * CH][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j) s[i][j][0] = s[i][j][1] = 0.0f;
        float dk[2 * CH][2][NB];
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j)
            two_scales<E4M3, NB>(st + (j / 2) * S::TILE + KV_TILE * (S::KS + S::VS) + ((j % 2) * 8 + 2 * t) * NB * S::SB, dk[j]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float acc[NT][2 * CH][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
#pragma unroll
            for (int dg = b * (E4M3 ? 4 : 1); dg < (b + 1) * (E4M3 ? 4 : 1) && dg < DG; ++dg) {
                uint4 a[NT][2];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    a[i][0] = qf[((dg * 2 + 0) * NT + i) * 32 + lane];
                    a[i][1] = qf[((dg * 2 + 1) * NT + i) * 32 + lane];
                }
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(st + (j / 2) * S::TILE + ((j % 2) * 8 + g) * S::KS + dg * 32 + t * 8);
                    const uint32_t x = code_bits<E4M3>(w.x), y = code_bits<E4M3>(w.y);
                    const uint32_t b0 = codes_f16<E4M3, false>(x), b1 = codes_f16<E4M3, true>(x);
                    const uint32_t b2 = codes_f16<E4M3, false>(y), b3 = codes_f16<E4M3, true>(y);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        mma_f16(acc[i][j], a[i][0].x, a[i][0].y, a[i][0].z, a[i][0].w, b0, b1);
                        mma_f16(acc[i][j], a[i][1].x, a[i][1].y, a[i][1].z, a[i][1].w, b2, b3);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j) {
                    s[i][j][0] = fmaf(acc[i][j][0] + acc[i][j][2], dk[j][0][b], s[i][j][0]);
                    s[i][j][1] = fmaf(acc[i][j][1] + acc[i][j][3], dk[j][1][b], s[i][j][1]);
                }
        }
        // ---- values' scales, and what is not seen
        float dv[2 * CH][2][NB], e[2 * CH][2];
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j)
            two_scales<E4M3, NB>(st + (j / 2) * S::TILE + KV_TILE * (S::KS + S::VS) + S::SCALES + ((j % 2) * 8 + 2 * t) * NB * S::SB, dv[j]);
        const bool edge = at < seen.first || at + TOK > seen.n || bad != 0;
        uint32_t hidden = 0;  // bit 2 j + x: token x of pair j
        if (edge) {
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int token = at + j * 8 + 2 * t + x;
                    const bool h = token < seen.first || token >= seen.n;
                    if (h) {
                        hidden |= 1u << (2 * j + x);
#pragma unroll
                        for (int b = 0; b < NB; ++b) dv[j][x][b] = 0.0f;
                    } else if (bad >> (j / 2) & 1) {
#pragma unroll
                        for (int i = 0; i < NT; ++i) s[i][j][x] = __int_as_float(0x7fffffff);
                    }
                }
        }
        // log2 of a token's largest scale, held where the sum of weights stays in range and infinities and NaN
        // stay in their own blocks
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float top = E4M3 ? 0x1p-88f : 0x1p-25f;
#pragma unroll
                for (int b = 0; b < NB; ++b) top = fmaxf(top, fabsf(dv[j][x][b]));
                asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(e[j][x]) : "f"(fminf(top, E4M3 ? 0x1p119f : 65504.0f)));
            }
        // ---- weights
        float f[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float top = -__int_as_float(0x7f800000);
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float u = fmaf(s[i][j][x], c[i], e[j][x]);
                    top = fmaxf(top, edge && (hidden >> (2 * j + x) & 1) ? top : u);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float now = fmaxf(m[i], top - 14.0f);
            f[i] = ex2_approx(m[i] - now);
            m[i] = now;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float p = ex2_approx(fmaf(s[i][j][x], c[i], -now));
                    if (edge && (hidden >> (2 * j + x) & 1)) p = 0.0f;
                    s[i][j][x] = p;
                    sum += p;
                }
            l[i] = fmaf(l[i], f[i], sum);
        }
        // the factors of the heads whose columns of O^T this lane holds
        float f0[NT], f1[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            f0[i] = __shfl_sync(0xffffffffu, f[i], 8 * t);
            f1[i] = __shfl_sync(0xffffffffu, f[i], 8 * t + 4);
        }
        // ---- O^T = f O^T + V^T P^T, this step's part summed by itself
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t hi[NT][CH][2], lo[NT][CH][2];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j) {
                    const float w0 = s[i][j][0] * dv[j][0][b], w1 = s[i][j][1] * dv[j][1][b];
                    const uint32_t h = pack_f16(w0, w1);
                    hi[i][j / 2][j % 2] = h;
                    if constexpr (SPLIT) {
                        const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                        lo[i][j / 2][j % 2] = pack_f16(w0 - back.x, w1 - back.y);
                    }
                }
#pragma unroll
            for (int dg = b * (E4M3 ? 4 : 1); dg < (b + 1) * (E4M3 ? 4 : 1) && dg < DG; ++dg) {
                float acc[NT][2][4];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) acc[i][x][0] = acc[i][x][1] = acc[i][x][2] = acc[i][x][3] = 0.0f;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    const uint8_t *v = st + ch * S::TILE + KV_TILE * S::KS + (2 * t) * S::VS + dg * 32 + g * 4;
                    const uint32_t v0 = code_bits<E4M3>(*reinterpret_cast<const uint32_t *>(v));
                    const uint32_t v1 = code_bits<E4M3>(*reinterpret_cast<const uint32_t *>(v + S::VS));
                    const uint32_t v8 = code_bits<E4M3>(*reinterpret_cast<const uint32_t *>(v + 8 * S::VS));
                    const uint32_t v9 = code_bits<E4M3>(*reinterpret_cast<const uint32_t *>(v + 9 * S::VS));
                    const uint32_t x0 = __byte_perm(v0, v1, 0x5140), x1 = __byte_perm(v0, v1, 0x7362);
                    const uint32_t y0 = __byte_perm(v8, v9, 0x5140), y1 = __byte_perm(v8, v9, 0x7362);
                    const uint32_t a0 = codes_f16<E4M3, false>(x0), a1 = codes_f16<E4M3, true>(x0);
                    const uint32_t a2 = codes_f16<E4M3, false>(y0), a3 = codes_f16<E4M3, true>(y0);
                    const uint32_t a4 = codes_f16<E4M3, false>(x1), a5 = codes_f16<E4M3, true>(x1);
                    const uint32_t a6 = codes_f16<E4M3, false>(y1), a7 = codes_f16<E4M3, true>(y1);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        if constexpr (SPLIT) {
                            mma_f16(acc[i][0], a0, a1, a2, a3, lo[i][ch][0], lo[i][ch][1]);
                            mma_f16(acc[i][1], a4, a5, a6, a7, lo[i][ch][0], lo[i][ch][1]);
                        }
                        mma_f16(acc[i][0], a0, a1, a2, a3, hi[i][ch][0], hi[i][ch][1]);
                        mma_f16(acc[i][1], a4, a5, a6, a7, hi[i][ch][0], hi[i][ch][1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float(&d)[4] = o[i][2 * dg + x];
                        d[0] = fmaf(d[0], f0[i], acc[i][x][0]);
                        d[1] = fmaf(d[1], f1[i], acc[i][x][1]);
                        d[2] = fmaf(d[2], f0[i], acc[i][x][2]);
                        d[3] = fmaf(d[3], f1[i], acc[i][x][3]);
                    }
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v)
{
    *reinterpret_cast<typename Vec4<T>::raw *>(p) = Vec4<T>::narrow(v);
}

// Four outputs of a head, o / l.
__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t row, int dim, int col, float4 v, float l)
{
    const float4 r = make_float4(__fdiv_rn(v.x, l), __fdiv_rn(v.y, l), __fdiv_rn(v.z, l), __fdiv_rn(v.w, l));
    if (a.out_bf16)
        store4(static_cast<__nv_bfloat16 *>(a.out) + row * dim + col, r);
    else
        store4(static_cast<float *>(a.out) + row * dim + col, r);
}

template <bool E4M3, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(AT_THREADS, AttnShape<E4M3, D, NT>::CTAS) attn_decode_kernel(const __grid_constant__ AttnArgs a)
{
    using S = AttnShape<E4M3, D, NT>;
    using A = Attn<E4M3, D, NT, SPLIT>;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4 *const qf = reinterpret_cast<uint4 *>(smem + S::RING);
    float *const meet = reinterpret_cast<float *>(smem + S::RING + S::QF);
    float2 *const ml = reinterpret_cast<float2 *>(smem + S::RING + S::QF + S::MEET);  // [warp][head]: m, l
    float *const qc = reinterpret_cast<float *>(ml + AT_WARPS * S::HEADS);
    __shared__ int64_t sums[AT_WARPS];
    __shared__ int64_t place_at[2];  // sequence, units into it
    __shared__ int last_one;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, items = a.c.heads * a.chunks;
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's stretch of the line of units: a scan over the sequences, a slice to a thread
    const int64_t per = (a.batch + AT_THREADS - 1) / AT_THREADS;
    const int64_t b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    bool empty = false;  // a sequence without tokens whose outputs this CTA writes
    for (int64_t b = cta + static_cast<int64_t>(tid) * gridDim.x; b < a.batch; b += static_cast<int64_t>(AT_THREADS) * gridDim.x) {
        const Seen s = seen_of(a, b);
        empty |= s.n <= s.first;
    }
    int64_t mine = 0;
    for (int64_t b = b0; b < b1; ++b) mine += static_cast<int64_t>(A::units(seen_of(a, b))) * items;
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    const bool any_empty = __syncthreads_or(empty);
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) {
        if (w < warp) incl += sums[w];
        total += sums[w];
    }
    if (any_empty) {
        for (int64_t b = cta; b < a.batch; b += gridDim.x) {
            const Seen s = seen_of(a, b);
            if (s.n > s.first) continue;
            for (int i = tid; i < a.q_heads * (D / 4); i += AT_THREADS)
                attn_store(a, b * a.q_heads + i / (D / 4), D, i % (D / 4) * 4, make_float4(0, 0, 0, 0), 1.0f);
            if (a.lse)
                for (int i = tid; i < a.q_heads; i += AT_THREADS) a.lse[b * a.q_heads + i] = -__int_as_float(0x7f800000);
        }
    }
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
    if (cta >= ctas) return;
    const int64_t share = total / ctas, more = total - share * ctas;  // the first `more` CTAs take one unit more
    const int64_t start = cta * share + min(static_cast<int64_t>(cta), more), end = start + share + (cta < more);
    if (start >= incl - mine && start < incl) {
        int64_t at = incl - mine, b = b0;
        for (;; ++b) {
            const int64_t n = static_cast<int64_t>(A::units(seen_of(a, b))) * items;
            if (start < at + n) break;
            at += n;
        }
        place_at[0] = b;
        place_at[1] = start - at;
    }
    __syncthreads();
    typename A::Place use;
    use.b = place_at[0];
    use.seen = seen_of(a, use.b);
    use.units = A::units(use.seen);
    use.item = static_cast<int>(place_at[1] / use.units);
    use.unit = static_cast<int>(place_at[1] - static_cast<int64_t>(use.item) * use.units);
    use.left = end - start;

    // ---- the first copies
    const uint32_t ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;
    typename A::Place load = use;
    typename A::Step ahead;
    ahead.find(a, load, warp);
    uint32_t bad = 0;  // CH bits per stage
    auto copy_next = [&](int stage) {
        if (ahead.any) {
            const uint32_t x = A::copy(a, load, ahead, ring + stage * S::STAGE, lane);
            bad = (bad & ~(((1u << S::CH) - 1) << (stage * S::CH))) | x << (stage * S::CH);
        }
        cp_async_commit();
        if (load.left > 0) {
            load.next(a);
            ahead.find(a, load, warp);
        }
    };
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) copy_next(i);

    A state;
    int stage = 0, fill = S::STAGES - 1;
    while (use.left > 0) {
        // ---- a segment: the part of one item that lies in the stretch
        const int h = use.item / a.chunks, h0 = (use.item - h * a.chunks) * S::HEADS;  // cache head; its first query head here
        const int heads = min(S::HEADS, a.group - h0);
        const int unit0 = use.unit, n_units = static_cast<int>(min(static_cast<int64_t>(use.units - unit0), use.left));
        for (int x = warp; x < S::HEADS; x += AT_WARPS) {
            constexpr int P = (D / 4 + 31) / 32;
            float4 v[P];
            float top = 0.0f;
            bool odd = false;  // infinities or NaN in the row: no factor
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int p = lane + 32 * i;
                v[i] = make_float4(0, 0, 0, 0);
                if (x < heads && p < D / 4) {
                    const int64_t at = use.b * a.q_row + (h * a.group + h0 + x) * a.q_head + p * 4;
                    v[i] = a.q_bf16 ? Vec4<__nv_bfloat16>::widen(*reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + at))
                                    : *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at);
                }
                top = fmaxf(top, max_abs4(v[i]));
                odd |= !(fabsf(v[i].x) <= FLT_MAX && fabsf(v[i].y) <= FLT_MAX && fabsf(v[i].z) <= FLT_MAX && fabsf(v[i].w) <= FLT_MAX);
            }
            top = warp_max_nonneg(top);
            // 2^(14 - exponent of the largest), within f32's exponents either way
            int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            ex = top == 0.0f || __any_sync(0xffffffffu, odd) ? 14 : max(ex, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int p = lane + 32 * i;
                if (p < D / 4) {
                    const float4 w = make_float4(v[i].x * up, v[i].y * up, v[i].z * up, v[i].w * up);
                    uint4 r;
                    r.x = pack_f16(w.x, w.y);
                    r.z = pack_f16(w.z, w.w);
                    const float2 b01 = __half22float2(*reinterpret_cast<const __half2 *>(&r.x));
                    const float2 b23 = __half22float2(*reinterpret_cast<const __half2 *>(&r.z));
                    r.y = pack_f16(w.x - b01.x, w.y - b01.y);
                    r.w = pack_f16(w.z - b23.x, w.w - b23.y);
                    // piece p: dims 32 dg + 8 t + 4 k
                    const int dg = p >> 3, t = p >> 1 & 3, k = p & 1;
                    qf[((dg * 2 + k) * NT + x / 8) * 32 + (x % 8) * 4 + t] = r;
                }
            }
            if (lane == 0) qc[x] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(ex - 14 + 127) << 23);
        }
        __syncthreads();
        float c[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) c[i] = qc[8 * i + (lane >> 2)];
        state.reset();
        for (int u = 0; u < n_units; ++u) {
            copy_next(fill);
            cp_async_wait<S::STAGES - 1>();
            __syncwarp();
            const int step = use.seen.first / S::TOK + (unit0 + u) * AT_WARPS + warp, at = step * S::TOK;
            if (at < use.seen.n)
                state.step(smem + (warp * S::STAGES + stage) * S::STAGE, qf, c, at, use.seen,
                           bad >> (stage * S::CH) & ((1u << S::CH) - 1), lane);
            __syncwarp();
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
            fill = fill + 1 == S::STAGES ? 0 : fill + 1;
        }
        // ---- the warps meet
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float l = state.l[i];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if ((lane & 3) == 0) ml[warp * S::HEADS + 8 * i + (lane >> 2)] = make_float2(state.m[i], l);
            float *row = meet + (warp * S::HEADS + 8 * i + 2 * (lane & 3)) * S::OROW + (lane >> 2) * 4;
#pragma unroll
            for (int dg = 0; dg < D / 32; ++dg) {
                const float(&p)[4] = state.o[i][2 * dg], (&r)[4] = state.o[i][2 * dg + 1];
                *reinterpret_cast<float4 *>(row + dg * 32) = make_float4(p[0], p[2], r[0], r[2]);
                *reinterpret_cast<float4 *>(row + S::OROW + dg * 32) = make_float4(p[1], p[3], r[1], r[3]);
            }
        }
        __syncthreads();
        const bool whole = n_units == use.units;
        float *const record = a.records + (static_cast<int64_t>(cta) * 2 + (unit0 == 0)) * S::RECORD;
        const int64_t row0 = use.b * a.q_heads + h * a.group + h0;
        for (int i = tid; i < heads * (D / 4); i += AT_THREADS) {
            const int x = i / (D / 4), col = i % (D / 4) * 4;
            float top = -FLT_MAX, l = 0.0f;
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < AT_WARPS; ++w) top = fmaxf(top, ml[w * S::HEADS + x].x);
#pragma unroll
            for (int w = 0; w < AT_WARPS; ++w) {
                const float2 y = ml[w * S::HEADS + x];
                const float k = ex2_approx(y.x - top);
                const float4 z = *reinterpret_cast<const float4 *>(meet + (w * S::HEADS + x) * S::OROW + col);
                l = fmaf(y.y, k, l);
                v = make_float4(fmaf(z.x, k, v.x), fmaf(z.y, k, v.y), fmaf(z.z, k, v.z), fmaf(z.w, k, v.w));
            }
            if (whole) {
                attn_store(a, row0 + x, D, col, v, l);
                if (a.lse && col == 0) a.lse[row0 + x] = (top + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(record + x * D + col) = v;
                if (col == 0) record[S::HEADS * D + 2 * x] = top, record[S::HEADS * D + 2 * x + 1] = l;
            }
        }
        if (!whole) {
            // the item's units [g0, g1) of the line, and the CTAs that share them
            const int64_t g0 = end - use.left - unit0, g1 = g0 + use.units;
            auto cta_of = [&](int64_t u) {
                const int64_t cut = more * (share + 1);
                return static_cast<int>(u < cut ? u / (share + 1) : more + (u - cut) / share);
            };
            const int c0 = cta_of(g0), c1 = cta_of(g1 - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const bool is = atomicAdd(a.counters + c0, 1) == c1 - c0;
                if (is) a.counters[c0] = 0;  // for the next call
                last_one = is;
                __threadfence();
            }
            __syncthreads();
            if (last_one) {
                auto part = [&](int p) { return a.records + (static_cast<int64_t>(c0 + p) * 2 + (p == 0)) * S::RECORD; };
                const int parts = c1 - c0 + 1;
                for (int i = tid; i < heads * (D / 4); i += AT_THREADS) {
                    const int x = i / (D / 4), col = i % (D / 4) * 4;
                    float top = -FLT_MAX, l = 0.0f;
                    float4 v = make_float4(0, 0, 0, 0);
                    for (int p = 0; p < parts; ++p) top = fmaxf(top, __ldcg(part(p) + S::HEADS * D + 2 * x));
#pragma unroll 4
                    for (int p = 0; p < parts; ++p) {
                        const float2 y = __ldcg(reinterpret_cast<const float2 *>(part(p) + S::HEADS * D + 2 * x));
                        const float4 z = __ldcg(reinterpret_cast<const float4 *>(part(p) + x * D + col));
                        const float k = ex2_approx(y.x - top);
                        l = fmaf(y.y, k, l);
                        v = make_float4(fmaf(z.x, k, v.x), fmaf(z.y, k, v.y), fmaf(z.z, k, v.z), fmaf(z.w, k, v.w));
                    }
                    attn_store(a, row0 + x, D, col, v, l);
                    if (a.lse && col == 0) a.lse[row0 + x] = (top + log2f(l)) * kLn2;
                }
            }
        }
        // ---- on to the next item
        use.left -= n_units;
        if (use.left > 0) {
            use.unit = 0;
            use.next_item(a);
        }
    }
    cp_async_wait<0>();
}

template <bool E4M3, int D, int NT, bool SPLIT>
cudaError_t launch_attn_shape(const AttnArgs &a, int64_t most_units, cudaStream_t st)
{
    using S = AttnShape<E4M3, D, NT>;
    const auto kernel = attn_decode_kernel<E4M3, D, NT, SPLIT>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), S::SMEM); e != cudaSuccess) return e;
    const int64_t room = static_cast<int64_t>(num_sms()) * S::CTAS;
    const int grid = static_cast<int>(most_units < 1 ? 1 : most_units < room ? most_units : room);
    return launch_pdl(kernel, dim3(grid), dim3(AT_THREADS), S::SMEM, st, a);
}

// One translation unit per format and head size: definitions in qg_attn_*.cu.
template <bool E4M3, int D>
cudaError_t launch_attn_dim(const AttnArgs &a, int64_t most_units, cudaStream_t st);

#define QG_ATTN_DIM(E4M3, D)                                                                                       \
    template <>                                                                                                    \
    cudaError_t launch_attn_dim<E4M3, D>(const AttnArgs &a, int64_t most_units, cudaStream_t st)                   \
    {                                                                                                              \
        if (a.group <= 8)                                                                                          \
            return a.out_bf16 ? launch_attn_shape<E4M3, D, 1, false>(a, most_units, st)                            \
                              : launch_attn_shape<E4M3, D, 1, true>(a, most_units, st);                            \
        return a.out_bf16 ? launch_attn_shape<E4M3, D, 2, false>(a, most_units, st)                                \
                          : launch_attn_shape<E4M3, D, 2, true>(a, most_units, st);                                \
    }

}  // namespace qg
