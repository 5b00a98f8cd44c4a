// Attention of one new token per sequence over the paged, block-quantized cache.
//
//   o = sum_t p_t V_t / sum_t p_t,  p_t = e^(scale q . K_t),  one pass with a running maximum
//
// The cache is read once for the query heads that share a cache head, up to 16 of them (again for every 16 more: serving's
// cache with 16 query heads to a head 140 us, with 32 264), so HBM bounds it: 2 (D + D/16) bytes a token and head (Q8_0).  What has to
// fit under that bound is the work on each byte - its code made a binary16 operand, two
// matrix products, the softmax - so both products run on mma.sync m16n8k16 with the codes
// as exact f16 integers (or e4m3 values), scales applied outside in f32:
//
//   S = Q K^T   16 rows x 8 tokens.  q's row is scaled by a power of two and, where queries are f32
//               (FINE), split into two f16 parts (22 bits): rows 0-7 of the tile
//               are eight heads' high parts, rows 8-15 their low parts, so the split costs no
//               instruction.  bf16's 8 bits need one part; rows 8-15 are then eight heads more
//               or none.  Per block of a scale the sums are exact up to the tensor core's
//               additions, then s += d_K * (high + low).
//   O^T = V^T P^T   16 dims x 8 heads.  S's accumulators are P^T's operand as they lie in
//               the registers; ldmatrix turns the values' bytes round, four tokens of a
//               dim to a register.  V's scale belongs to the summed index, so it goes into the
//               weight: p_t d_V,t.  The running maximum is taken over s_t + log2 d_V,t, with the
//               largest of the token's scales, less 14: the largest weight is about 2^14 whatever the
//               scales are.  The weight is split into
//               two f16 parts like q (22 bits), whatever the outputs' type is: one part alone (11 bits, serving 97 us for 100)
//               moved 8 to 10 % of bf16 outputs by a step, two 0.1 %.  Each step's part is summed by itself and added in f32, which
//               the tensor core's own additions would not do to half a step.
//               The other blocks' weights are then as large as their scales are near to the token's largest.  Where
//               a token's scales lie more than 2^8 apart (AT_NEAR), from there to the item's end each step brings the weights of
//               each block to 2^14 by a power of two of their own and takes it off the sums.  Looking for such tokens, one to a
//               lane, and the branch cost 1 to 4 % (serving 100.4 us, 104.0 with them; e4m3 93.5, 93.7) and such items 15 to
//               35 % (a block 2^-12 of the others in every token: serving 120); without
//               them a block 2^-36 of its neighbour came out wrong by a half.
//
// A warp takes TOK tokens a step and copies its own steps to shared memory by cp.async, one step ahead: no barrier,
// nothing shared between warps.
//
// Three forms.  In the line (attn_decode_kernel) work is split evenly whatever the lengths are: the units (a step of each of
// the CTA's warps) of all sequences and heads lie in one line, each item - a cache head of a sequence and up to 16 of its
// query heads - behind COST places that stand for its beginning and end, and each CTA takes a stretch of it, which it
// finds by a scan over the lengths.  An item that lies inside one stretch is finished there; the parts of the others go to
// the workspace, and the CTA that brings the last of them (a counter per CTA in which an item begins) joins them in
// order.  Where an item has few units at most, as the page tables' width tells the host, the direct form
// (attn_direct_kernel) gives it a cluster, without scan, workspace and counter (one sequence of 700 tokens: 5.1 us, 7.2 in
// the line), and where there are many such items the warps' form (attn_warps_kernel) gives it a warp.
//
// What bounds it: HBM where there is much to read, issue for narrow heads, latency below some 50 MB: about 4 us to
// the first unit's end (length, pages, tokens, each a round trip to memory), 2 us from the last to the joined output.
// Measured, the share of the copy rate and the names that the comments below give the cases:
//   serving   64 sequences of up to 8192 tokens, 8 heads of 128, 64 query heads, bf16: Q8_0 104 us (83 %), e4m3 94 us (88 %)
//   document  one sequence of 131072 tokens, 8 heads of 128, 32 query heads, Q8_0, bf16: 54 us (79 %)
//   chats     256 sequences of up to 1000 tokens, 16 heads of 64, a query head each, Q8_0, bf16: 76 us (55 %; 0.6
//             instructions a cycle and scheduler, seven eighths of the MMAs' columns unused)
//   windows   32 sequences of up to 16384 tokens, the last 1024 of them, 4 heads of 256, 8 query heads, e4m3, f32: 19 us (52 %)
// Figures of a choice are of the day it was made: they compare its two sides.  Times in these files are of graph replays
// over operands that rotate.
#pragma once

#include <cfloat>

#include "qg_kv.cuh"

namespace qg {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = 32 * AT_WARPS;
constexpr int AT_CTAS_MAX = 4;  // per SM
constexpr int AT_FEW = 4;      // rows of 32 sequences that every warp scans for itself
constexpr int AT_CLUSTER = 8;  // CTAs to an item in the direct form, at most
// Between these scales the running maximum follows a token's largest (all of binary16's; e4m3's are f32).  Below the least
// weights reach 2^(14 + 25) of the softmax's: 2^30 tokens of them stay in range.  Above the most, 2^119.2 at the end,
// 2^30 tokens' sums of values stay in range as their p are under 2^-31.  2^70 between the two: where the maximum moves by so
// much, from a token without values to one of large ones, the factor 2^-70 of what came before is far from f32's end.
constexpr float AT_LEAST = 0x1p-25f;
template <bool E4M3>
constexpr float kAttnMost = E4M3 ? 0x1p45f : 65504.0f;
constexpr float AT_NEAR = 256.0f;  // a token's scales this near to one another share a reference for the weights' 16 bits
constexpr int AT_SHORT = 8;  // steps of an item in the warps' form, at most; twice as many where there are many items

struct AttnArgs {
    KvPlanes c;
    const void *q;
    int64_t q_row, q_head;
    int q_bf16, group, q_heads, chunks;  // chunks: of 8 NT query heads to a cache head
    int page_shift;                      // log2 of the page size, or -1
    int64_t batch;
    const int32_t *pages, *lengths;
    int64_t max_pages;
    int held, window;  // tokens that a page table holds; 0: no window
    float factor, most;  // scale log2(e) = factor 2^exponent; what a row's factor is held at, infinity where the scale is not finite
    int exponent;        // 0, or 2 where factor would leave f32
    void *out;
    int out_bf16;
    float *lse;
    int *counters;   // one per CTA, zero between calls
    float *records;  // two per CTA
    int cluster;     // direct form: CTAs to an item; 0: the line; -1: warps
    bool narrow;     // the line has fewer than 2^31 places
};

template <bool E4M3, int D, int NT>
struct AttnShape {
    static constexpr int NB = kv_blocks(E4M3, D);
    static constexpr int SB = E4M3 ? 4 : 2;      // bytes of a scale
    // Tiles of 16 tokens to a step.  128 values: two (serving 105 us, 108 with one); 256: one (30.7, 44 with two, whose
    // stages leave room for one CTA an SM).
    static constexpr int CH = D <= 128 ? 2 : 1;
    static constexpr int TOK = KV_TILE * CH;
    static constexpr int STAGES = 2;  // a third costs a CTA an SM (32 x 4000 tokens, 256 values: 31.8 us, 33.4 with three)
    static constexpr int SCALES = KV_TILE * NB * SB;      // bytes of a tile's scales
    static constexpr int CODES = KV_TILE * D;             // and of its keys' or values' codes
    static constexpr int TILE = 2 * CODES + 2 * SCALES;
    static constexpr int STAGE = CH * TILE;
    static constexpr int HEADS = 8 * NT;
    static constexpr int OROW = D + 4;  // floats of a head's row when warps meet
    static_assert(8 * OROW * 4 <= STAGE, "the warps' sums meet in the stages just read");
    static constexpr int RING = AT_WARPS * STAGES * STAGE;
    static constexpr int QF = HEADS * D * 4;  // bytes of q's fragments
    static constexpr int SMEM = RING + QF + AT_WARPS * HEADS * 8 + HEADS * 4;
    static constexpr int RECORD_AT = (SMEM + 15) / 16 * 16;  // direct form: the CTA's part behind it
    // CTAs an SM: four for 64 values (chats 78 us, 113 with two), three for 96 (48, 53 with four, whose 128 registers
    // spill), two for more (131072 tokens of 128: 55, 60 with three: the stretches get shorter, not the latencies).
    static constexpr int WANT = D <= 64 ? 4 : D <= 96 ? 3 : 2, FIT = 227 * 1024 / (SMEM + 1024);
    static constexpr int CTAS = FIT < WANT ? FIT : WANT;
    static_assert(CTAS >= 1 && CTAS <= AT_CTAS_MAX, "the workspace has counters for so many");
    static constexpr int RECORD = HEADS * (D + 2);  // floats
    // Records that are on their way at a time where an item's parts are joined: one sequence of 32768 tokens, 4 heads 18.8
    // us, 19.8 with 8, 17.9 with 24; 48 ragged sequences 35.2, 34.8, 36.0; the 128 registers of 64 values leave room for 8
    // (chats 69 us, 72 with 16).
    static constexpr int JOIN = D <= 64 ? 8 : 16;
    static constexpr int QUERY = (QF + HEADS * 4 + 15) / 16 * 16;  // warps' form: a warp's query
    static constexpr int SMEM_WARPS = RING + AT_WARPS * QUERY, FIT_WARPS = 227 * 1024 / (SMEM_WARPS + 1024);
    static constexpr int CTAS_WARPS = FIT_WARPS < WANT ? FIT_WARPS : WANT;
    // Of an item's beginning and end, in units: with 1, 2, 3 the serving batch takes 99.4, 97.7, 98.7 us, in e4m3 with 16
    // query heads to a head (48 of up to 6000) 37.4, 35.2, 35.0, windows 20.2, 19.3, 19.7.
    static constexpr int COST = 2;
    static constexpr int QW = HEADS / AT_WARPS, QP = (D / 4 + 31) / 32;  // heads of q to a warp, 4 values a lane each

    // A tile's keys and values in shared memory.  Fragments of keys are 32-byte pieces of four rows at a time, of values 16
    // bytes of eight rows (ldmatrix), which have to lie in banks of their own, and copies are fastest into whole lines of
    // 128 bytes: so rows are unpadded and the pieces of a line change places with the row.  Rows of 96 and 192 bytes are
    // two planes, of 64 and 32 and of 128 and 64 bytes to a row.
    static __host__ __device__ constexpr int plane(int piece) { return D == 96 ? (piece < 2 ? 64 : 32) : D == 192 ? (piece < 4 ? 128 : 64) : D; }
    static __host__ __device__ constexpr int plane_at(int piece) { return D == 96 && piece >= 2 ? KV_TILE * 64 : D == 192 && piece >= 4 ? KV_TILE * 128 : 0; }
    static __host__ __device__ constexpr int first_piece(int piece) { return D == 96 && piece >= 2 ? 2 : D == 192 && piece >= 4 ? 4 : 0; }
    // 32-byte piece of a row of keys.
    static __device__ __forceinline__ int key_piece(int r, int piece)
    {
        const int w = plane(piece), d = piece - first_piece(piece);
        return plane_at(piece) + r * w + ((w >= 128 ? d ^ (r & 3) : w == 64 ? d ^ (r >> 1 & 1) : d) << 5);
    }
    // 16-byte pieces, c, of token r: keys, and values, whose rows are in the order in which ldmatrix hands them to the
    // lanes: tokens 2 t, 2 t + 1, 2 t + 8 and 2 t + 9 are rows 4 t to 4 t + 3.
    static __device__ __forceinline__ int key_at(int r, int c) { return key_piece(r, c >> 1) + ((c & 1) << 4); }
    static __device__ __forceinline__ int value_row_at(int r, int c)
    {
        const int w = plane(c >> 1), d = c - 2 * first_piece(c >> 1);
        return plane_at(c >> 1) + r * w + ((w >= 128 ? d ^ (r & 7) : w == 64 ? d ^ (r >> 1 & 3) : d ^ (r >> 2 & 1)) << 4);
    }
    static __device__ __forceinline__ int value_at(int r, int c) { return value_row_at((r >> 1 & 3) * 4 + (r >> 3 & 1) * 2 + (r & 1), c); }
    static constexpr int NX = D >= 128 && D != 192 ? 4 : D / 32;  // pieces whose places differ by more than a constant
    static __host__ __device__ constexpr int piece_at(int piece) { return D == 256 ? piece / 4 * 128 : 0; }  // that constant
};

struct Quad {
    float v[4];
};
__device__ __forceinline__ Quad mma_f16(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, const Quad &c)
{
    Quad d;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%11,%12,%13};"
                 : "=f"(d.v[0]), "=f"(d.v[1]), "=f"(d.v[2]), "=f"(d.v[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c.v[0]), "f"(c.v[1]), "f"(c.v[2]), "f"(c.v[3]));
    return d;
}

// The same from zero.
__device__ __forceinline__ Quad mma_f16(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    Quad d;
    asm("{ .reg .f32 z; mov.f32 z, 0f00000000; mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {z,z,z,z}; }"
                 : "=f"(d.v[0]), "=f"(d.v[1]), "=f"(d.v[2]), "=f"(d.v[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    return d;
}

// Two codes, in bytes 0 and 1 of w (HI: 2 and 3), as an f16 pair.  Q8_0: w holds code + 128, which placed in the
// mantissa of 1024 gives 1152 + code; less 1152, the code.  All exact.  (Codes with the 1152 left on, which the sums then
// start without, took as long, and left a residue of it where codes are small.)
template <bool E4M3, bool HI>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w)
{
    if constexpr (E4M3) {
        uint32_t r;
        const uint16_t h = static_cast<uint16_t>(HI ? w >> 16 : w);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
        return r;
    } else {
        const uint32_t m = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140), k = 0x64806480u;
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&m), *reinterpret_cast<const __half2 *>(&k));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <bool E4M3>
__device__ __forceinline__ uint32_t code_bits(uint32_t w)
{
    return E4M3 ? w : w ^ 0x80808080u;
}

// The NB scales of two neighbouring tokens, [token][block], as they lie in memory (4-byte aligned at least).
template <bool E4M3, int NB>
struct PairScales {
    static constexpr int WORDS = E4M3 ? 2 * NB : NB;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const uint8_t *p)
    {
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
    }
    __device__ __forceinline__ float get(int token, int b) const  // both known at compile time
    {
        const int i = token * NB + b;
        if constexpr (E4M3) return __uint_as_float(w[i]);
        const __half2 h = *reinterpret_cast<const __half2 *>(&w[i / 2]);
        return i % 2 ? __high2float(h) : __low2float(h);
    }
};

// Whether a token's values' scales, as they lie in memory, are not all within AT_NEAR of one another and in the range that
// the running maximum follows; all zero is not either.
template <bool E4M3, int NB>
__device__ __forceinline__ bool scales_far(const uint8_t *p)
{
    if constexpr (E4M3) {
        const float *const d = reinterpret_cast<const float *>(p);
        const float a = fabsf(d[0]), b = fabsf(d[NB - 1]);
        return !(fminf(a, b) * AT_NEAR > fmaxf(fmaxf(a, b), AT_LEAST) && fmaxf(a, b) <= kAttnMost<E4M3>);
    } else {
        uint32_t w[(NB + 1) / 2];
        if constexpr (NB % 2) {  // 6 bytes, at even addresses
            const uint16_t *const h = reinterpret_cast<const uint16_t *>(p);
            w[0] = h[0] | static_cast<uint32_t>(h[1]) << 16, w[1] = h[2] | static_cast<uint32_t>(h[2]) << 16;
        } else if constexpr (NB == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (NB == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        }
        __half2 top = __habs2(*reinterpret_cast<const __half2 *>(&w[0])), low = top;  // NaN is passed over
#pragma unroll
        for (int i = 1; i < (NB + 1) / 2; ++i) {
            const __half2 h = __habs2(*reinterpret_cast<const __half2 *>(&w[i]));
            top = __hmax2(top, h), low = __hmin2(low, h);
        }
        return !(fminf(__low2float(low), __high2float(low)) * AT_NEAR > fmaxf(__low2float(top), __high2float(top)));
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

// What a pair rounded to f16 leaves of its two values, as an f16 pair.  (With the pair widened first: serving 100.9 us, 100.3 so.)
__device__ __forceinline__ uint32_t rest_f16(uint32_t rounded, float lo, float hi)
{
    float x, y;
    asm("{ .reg .b16 a, b, m; mov.b32 {a, b}, %2; mov.b16 m, 0xBC00; fma.rn.f32.f16 %0, a, m, %3; fma.rn.f32.f16 %1, b, m, %4; }"
        : "=f"(x), "=f"(y) : "r"(rounded), "f"(lo), "f"(hi));
    return pack_f16(x, y);
}

// One sequence's tokens in steps of TOK: the first and the end of what it sees.
struct Seen {
    int first, n;
};
__device__ __forceinline__ Seen seen_of(const AttnArgs &a, int64_t b)
{
    const int n = min(max(a.lengths[b], 0), a.held);
    return {a.window > 0 ? max(n - a.window, 0) : 0, n};
}

template <bool E4M3, int D, int NT, bool FINE>
struct Attn {
    using S = AttnShape<E4M3, D, NT>;
    static constexpr int NB = S::NB, CH = S::CH, TOK = S::TOK, DG = D / 32;

    static __device__ __forceinline__ int steps(Seen s) { return s.n > s.first ? (s.n + TOK - 1) / TOK - s.first / TOK : 0; }
    static __device__ __forceinline__ int units(Seen s) { return (steps(s) + AT_WARPS - 1) / AT_WARPS; }

    // A place in the line: sequence, item (a cache head and a chunk of its query heads), place in the item, whose first
    // COST places stand for what beginning and ending it costs and whose others are its units.
    struct Place {
        int b, left;  // left: places of the CTA's stretch from here on
        Seen seen;
        int units, item, at;
        __device__ __forceinline__ int unit() const { return at - S::COST; }
        __device__ __forceinline__ void settle()  // on to the item's units
        {
            if (at < S::COST) {
                const int skip = min(S::COST - at, left);
                at += skip;
                left -= skip;
            }
        }
        __device__ __forceinline__ void next_item(const AttnArgs &a)
        {
            at = 0;
            if (++item == a.c.heads * a.chunks) {
                item = 0;
                if (left <= 0) return;
                do {  // there is a further sequence with units while any of the stretch is left
                    seen = seen_of(a, ++b);
                    units = Attn::units(seen);
                } while (units == 0 && b + 1 < a.batch);
                if (units == 0) left = 0;
            }
            settle();
        }
    };

    // Start the copies of a step into a stage.  Rows outside the tokens seen are zeros (their codes may be NaN's); their
    // scales come as they are and are passed over where they are used.  Bit i of the answer: tile i has tokens seen on a
    // page outside the cache (nothing is copied).
    template <bool WHOLE>
    static __device__ __forceinline__ void copy_tile(const AttnArgs &a, Seen seen, int t, int64_t row, uint32_t dk, int lane)
    {
        const uint8_t *k = a.c.kq + row * D + lane * 16, *v = a.c.vq + row * D + lane * 16;
        const uint32_t dv = dk + S::CODES, ds = dv + S::CODES;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int u = lane + 32 * j, r = u / (D / 16), c = u % (D / 16);
            if constexpr (WHOLE) {
                cp_async_16(dk + S::key_at(r, c), k + j * 512);
                cp_async_16(dv + S::value_at(r, c), v + j * 512);
            } else {
                const bool there = t + r >= seen.first && t + r < seen.n;
                cp_async_16_if(dk + S::key_at(r, c), k + j * 512, there);
                cp_async_16_if(dv + S::value_at(r, c), v + j * 512, there);
            }
        }
        const int x = lane & 15;  // the tile's scales: keys' by lanes 0-15, values' by 16-31
        if (x < S::SCALES / 16) {
            const uint8_t *src = static_cast<const uint8_t *>(lane < 16 ? a.c.kd : a.c.vd) + row * (NB * S::SB);
            cp_async_16(ds + (lane < 16 ? 0 : S::SCALES) + x * 16, src + x * 16);
        }
    }
    // at: the step's first token; rows: of each tile the planes' row of its first token, kNone if none of it is seen, kBad
    // for a page outside the cache.
    static constexpr int64_t kNone = -1, kBad = -2;
    static __device__ __forceinline__ uint32_t copy(const AttnArgs &a, Seen seen, int at, const int64_t (&rows)[CH], uint32_t stage, int lane)
    {
        bool plain = at >= seen.first && at + TOK <= seen.n, none = true;
#pragma unroll
        for (int i = 0; i < CH; ++i) plain = plain && rows[i] >= 0, none = none && rows[i] == kNone;
        if (plain) {
#pragma unroll
            for (int i = 0; i < CH; ++i) copy_tile<true>(a, seen, 0, rows[i], stage + i * S::TILE, lane);
            return 0;
        }
        uint32_t bad = 0;
        if (none) return bad;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (rows[i] >= 0) {
                copy_tile<false>(a, seen, at + i * KV_TILE, rows[i], stage + i * S::TILE, lane);
            } else {  // zeros, without a page to read from
                if (rows[i] == kBad) bad |= 1u << i;
                for (int x = lane; x < S::TILE / 16; x += 32)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(stage + i * S::TILE + x * 16), "r"(0) : "memory");
            }
        }
        return bad;
    }

    // Tiles of S: rows 0-7 are eight heads; rows 8-15 the low parts of the same heads (FINE), or eight heads more.
    static constexpr int ST = FINE ? NT : 1;

    Quad o[NT][2 * DG];  // O^T: tiles of 16 dims, of which this lane has dims g and g + 8 of heads 2 t and 2 t + 1
    float m[NT], l[NT];  // of head lane / 4 of each tile: the running reference, this lane's part of the sum
    float c[NT];         // the factor of its scores, in log2 units
    bool far;            // a token of this item had scales far from one another

    __device__ __forceinline__ void begin(const float *qc, int lane)
    {
        far = false;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            m[i] = -FLT_MAX;
            l[i] = 0.0f;
            c[i] = qc[8 * i + (lane >> 2)];
#pragma unroll
            for (int j = 0; j < 2 * DG; ++j) o[i][j] = Quad{};
        }
    }

    // Tile i's eight heads to rows of OROW floats.
    __device__ __forceinline__ void put(int i, float *rows, int lane) const
    {
        float *const to = rows + 2 * (lane & 3) * S::OROW + (lane >> 2);
#pragma unroll
        for (int j = 0; j < 2 * DG; ++j) {
            const float(&p)[4] = o[i][j].v;
            to[j * 16] = p[0], to[j * 16 + 8] = p[2];
            to[S::OROW + j * 16] = p[1], to[S::OROW + j * 16 + 8] = p[3];
        }
    }

    // Query heads first, first + AT_WARPS, ... of a place's item: lane's pieces of four values.
    struct Query {
        uint4 v[S::QW][S::QP];  // as they lie in memory: bf16 in the first two words
        __device__ __forceinline__ void load(const AttnArgs &a, const Place &p, int first, int lane)
        {
            const int h = a.chunks == 1 ? p.item : p.item / a.chunks, h0 = (p.item - h * a.chunks) * S::HEADS;
            constexpr int size = FINE ? 4 : 2;
            const uint8_t *const row = static_cast<const uint8_t *>(a.q) + (p.b * a.q_row + (h * a.group + h0) * a.q_head) * size;
#pragma unroll
            for (int y = 0; y < S::QW; ++y)
#pragma unroll
                for (int i = 0; i < S::QP; ++i) {
                    const int x = y * AT_WARPS + first, piece = lane + 32 * i;
                    v[y][i] = make_uint4(0, 0, 0, 0);
                    if (h0 + x < a.group && piece < D / 4) {
                        const uint8_t *const at = row + (x * a.q_head + piece * 4) * size;
                        if constexpr (FINE) {
                            v[y][i] = *reinterpret_cast<const uint4 *>(at);
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2 *>(at);
                            v[y][i].x = w.x, v[y][i].y = w.y;
                        }
                    }
                }
        }
        __device__ __forceinline__ float4 get(int y, int i) const
        {
            const uint4 w = v[y][i];
            if constexpr (FINE) return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
            else return Vec4<__nv_bfloat16>::widen(make_uint2(w.x, w.y));
        }
    };

    // Piece p, dims 4 p to 4 p + 3 = 32 dg + 8 t + 4 k, of row x among q's fragments: high parts, low, high, low.
    static __device__ __forceinline__ void put_piece(uint4 *qf, int x, int p, uint4 r)
    {
        const int dg = p >> 3, t = p >> 1 & 3, k = p & 1;
        if constexpr (FINE || NT == 1) {
            if constexpr (!FINE) r.y = r.w = 0;
            qf[((dg * 2 + k) * NT + x / 8) * 32 + (x % 8) * 4 + t] = r;
        } else {  // rows 8-15: the second eight heads
            uint32_t *const at = reinterpret_cast<uint32_t *>(qf + (dg * 2 + k) * 32 + (x % 8) * 4 + t) + x / 8;
            at[0] = r.x, at[2] = r.z;
        }
    }

    // Their fragments and factors to shared memory.  Rows past the group's are zeros like any other: a
    // branch around them keeps a warp's rows from running beside one another (4 sequences of 16 tokens: 3.4 us, 4.0 with it).
    static __device__ __forceinline__ void put_query(const AttnArgs &a, const Query &query, uint4 *qf, float *qc, int first, int lane)
    {
#pragma unroll
        for (int y = 0; y < S::QW; ++y) {
            const int x = y * AT_WARPS + first;
            float4 v[S::QP];
#pragma unroll
            for (int i = 0; i < S::QP; ++i) v[i] = query.get(y, i);
            float top = 0.0f;
            bool odd = false;  // infinities or NaN in the row: no factor
#pragma unroll
            for (int i = 0; i < S::QP; ++i) {
                top = fmaxf(top, max_abs4(v[i]));
                odd |= !(fabsf(v[i].x) <= FLT_MAX && fabsf(v[i].y) <= FLT_MAX && fabsf(v[i].z) <= FLT_MAX && fabsf(v[i].w) <= FLT_MAX);
            }
            top = warp_max_nonneg(top);
            // 2^(14 - exponent of the largest), within f32's exponents either way
            int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            ex = top == 0.0f || __any_sync(0xffffffffu, odd) ? 14 : max(ex, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
#pragma unroll
            for (int i = 0; i < S::QP; ++i) {
                const int p = lane + 32 * i;
                const float4 w = make_float4(v[i].x * up, v[i].y * up, v[i].z * up, v[i].w * up);
                uint4 r;
                r.x = pack_f16(w.x, w.y);
                r.z = pack_f16(w.z, w.w);
                const float2 b01 = __half22float2(*reinterpret_cast<const __half2 *>(&r.x));
                const float2 b23 = __half22float2(*reinterpret_cast<const __half2 *>(&r.z));
                r.y = pack_f16(w.x - b01.x, w.y - b01.y);
                r.w = pack_f16(w.z - b23.x, w.w - b23.y);
                if (p < D / 4) put_piece(qf, x, p, r);
            }
            // finite where the scale is, so that scores of zero stay zero
            const float k = a.factor * __uint_as_float(static_cast<uint32_t>(ex - 14 + a.exponent + 127) << 23);
            if (lane == 0) qc[x] = k == k ? fminf(fmaxf(k, -a.most), a.most) : k;
        }
    }

    // Four tokens' codes of dims g, g + 8, g + 16 and g + 24 of 32.
    static __device__ __forceinline__ void values(uint32_t at, uint32_t (&r)[4])
    {
        asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    }

    // O^T = f O^T + V^T P^T, where s holds the tokens' p, vx where their values lie, early the first of them.  FAR: the weights
    // of each block of values are brought to 2^14 by a power of two of their own, so that f16 holds them wherever the block's
    // scales lie.
    template <bool FAR>
    __device__ __forceinline__ void add(const float (&s)[NT][2 * CH][2], const float (&dv)[2 * CH][2][NB], const float (&f0)[NT],
                                        const float (&f1)[NT], const uint32_t (&vx)[S::NX], const uint32_t (&early)[CH][4], int lane)
    {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t hi[NT][CH][2], lo[NT][CH][2];
            float down0[NT], down1[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float lift = 1.0f;
                if constexpr (FAR) {
                    float top = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2 * CH; ++j)
                        top = fmaxf(top, fmaxf(fabsf(s[i][j][0] * dv[j][0][b]), fabsf(s[i][j][1] * dv[j][1][b])));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int k = min(max(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), -110), 110);
                    lift = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                    down0[i] = __shfl_sync(0xffffffffu, down, 8 * (lane & 3));
                    down1[i] = __shfl_sync(0xffffffffu, down, 8 * (lane & 3) + 4);
                }
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j) {
                    float w0 = s[i][j][0] * dv[j][0][b], w1 = s[i][j][1] * dv[j][1][b];
                    if constexpr (FAR) w0 *= lift, w1 *= lift;
                    const uint32_t h = pack_f16(w0, w1);
                    hi[i][j / 2][j % 2] = h;
                    if constexpr (FAR)  // an infinite scale's weight has no second part
                        lo[i][j / 2][j % 2] = rest_f16(h, w0, w1) & (fabsf(w0) <= FLT_MAX ? 0xffffu : 0u) |
                                              rest_f16(h, w0, w1) & (fabsf(w1) <= FLT_MAX ? 0xffff0000u : 0u);
                    else
                        lo[i][j / 2][j % 2] = rest_f16(h, w0, w1);
                }
            }
#pragma unroll
            for (int dg = b * (E4M3 ? 4 : 1); dg < (b + 1) * (E4M3 ? 4 : 1) && dg < DG; ++dg) {
                Quad acc[NT][2];
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    uint32_t r[4];
                    if (dg == 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[i] = early[ch][i];
                    } else {
                        values(vx[dg % S::NX] + S::piece_at(dg) + ch * S::TILE, r);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = code_bits<E4M3>(r[i]);
                    const uint32_t va[2][4] = {{codes_f16<E4M3, false>(r[0]), codes_f16<E4M3, false>(r[1]),
                                                codes_f16<E4M3, true>(r[0]), codes_f16<E4M3, true>(r[1])},
                                               {codes_f16<E4M3, false>(r[2]), codes_f16<E4M3, false>(r[3]),
                                                codes_f16<E4M3, true>(r[2]), codes_f16<E4M3, true>(r[3])}};
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t(&q)[4] = va[x];
                            Quad &d = acc[i][x];
                            d = ch == 0 ? mma_f16(q[0], q[1], q[2], q[3], lo[i][ch][0], lo[i][ch][1])
                                        : mma_f16(q[0], q[1], q[2], q[3], lo[i][ch][0], lo[i][ch][1], d);
                            d = mma_f16(q[0], q[1], q[2], q[3], hi[i][ch][0], hi[i][ch][1], d);
                        }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float(&d)[4] = o[i][2 * dg + x].v;
                        if constexpr (FAR)
#pragma unroll
                            for (int y = 0; y < 4; ++y) acc[i][x].v[y] *= y % 2 ? down1[i] : down0[i];
                        d[0] = fmaf(d[0], f0[i], acc[i][x].v[0]);
                        d[1] = fmaf(d[1], f1[i], acc[i][x].v[1]);
                        d[2] = fmaf(d[2], f0[i], acc[i][x].v[2]);
                        d[3] = fmaf(d[3], f1[i], acc[i][x].v[3]);
                    }
            }
        }
    }

    // One step: `st` its stage, `qf` q's fragments.  EDGE: some of its tokens are not seen, or on a page outside the cache.
    template <bool EDGE>
    __device__ __forceinline__ void step(const uint8_t *st, const uint4 *qf, int at, Seen seen, uint32_t bad, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        const uint8_t *kx[S::NX];
        uint32_t vx[S::NX];
#pragma unroll
        for (int i = 0; i < S::NX; ++i) {
            kx[i] = st + S::key_piece(g, i) + t * 8;
            vx[i] = smem_addr(st) + S::CODES + S::value_row_at(lane & 15, 2 * i + (lane >> 4));
        }
        // ---- scores
        float s[NT][2 * CH][2];
        PairScales<E4M3, NB> dk[2 * CH];
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j)
            dk[j].load(st + (j / 2) * S::TILE + 2 * S::CODES + ((j % 2) * 8 + 2 * t) * NB * S::SB);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            Quad acc[ST][2 * CH];
#pragma unroll
            for (int dg = b * (E4M3 ? 4 : 1); dg < (b + 1) * (E4M3 ? 4 : 1) && dg < DG; ++dg) {
                const bool first = dg == b * (E4M3 ? 4 : 1);
                uint4 qa[ST][2];
#pragma unroll
                for (int i = 0; i < ST; ++i) {
                    qa[i][0] = qf[((dg * 2 + 0) * ST + i) * 32 + lane];
                    qa[i][1] = qf[((dg * 2 + 1) * ST + i) * 32 + lane];
                }
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(kx[dg % S::NX] + S::piece_at(dg) + (j / 2) * S::TILE + (j % 2) * 8 * S::plane(dg));
                    const uint32_t x = code_bits<E4M3>(w.x), y = code_bits<E4M3>(w.y);
                    const uint32_t b0 = codes_f16<E4M3, false>(x), b1 = codes_f16<E4M3, true>(x);
                    const uint32_t b2 = codes_f16<E4M3, false>(y), b3 = codes_f16<E4M3, true>(y);
#pragma unroll
                    for (int i = 0; i < ST; ++i) {
                        acc[i][j] = first ? mma_f16(qa[i][0].x, qa[i][0].y, qa[i][0].z, qa[i][0].w, b0, b1)
                                          : mma_f16(qa[i][0].x, qa[i][0].y, qa[i][0].z, qa[i][0].w, b0, b1, acc[i][j]);
                        acc[i][j] = mma_f16(qa[i][1].x, qa[i][1].y, qa[i][1].z, qa[i][1].w, b2, b3, acc[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float v = FINE ? acc[FINE ? i : 0][j].v[x] + acc[FINE ? i : 0][j].v[2 + x]
                                             : acc[0][j].v[2 * i + x];
                        s[i][j][x] = b == 0 ? v * dk[j].get(x, 0) : fmaf(v, dk[j].get(x, b), s[i][j][x]);
                    }
            }
        }
        // ---- a token to each lane: are its values' scales near one another?
        {
            const int token = lane % TOK;
            bool is = scales_far<E4M3, NB>(st + token / KV_TILE * S::TILE + 2 * S::CODES + S::SCALES + token % KV_TILE * NB * S::SB);
            if constexpr (EDGE) is = is && at + token >= seen.first && at + token < seen.n;
            far = __any_sync(0xffffffffu, is) || far;
        }
        // ---- values' scales, and what is not seen
        float dv[2 * CH][2][NB], e[2 * CH][2];
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j) {
            PairScales<E4M3, NB> d;
            d.load(st + (j / 2) * S::TILE + 2 * S::CODES + S::SCALES + ((j % 2) * 8 + 2 * t) * NB * S::SB);
#pragma unroll
            for (int b = 0; b < NB; ++b) dv[j][0][b] = d.get(0, b), dv[j][1][b] = d.get(1, b);
        }
        uint32_t hidden = 0;  // bit 2 j + x: token x of pair j
        if constexpr (EDGE) {
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int token = at + j * 8 + 2 * t + x;
                    if (token < seen.first || token >= seen.n) {
                        hidden |= 1u << (2 * j + x);
#pragma unroll
                        for (int b = 0; b < NB; ++b) dv[j][x][b] = 0.0f;
                    } else if (bad >> (j / 2) & 1) {
#pragma unroll
                        for (int i = 0; i < NT; ++i) s[i][j][x] = __int_as_float(0x7fffffff);
                    }
                }
        }
        // log2 of a token's largest scale, held where sums stay in range
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float top = AT_LEAST;
#pragma unroll
                for (int b = 0; b < NB; ++b) top = fmaxf(top, fabsf(dv[j][x][b]));
                asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(e[j][x]) : "f"(fminf(top, kAttnMost<E4M3>)));
            }
        uint32_t early[CH][4];  // before the branch, which would wait for them
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) values(vx[0] + ch * S::TILE, early[ch]);
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
                    if (!EDGE || !(hidden >> (2 * j + x) & 1)) top = fmaxf(top, u);
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
                    if (EDGE && (hidden >> (2 * j + x) & 1)) p = 0.0f;
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
        if (far)
            add<true>(s, dv, f0, f1, vx, early, lane);
        else
            add<false>(s, dv, f0, f1, vx, early, lane);
    }
};

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v)
{
    *reinterpret_cast<typename Vec4<T>::raw *>(p) = Vec4<T>::narrow(v);
}

// Four outputs of a head, o / l; by the correctly rounded reciprocal where they are rounded to bf16: within 1.5 * 2^-24 of
// the quotient, against the half step of 2^-8 that follows, and 142 sequences of 11 tokens with 168 query heads of 256 take
// 33 us, 58 with four divisions.
__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t row, int dim, int col, float4 v, float l)
{
    float4 r;
    if (a.out_bf16) {
        const float k = __frcp_rn(l);
        r = make_float4(v.x * k, v.y * k, v.z * k, v.w * k);
    } else {
        r = make_float4(__fdiv_rn(v.x, l), __fdiv_rn(v.y, l), __fdiv_rn(v.z, l), __fdiv_rn(v.w, l));
    }
    if (a.out_bf16)
        store4(static_cast<__nv_bfloat16 *>(a.out) + row * dim + col, r);
    else
        store4(static_cast<float *>(a.out) + row * dim + col, r);
}

// The line's `total` places in equal stretches, the first `more` of them one longer.
struct Share {
    int64_t each, more;
    int ctas;
    __device__ __forceinline__ Share(int64_t total, unsigned grid)
    {
        if (total < (int64_t(1) << 31)) {
            const uint32_t t = static_cast<uint32_t>(total), n = min(t, grid);
            ctas = static_cast<int>(n);
            each = n ? t / n : 0;
            more = n ? t % n : 0;
        } else {
            ctas = static_cast<int>(grid);
            each = total / grid;
            more = total - each * grid;
        }
    }
    __device__ __forceinline__ int64_t start(int c) const { return c * each + min(static_cast<int64_t>(c), more); }
    __device__ __forceinline__ int cta_of(int64_t at) const
    {
        const int64_t cut = more * (each + 1);
        if (cut + at < (int64_t(1) << 31) && each < (int64_t(1) << 30))
            return at < cut ? static_cast<uint32_t>(at) / static_cast<uint32_t>(each + 1)
                            : static_cast<int>(more) + static_cast<uint32_t>(at - cut) / static_cast<uint32_t>(each);
        return static_cast<int>(at < cut ? at / (each + 1) : more + (at - cut) / each);
    }
};

// Outputs of a sequence that sees nothing: query heads [first, first + heads).
template <int D, int THREADS = AT_THREADS>
__device__ __forceinline__ void attn_nothing(const AttnArgs &a, int64_t b, int first, int heads)
{
    const int64_t row = b * a.q_heads + first;
    for (int i = threadIdx.x % THREADS; i < heads * (D / 4); i += THREADS)
        attn_store(a, row + i / (D / 4), D, i % (D / 4) * 4, make_float4(0, 0, 0, 0), 1.0f);
    if (a.lse)
        for (int i = threadIdx.x % THREADS; i < heads; i += THREADS) a.lse[row + i] = -__int_as_float(0x7f800000);
}

__device__ __forceinline__ float2 ld_cluster_f2(const float *local, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(remote) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(const float *local, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(remote) : "memory");
    return v;
}

// What a warp copies ahead of its steps.  Page numbers are looked up for 32 tiles at a time, one to a lane, and turned
// into rows when the first of them is used.
template <bool E4M3, int D, int NT, bool FINE>
struct Feed {
    using S = AttnShape<E4M3, D, NT>;
    using A = Attn<E4M3, D, NT, FINE>;
    typename A::Place load;
    int64_t row;      // of this lane's tile
    uint32_t token;   // its first token
    int page, used;   // its page (0 where not looked up); tiles of the 32 that have been copied, -1 before the first
    uint32_t bad, ring;  // bad: CH bits per stage

    __device__ __forceinline__ void start(const typename A::Place &p, uint8_t *smem, int warp)
    {
        load = p;
        bad = 0;
        ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;
    }
    // The pages of this warp's tiles from p's unit on, units of W steps `stride` apart, of tokens in [first, end).
    template <int W>
    __device__ __forceinline__ void look_up(const AttnArgs &a, const typename A::Place &p, int first, int end, int stride, int warp, int lane)
    {
        const uint32_t step = static_cast<uint32_t>(first) / S::TOK + (p.unit() + lane / S::CH * stride) * W + warp;
        token = step * S::TOK + lane % S::CH * KV_TILE;
        page = 0;
        used = -1;
        if (token < static_cast<uint32_t>(end) && token + KV_TILE > static_cast<uint32_t>(first)) {
            const uint32_t col = a.page_shift >= 0 ? token >> a.page_shift : token / static_cast<uint32_t>(a.c.page);
            page = a.pages[p.b * a.max_pages + col];
        }
    }
    __device__ __forceinline__ void resolve(const AttnArgs &a)
    {
        used = 0;
        row = A::kNone;
        if (load.left > 0 && token < static_cast<uint32_t>(load.seen.n) && token + KV_TILE > static_cast<uint32_t>(load.seen.first)) {
            const int h = a.chunks == 1 ? load.item : load.item / a.chunks;
            const uint32_t off = a.page_shift >= 0 ? token & (a.c.page - 1) : token % static_cast<uint32_t>(a.c.page);
            row = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.n_pages)
                      ? (static_cast<int64_t>(page) * a.c.heads + h) * a.c.page + off : A::kBad;
        }
    }

    // The copies of the step ahead into a stage, and on to the one after it: the next unit of the stretch, or
    // (DIRECT) of the item, `stride` on.
    template <bool DIRECT, int W>
    __device__ __forceinline__ void next(const AttnArgs &a, int stage, int stride, int warp, int lane)
    {
        if (used < 0) resolve(a);
        if (load.left > 0) {
            int64_t rows[S::CH];
#pragma unroll
            for (int i = 0; i < S::CH; ++i) rows[i] = __shfl_sync(0xffffffffu, row, used + i);
            const int at = (static_cast<uint32_t>(load.seen.first) / S::TOK + load.unit() * W + warp) * S::TOK;
            const uint32_t x = A::copy(a, load.seen, at, rows, ring + stage * S::STAGE, lane);
            bad = (bad & ~(((1u << S::CH) - 1) << (stage * S::CH))) | x << (stage * S::CH);
            used += S::CH;
            bool look = used == 32;
            --load.left;
            if constexpr (DIRECT) {
                load.at += stride;
            } else if (++load.at == load.units + S::COST) {
                load.next_item(a);
                look = true;
            }
            if (look && load.left > 0) look_up<W>(a, load, load.seen.first, load.seen.n, stride, warp, lane);
        }
        cp_async_commit();
    }
};

// n_units units of W steps of an item, `stride` apart from unit0 on, after the copies of the first STAGES - 1 have begun.  Returns
// the stage that was read last.
template <bool DIRECT, int W, bool E4M3, int D, int NT, bool FINE>
__device__ __forceinline__ int attn_units(const AttnArgs &a, Attn<E4M3, D, NT, FINE> &state, Feed<E4M3, D, NT, FINE> &feed, Seen seen,
                                          int unit0, int n_units, int stride, int &stage, const uint8_t *ring, const uint4 *qf, int warp, int lane)
{
    using S = AttnShape<E4M3, D, NT>;
    int last = 0;
#pragma unroll 1
    for (int u = 0; u < n_units; ++u) {
        feed.template next<DIRECT, W>(a, stage == 0 ? S::STAGES - 1 : stage - 1, stride, warp, lane);
        cp_async_wait<S::STAGES - 1>();
        __syncwarp();
        const int step = static_cast<uint32_t>(seen.first) / S::TOK + (unit0 + u * stride) * W + warp, at = step * S::TOK;
        const uint8_t *const st = ring + stage * S::STAGE;
        const uint32_t off = feed.bad >> (stage * S::CH) & ((1u << S::CH) - 1);
        if (at < seen.n) {
            // one code for both where a CTA does a few steps and first has to fetch it (32 sequences of 64 tokens: 4.0 us, 4.7
            // with two; but 256 of 1000 in the line: 74, 69 with two)
            if (DIRECT || at < seen.first || at + S::TOK > seen.n || off != 0)
                state.template step<true>(st, qf, at, seen, off, lane);
            else
                state.template step<false>(st, qf, at, seen, 0, lane);
        }
        __syncwarp();
        last = stage;
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
    }
    return last;
}

// The warps meet, eight heads at a time, each in its stage `last`, into which no copy is under way.
// out(head, column, four sums, their reference, the sum of weights).
template <bool E4M3, int D, int NT, bool FINE, typename Out>
__device__ __forceinline__ void attn_meet(const Attn<E4M3, D, NT, FINE> &state, uint8_t *smem, int last, float2 *ml, int heads, const Out &out)
{
    using S = AttnShape<E4M3, D, NT>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *const meet = reinterpret_cast<float *>(smem + last * S::STAGE);
    constexpr int MEET = S::STAGES * S::STAGE / 4;  // floats from warp to warp
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (i > 0) __syncthreads();
        float l = state.l[i];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if ((lane & 3) == 0) ml[warp * S::HEADS + 8 * i + (lane >> 2)] = make_float2(state.m[i], l);
        state.put(i, meet + warp * MEET, lane);
        __syncthreads();
        for (int j = tid; j < min(heads - 8 * i, 8) * (D / 4); j += AT_THREADS) {
            const int y = j / (D / 4), x = 8 * i + y, col = j % (D / 4) * 4;
            float top = -FLT_MAX, sum = 0.0f;
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < AT_WARPS; ++w) top = fmaxf(top, ml[w * S::HEADS + x].x);
#pragma unroll
            for (int w = 0; w < AT_WARPS; ++w) {
                const float2 part = ml[w * S::HEADS + x];
                const float k = ex2_approx(part.x - top);
                const float4 z = *reinterpret_cast<const float4 *>(meet + w * MEET + y * S::OROW + col);
                sum = fmaf(part.y, k, sum);
                v = make_float4(fmaf(z.x, k, v.x), fmaf(z.y, k, v.y), fmaf(z.z, k, v.z), fmaf(z.w, k, v.w));
            }
            out(x, col, v, top, sum);
        }
    }
}

// Parts of an item joined in order, N of them on their way at a time.  part(p, y, z): part p's reference and sum
// of weights, and its four sums.
template <int N, typename Part>
__device__ __forceinline__ void attn_join(int parts, const Part &part, float4 &v, float &top, float &l)
{
    top = -FLT_MAX, l = 0.0f;
    v = make_float4(0, 0, 0, 0);
    for (int p0 = 0; p0 < parts; p0 += N) {
        float2 y[N];
        float4 z[N];
#pragma unroll
        for (int p = 0; p < N; ++p) {
            y[p] = make_float2(-FLT_MAX, 0.0f);
            z[p] = make_float4(0, 0, 0, 0);
            if (p0 + p < parts) part(p0 + p, y[p], z[p]);
        }
        float now = top;
#pragma unroll
        for (int p = 0; p < N; ++p) now = fmaxf(now, y[p].x);
        const float f = ex2_approx(top - now);
        top = now;
        l *= f;
        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const float k = ex2_approx(y[p].x - top);
            l = fmaf(y[p].y, k, l);
            v = make_float4(fmaf(z[p].x, k, v.x), fmaf(z[p].y, k, v.y), fmaf(z[p].z, k, v.z), fmaf(z[p].w, k, v.w));
        }
    }
}

__device__ __forceinline__ void attn_store_lse(const AttnArgs &a, int64_t row, int col, float top, float l)
{
    if (a.lse && col == 0) a.lse[row] = (top + log2f(l)) * kLn2;
}

template <bool E4M3, int D, int NT, bool FINE>
__global__ void __launch_bounds__(AT_THREADS, AttnShape<E4M3, D, NT>::CTAS) attn_decode_kernel(const __grid_constant__ AttnArgs a)
{
    using S = AttnShape<E4M3, D, NT>;
    using A = Attn<E4M3, D, NT, FINE>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint4 *const qf = reinterpret_cast<uint4 *>(smem + S::RING);
    float2 *const ml = reinterpret_cast<float2 *>(smem + S::RING + S::QF);  // [warp][head]: m, l
    float *const qc = reinterpret_cast<float *>(ml + AT_WARPS * S::HEADS);
    __shared__ int64_t sums[AT_WARPS];
    __shared__ int64_t found_at;
    __shared__ int found_b;
    __shared__ int last_one;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, items = a.c.heads * a.chunks;
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's stretch of the line, by a scan over the sequences
    typename A::Place use;
    int64_t total, start, end;
    bool any_empty;  // a sequence without tokens whose outputs this CTA writes
    if (a.narrow && a.batch <= 32 * AT_FEW) {  // every warp for itself, rows of 32 sequences: no barrier
        int incl[AT_FEW], base = 0;
        bool empty = false;
#pragma unroll
        for (int r = 0; r < AT_FEW; ++r) {
            const int b = r * 32 + lane;
            incl[r] = 0;
            if (r * 32 >= a.batch) continue;
            if (b < a.batch) {
                const int n = A::units(seen_of(a, b));
                incl[r] = n > 0 ? (n + S::COST) * items : 0;
                empty |= n == 0 && b % gridDim.x == cta;
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl[r], off);
                if (lane >= off) incl[r] += up;
            }
            incl[r] += base;
            base = __shfl_sync(0xffffffffu, incl[r], 31);
        }
        any_empty = __any_sync(0xffffffffu, empty);
        total = base;
        base = 0;
        const Share share(total, gridDim.x);
        start = share.start(cta), end = share.start(cta + 1);
        use.b = 0, use.at = static_cast<int>(start);
        bool found = cta >= share.ctas;
#pragma unroll
        for (int r = 0; r < AT_FEW; ++r) {
            if (found || r * 32 >= a.batch) continue;
            const uint32_t past = __ballot_sync(0xffffffffu, incl[r] > static_cast<int>(start));
            if (past) {
                const int at = __ffs(past) - 1;
                const int before = __shfl_sync(0xffffffffu, incl[r], at > 0 ? at - 1 : 0);
                use.b = r * 32 + at;
                use.at = static_cast<int>(start) - (at > 0 ? before : base);
                found = true;
            } else {
                base = __shfl_sync(0xffffffffu, incl[r], 31);
            }
        }
    } else {
        const int64_t per = (a.batch + AT_THREADS - 1) / AT_THREADS;
        const int64_t b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
        bool empty = false;
        int64_t mine = 0;
        for (int64_t b = b0; b < b1; ++b) {
            const int n = A::units(seen_of(a, b));
            mine += n > 0 ? static_cast<int64_t>(n + S::COST) * items : 0;
            empty |= n == 0 && b % gridDim.x == cta;
        }
        int64_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += up;
        }
        if (lane == 31) sums[warp] = incl;
        any_empty = __syncthreads_or(empty);
        total = 0;
#pragma unroll
        for (int w = 0; w < AT_WARPS; ++w) {
            if (w < warp) incl += sums[w];
            total += sums[w];
        }
        const Share share(total, gridDim.x);
        start = share.start(cta), end = share.start(cta + 1);
        if (cta < share.ctas && start >= incl - mine && start < incl) {
            int64_t at = incl - mine, b = b0;
            for (;; ++b) {
                const int n = A::units(seen_of(a, b));
                const int64_t cost = n > 0 ? static_cast<int64_t>(n + S::COST) * items : 0;
                if (start < at + cost || b + 1 == b1) break;
                at += cost;
            }
            found_b = static_cast<int>(b);
            found_at = start - at;
        }
        __syncthreads();
        use.b = found_b;
        use.at = 0;
    }
    if (any_empty) {
        for (int64_t b = cta; b < a.batch; b += gridDim.x) {
            const Seen s = seen_of(a, b);
            if (s.n <= s.first) attn_nothing<D>(a, b, 0, a.q_heads);
        }
    }
    const Share share(total, gridDim.x);
    if (cta >= share.ctas) return;
    use.seen = seen_of(a, use.b);
    use.units = A::units(use.seen);
    if (use.units == 0) return;  // the lengths have changed under the call
    if (a.narrow && a.batch <= 32 * AT_FEW) {
        use.item = static_cast<int>(static_cast<uint32_t>(use.at) / static_cast<uint32_t>(use.units + S::COST));
        use.at -= use.item * (use.units + S::COST);
    } else {
        use.item = static_cast<int>(found_at / (use.units + S::COST));
        use.at = static_cast<int>(found_at - static_cast<int64_t>(use.item) * (use.units + S::COST));
    }
    use.left = static_cast<int>(end - start);  // the host's bound on the line keeps it below 2^31
    use.settle();
    if (use.left <= 0) return;

    typename A::Query query;
    query.load(a, use, warp, lane);
    // ---- the first copies
    Feed<E4M3, D, NT, FINE> feed;
    feed.start(use, smem, warp);
    feed.template look_up<AT_WARPS>(a, use, use.seen.first, use.seen.n, 1, warp, lane);
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) feed.template next<false, AT_WARPS>(a, i, 1, warp, lane);

    A state;
    int stage = 0;
    while (use.left > 0) {
        // ---- a segment: the part of one item that lies in the stretch
        const int h = a.chunks == 1 ? use.item : use.item / a.chunks, h0 = (use.item - h * a.chunks) * S::HEADS;  // cache head; its first query head here
        const int heads = min(S::HEADS, a.group - h0);
        const int unit0 = use.unit(), n_units = min(use.units - unit0, use.left);
        A::put_query(a, query, qf, qc, warp, lane);
        __syncthreads();
        state.begin(qc, lane);
        const int last = attn_units<false, AT_WARPS>(a, state, feed, use.seen, unit0, n_units, 1, stage, smem + warp * S::STAGES * S::STAGE, qf, warp, lane);
        // ---- the warps meet: no copy into the stage read last is begun before the next segment's first barrier
        const bool whole = n_units == use.units;
        const int64_t first_unit = end - use.left - unit0;  // of the item, in the line
        const int units = use.units;
        float *const record = a.records + (static_cast<int64_t>(cta) * 2 + (unit0 == 0)) * S::RECORD;
        const int64_t row0 = static_cast<int64_t>(use.b) * a.q_heads + h * a.group + h0;
        use.left -= n_units;
        if (use.left > 0) {
            use.next_item(a);
            if (use.left > 0) query.load(a, use, warp, lane);  // the next segment's, on its way while this one ends
        }
        attn_meet(state, smem, last, ml, heads, [&](int x, int col, float4 v, float top, float sum) {
            if (whole) {
                attn_store(a, row0 + x, D, col, v, sum);
                attn_store_lse(a, row0 + x, col, top, sum);
            } else {
                *reinterpret_cast<float4 *>(record + x * D + col) = v;
                if (col == 0) *reinterpret_cast<float2 *>(record + S::HEADS * D + 2 * x) = make_float2(top, sum);
            }
        });
        if (!whole) {
            // the CTAs that share the item's units
            const int c0 = share.cta_of(first_unit), c1 = share.cta_of(first_unit + units - 1);
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
                const int parts = c1 - c0 + 1;
                for (int i = tid; i < heads * (D / 4); i += AT_THREADS) {
                    const int x = i / (D / 4), col = i % (D / 4) * 4;
                    float top, l;
                    float4 v;
                    attn_join<S::JOIN>(parts, [&](int p, float2 &y, float4 &z) {
                        const float *const from = a.records + (static_cast<int64_t>(c0 + p) * 2 + (p == 0)) * S::RECORD;
                        y = __ldcg(reinterpret_cast<const float2 *>(from + S::HEADS * D + 2 * x));
                        z = __ldcg(reinterpret_cast<const float4 *>(from + x * D + col));
                    }, v, top, l);
                    attn_store(a, row0 + x, D, col, v, l);
                    attn_store_lse(a, row0 + x, col, top, l);
                }
            }
        }
    }
    cp_async_wait<0>();
}

// The direct form, for few units to an item: a cluster of a.cluster CTAs to each item, whose CTAs take its units in turn
// and join their parts through distributed shared memory.  No scan, no workspace, no counter; the first page numbers
// are loaded beside the length.
template <bool E4M3, int D, int NT, bool FINE>
__global__ void __launch_bounds__(AT_THREADS, AttnShape<E4M3, D, NT>::CTAS) attn_direct_kernel(const __grid_constant__ AttnArgs a)
{
    using S = AttnShape<E4M3, D, NT>;
    using A = Attn<E4M3, D, NT, FINE>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint4 *const qf = reinterpret_cast<uint4 *>(smem + S::RING);
    float2 *const ml = reinterpret_cast<float2 *>(smem + S::RING + S::QF);  // [warp][head]: m, l
    float *const qc = reinterpret_cast<float *>(ml + AT_WARPS * S::HEADS);
    float *const record = reinterpret_cast<float *>(smem + S::RECORD_AT);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = a.cluster, rank = static_cast<int>(blockIdx.x) % ctas;  // clusters are runs of the grid
    const int items = a.c.heads * a.chunks, which = static_cast<int>(blockIdx.x) / ctas;
    typename A::Place use;
    use.b = which / items;
    use.item = which - use.b * items;
    use.at = S::COST + rank;
    pdl_wait();
    pdl_trigger();
    typename A::Query query;
    query.load(a, use, warp, lane);
    Feed<E4M3, D, NT, FINE> feed;
    if (a.window == 0) feed.template look_up<AT_WARPS>(a, use, 0, a.held, ctas, warp, lane);
    use.seen = seen_of(a, use.b);
    use.units = A::units(use.seen);
    use.left = use.units > rank ? (use.units - rank + ctas - 1) / ctas : 0;
    const int h = a.chunks == 1 ? use.item : use.item / a.chunks, h0 = (use.item - h * a.chunks) * S::HEADS;
    const int heads = min(S::HEADS, a.group - h0);
    if (use.units == 0) {
        if (rank == 0) attn_nothing<D>(a, use.b, h * a.group + h0, heads);
        return;  // the whole cluster
    }
    const int64_t row0 = static_cast<int64_t>(use.b) * a.q_heads + h * a.group + h0;
    const bool alone = use.units == 1 || ctas == 1;
    if (use.left > 0) {
        feed.start(use, smem, warp);
        if (a.window > 0) feed.template look_up<AT_WARPS>(a, use, use.seen.first, use.seen.n, ctas, warp, lane);
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) feed.template next<true, AT_WARPS>(a, i, ctas, warp, lane);
        A::put_query(a, query, qf, qc, warp, lane);
        __syncthreads();
        A state;
        state.begin(qc, lane);
        int stage = 0;
        const int last = attn_units<true, AT_WARPS>(a, state, feed, use.seen, rank, use.left, ctas, stage, smem + warp * S::STAGES * S::STAGE, qf, warp, lane);
        cp_async_wait<0>();
        attn_meet(state, smem, last, ml, heads, [&](int x, int col, float4 v, float top, float sum) {
            if (alone) {
                attn_store(a, row0 + x, D, col, v, sum);
                attn_store_lse(a, row0 + x, col, top, sum);
            } else {
                *reinterpret_cast<float4 *>(record + x * D + col) = v;
                if (col == 0) *reinterpret_cast<float2 *>(record + S::HEADS * D + 2 * x) = make_float2(top, sum);
            }
        });
    }
    if (alone) return;  // the whole cluster
    cluster_sync();
    const int parts = min(use.units, ctas), pieces = heads * (D / 4);
    for (int i = rank + ctas * tid; i < pieces; i += ctas * AT_THREADS) {
        const int x = i / (D / 4), col = i % (D / 4) * 4;
        float top, l;
        float4 v;
        attn_join<AT_CLUSTER>(parts, [&](int p, float2 &y, float4 &z) {
            y = ld_cluster_f2(record + S::HEADS * D + 2 * x, p);
            z = ld_cluster_f4(record + x * D + col, p);
        }, v, top, l);
        attn_store(a, row0 + x, D, col, v, l);
        attn_store_lse(a, row0 + x, col, top, l);
    }
    cluster_sync();  // no CTA leaves while another reads its part
}

// The warps' form, for many items of few steps: an item to each warp, which finishes it by itself.
template <bool E4M3, int D, int NT, bool FINE>
__global__ void __launch_bounds__(AT_THREADS, AttnShape<E4M3, D, NT>::CTAS_WARPS) attn_warps_kernel(const __grid_constant__ AttnArgs a)
{
    using S = AttnShape<E4M3, D, NT>;
    using A = Attn<E4M3, D, NT, FINE>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t *const ring = smem + warp * S::STAGES * S::STAGE;
    uint4 *const qf = reinterpret_cast<uint4 *>(smem + S::RING + warp * S::QUERY);
    float *const qc = reinterpret_cast<float *>(qf) + S::QF / 4;
    const int items = a.c.heads * a.chunks;
    const int64_t which = static_cast<int64_t>(blockIdx.x) * AT_WARPS + warp;
    pdl_wait();
    pdl_trigger();
    if (which >= a.batch * items) return;  // no barrier of the CTA's below
    typename A::Place use;
    use.b = static_cast<int>(which / items);
    use.item = static_cast<int>(which - static_cast<int64_t>(use.b) * items);
    use.at = S::COST;
    typename A::Query query[AT_WARPS];
#pragma unroll
    for (int i = 0; i < AT_WARPS; ++i) query[i].load(a, use, i, lane);
    Feed<E4M3, D, NT, FINE> feed;
    if (a.window == 0) feed.template look_up<1>(a, use, 0, a.held, 1, 0, lane);
    use.seen = seen_of(a, use.b);
    use.units = use.left = A::steps(use.seen);  // units of one step here
    const int h = a.chunks == 1 ? use.item : use.item / a.chunks, h0 = (use.item - h * a.chunks) * S::HEADS;
    const int heads = min(S::HEADS, a.group - h0);
    if (use.units == 0) {
        attn_nothing<D, 32>(a, use.b, h * a.group + h0, heads);
        return;
    }
    feed.start(use, ring, 0);
    if (a.window > 0) feed.template look_up<1>(a, use, use.seen.first, use.seen.n, 1, 0, lane);
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) feed.template next<true, 1>(a, i, 1, 0, lane);
#pragma unroll
    for (int i = 0; i < AT_WARPS; ++i) A::put_query(a, query[i], qf, qc, i, lane);
    __syncwarp();
    A state;
    state.begin(qc, lane);
    int stage = 0;
    attn_units<true, 1>(a, state, feed, use.seen, 0, use.units, 1, stage, ring, qf, 0, lane);
    cp_async_wait<0>();
    const int64_t row0 = static_cast<int64_t>(use.b) * a.q_heads + h * a.group + h0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        float l = state.l[i];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        float *const rows = reinterpret_cast<float *>(ring);  // nothing is being copied
        __syncwarp();
        state.put(i, rows, lane);
        __syncwarp();
#pragma unroll
        for (int j = lane; j < 8 * (D / 4); j += 32) {
            const int y = j / (D / 4), col = j % (D / 4) * 4;
            const float total = __shfl_sync(0xffffffffu, l, 4 * y), top = __shfl_sync(0xffffffffu, state.m[i], 4 * y);
            if (8 * i + y < heads) {
                attn_store(a, row0 + 8 * i + y, D, col, *reinterpret_cast<const float4 *>(rows + y * S::OROW + col), total);
                attn_store_lse(a, row0 + 8 * i + y, col, top, total);
            }
        }
    }
}

template <bool E4M3, int D, int NT, bool FINE>
cudaError_t launch_attn_line(const AttnArgs &a, int64_t most, cudaStream_t st)
{
    using S = AttnShape<E4M3, D, NT>;
    const auto kernel = attn_decode_kernel<E4M3, D, NT, FINE>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), S::SMEM); e != cudaSuccess) return e;
    const int64_t room = static_cast<int64_t>(num_sms()) * S::CTAS;
    const int grid = static_cast<int>(most < 1 ? 1 : most < room ? most : room);
    return launch_pdl(kernel, dim3(grid), dim3(AT_THREADS), S::SMEM, st, a);
}

template <bool E4M3, int D, int NT, bool FINE>
cudaError_t launch_attn_direct(const AttnArgs &a, cudaStream_t st)
{
    using S = AttnShape<E4M3, D, NT>;
    constexpr int SMEM = S::RECORD_AT + S::RECORD * 4;
    const auto kernel = attn_direct_kernel<E4M3, D, NT, FINE>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), SMEM); e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.batch * a.c.heads * a.chunks * a.cluster));
    if (a.cluster == 1) return launch_pdl(kernel, grid, dim3(AT_THREADS), SMEM, st, a);
    return launch_pdl_cluster(kernel, grid, dim3(AT_THREADS), SMEM, st, static_cast<unsigned>(a.cluster), a);
}

// One translation unit per format and head size: definitions in qg_attn_*.cu.  most: the places that the line can have.
template <bool E4M3, int D>
cudaError_t launch_attn_dim(const AttnArgs &a, int64_t most, cudaStream_t st);

template <bool E4M3, int D, int NT, bool FINE>
cudaError_t launch_attn_warps(const AttnArgs &a, cudaStream_t st)
{
    using S = AttnShape<E4M3, D, NT>;
    const auto kernel = attn_warps_kernel<E4M3, D, NT, FINE>;
    if (cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kernel), S::SMEM_WARPS); e != cudaSuccess) return e;
    const int64_t items = a.batch * a.c.heads * a.chunks;
    return launch_pdl(kernel, dim3(static_cast<unsigned>((items + AT_WARPS - 1) / AT_WARPS)), dim3(AT_THREADS), S::SMEM_WARPS, st, a);
}

template <bool E4M3, int D, int NT, bool FINE>
cudaError_t launch_attn_shape(const AttnArgs &a, int64_t most, cudaStream_t st)
{
    if (a.cluster < 0) return launch_attn_warps<E4M3, D, NT, FINE>(a, st);
    return a.cluster > 0 ? launch_attn_direct<E4M3, D, NT, FINE>(a, st) : launch_attn_line<E4M3, D, NT, FINE>(a, most, st);
}

#define QG_ATTN_DIM(E4M3, D)                                                                                       \
    template <>                                                                                                    \
    cudaError_t launch_attn_dim<E4M3, D>(const AttnArgs &a, int64_t most, cudaStream_t st)                         \
    {                                                                                                              \
        const bool fine = !a.q_bf16;                                                                               \
        if (a.group <= 8)                                                                                          \
            return fine ? launch_attn_shape<E4M3, D, 1, true>(a, most, st)                                         \
                        : launch_attn_shape<E4M3, D, 1, false>(a, most, st);                                       \
        return fine ? launch_attn_shape<E4M3, D, 2, true>(a, most, st)                                             \
                    : launch_attn_shape<E4M3, D, 2, false>(a, most, st);                                           \
    }

}  // namespace qg
