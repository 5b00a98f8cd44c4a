// Activations to e4m3 codes with one scale per row and block of 128, alone or
// behind the residual's addition and the RMSNorm.
//
// Times in this file are of graph replays over operands that rotate through 400 MB.
#include <cfloat>
#include <type_traits>

#include "qg_e4m3.cuh"
#include "qg_norm.cuh"
#include "qg_tc.cuh"

namespace qg {

// x[rows][k] -> q[rows][k], d[rows][kb].  A warp holds one block per step, four
// values per lane, so a block is one load, one warp maximum and one 128-byte
// store of codes; it takes QB consecutive blocks (rows run on into one another)
// with all loads in flight before the first maximum, and lane i divides for
// block i, so the two IEEE divisions are paid once per QB blocks.  Bound by HBM
// where rows are many (8192x9216 bf16: 33.2 us for 229 MB, 6.9 TB/s), by issue before that: EVEN is the
// form for k a multiple of 128, where the blocks follow one another in memory and
// every lane of a whole group is live, and no position is computed per block.
constexpr int QB = 8;
constexpr int QT = 256;

template <typename T, bool EVEN>
__global__ void __launch_bounds__(QT) quantize_e4m3_kernel(const T *x, int64_t n_blocks, int kb, int k, uint8_t *q,
                                                           float *d)
{
    using V = Vec4<T>;
    const int lane = threadIdx.x & 31;
    const int64_t b0 = (static_cast<int64_t>(blockIdx.x) * (QT / 32) + (threadIdx.x >> 5)) * QB;
    const int n = static_cast<int>(min(static_cast<int64_t>(QB), n_blocks - b0));
    pdl_wait();
    pdl_trigger();
    if (n <= 0) return;
    typename V::raw v[QB];
    int64_t pos[EVEN ? 1 : QB];  // of this lane's values of each block, -1 past the row's end
    if constexpr (EVEN) {
        pos[0] = b0 * EB + lane * 4;
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            v[i] = typename V::raw{};
            if (i < n) v[i] = *reinterpret_cast<const typename V::raw *>(x + pos[0] + i * EB);
        }
    } else {
        const int64_t row0 = n_blocks < (int64_t(1) << 31) ? static_cast<uint32_t>(b0) / static_cast<uint32_t>(kb) : b0 / kb;
        int c = static_cast<int>(b0 - row0 * kb);              // block in its row
        int64_t at = row0 * k + static_cast<int64_t>(c) * EB;  // its first value
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int left = k - c * EB;  // values from here to the row's end
            pos[i] = i < n && lane * 4 < left ? at + lane * 4 : -1;
            v[i] = typename V::raw{};
            if (pos[i] >= 0) v[i] = *reinterpret_cast<const typename V::raw *>(x + pos[i]);
            at += min(left, EB);
            if (++c == kb) c = 0;
        }
    }
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const float a = warp_max_nonneg(V::max_abs(v[i]));
        if (lane == i) mine = a;
    }
    mine = e4m3_floor(mine);
    const float inv = __fdiv_rn(448.0f, mine);
    if (lane < n) d[b0 + lane] = __fdiv_rn(mine, 448.0f);
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const float f = __shfl_sync(0xffffffffu, inv, i);
        const float4 w = V::widen(v[i]);
        const uint32_t codes = e4m3_pack4(w.x * f, w.y * f, w.z * f, w.w * f);
        if constexpr (EVEN) {
            if (i < n) *reinterpret_cast<uint32_t *>(q + pos[0] + i * EB) = codes;
        } else {
            if (pos[i] >= 0) *reinterpret_cast<uint32_t *>(q + pos[i]) = codes;
        }
    }
}

// s = x + residual (rounded once to the stream's type), r = 1/sqrt(mean(s^2) + eps)
// as in f64 rounded once to f32, v = (s * r) * gamma (two f32 products), then the
// codes of v.  One CTA per row; block b of the row belongs to warp b mod W.  Bound by
// HBM where rows are many and long (16383x4112 f32: 124.3 us for 878 MB, 7.1 TB/s; read
// twice it took 12 us more), by issue for bf16 rows of a few blocks (4096x2560: 13.6 us,
// 80 % of the copy rate), by one row's chain of loads, sums and divisions below that.
template <typename T>
struct NormArgs {
    const T *x, *residual, *gamma;
    T *s;
    uint8_t *q;
    float *d;
    int k, kb;
    float inv_k, eps;
};

template <typename T>
__device__ __forceinline__ float4 stream_sum(typename Vec4<T>::raw x, typename Vec4<T>::raw r, typename Vec4<T>::raw &s)
{
    const float4 a = Vec4<T>::widen(x), b = Vec4<T>::widen(r);
    s = Vec4<T>::narrow(make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w)));
    return Vec4<T>::widen(s);
}

// The compensated sum of exact squares (pair_add_square) two values at a time: the
// row's even and odd values have a pair of their own, and the two-sum takes packed
// additions, the differences among them as fma(x, -1, y), which rounds as y - x does.
struct f32pair2 {
    uint64_t hi, lo;
};

template <typename T>
__device__ __forceinline__ void add_square2(f32pair2 &acc, float x, float y)
{
    const uint64_t v = pack2(x, y), minus = pack2(-1.0f, -1.0f);
    const uint64_t p = mul2(v, v);
    const uint64_t s = add2(acc.hi, p);
    const uint64_t bb = fma2(acc.hi, minus, s);
    const uint64_t err = add2(fma2(fma2(bb, minus, s), minus, acc.hi), fma2(bb, minus, p));
    acc.hi = s;
    acc.lo = add2(acc.lo, err);
    // what the square lost in rounding; nothing where the value has eight bits
    if constexpr (std::is_same<T, float>::value) acc.lo = add2(acc.lo, fma2(v, v, mul2(p, minus)));
}

template <typename T>
__device__ __forceinline__ void add_squares(f32pair2 &acc, float4 v)
{
    add_square2<T>(acc, v.x, v.y);
    add_square2<T>(acc, v.z, v.w);
}

// r for the CTA's row: every warp merges the W warps' sums itself (one barrier).  The pairs
// hold for a = mean(s^2) + eps from 2^-100 (below, what a square loses in rounding is itself
// rounded; the sum's error is under 2^-150 k) up to f32's end.  Any other row, NaN and
// infinities among its values, is summed again in f64: the whole CTA, as every thread has the
// same a.  values(f) calls f with each of this thread's values of s.
template <int W, typename Values>
__device__ __forceinline__ float row_rms_inv(f32pair2 sums, int k, float inv_k, float eps, f32pair *scratch,
                                             const Values &values)
{
    const float2 hi = unpack2(sums.hi), lo = unpack2(sums.lo);
    const f32pair acc = warp_pair_sum(pair_merge({hi.x, lo.x}, {hi.y, lo.y}));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = acc;
    __syncthreads();
    f32pair v = scratch[threadIdx.x & (W - 1)];
#pragma unroll
    for (int o = W / 2; o >= 1; o >>= 1) {
        f32pair w;
        w.hi = __shfl_xor_sync(0xffffffffu, v.hi, o);
        w.lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
        v = pair_merge(v, w);
    }
    const float a = fmaf(v.hi, inv_k, eps);
    if (a >= 0x1p-100f && a <= FLT_MAX) return rms_inv_from_pair(v, k, inv_k, eps);
    double sum = 0.0;
    values([&](float s) { sum = fma(static_cast<double>(s), static_cast<double>(s), sum); });
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    double *total = reinterpret_cast<double *>(scratch);
    __syncthreads();  // every warp has read the pairs
    if ((threadIdx.x & 31) == 0) total[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll 1
    for (int w = 0; w < W; ++w) sum += total[w];
    return static_cast<float>(1.0 / sqrt(sum / k + static_cast<double>(eps)));
}

// The codes of four values of one block, the whole warp on that block; live: this
// lane's values exist.
__device__ __forceinline__ void store_codes(float4 v, bool live, uint8_t *q, float *d, int lane)
{
    const float a = e4m3_floor(warp_max_nonneg(max_abs4(v)));
    const float f = __fdiv_rn(448.0f, a);
    if (live) *reinterpret_cast<uint32_t *>(q) = e4m3_pack4(v.x * f, v.y * f, v.z * f, v.w * f);
    if (lane == 0) *d = __fdiv_rn(a, 448.0f);
}

// (s * r) * gamma, two f32 products.
__device__ __forceinline__ float4 normalised(float4 s, float r, float4 g)
{
    const uint64_t rr = pack2(r, r);
    const float2 a = unpack2(mul2(mul2(pack2(s.x, s.y), rr), pack2(g.x, g.y)));
    const float2 b = unpack2(mul2(mul2(pack2(s.z, s.w), rr), pack2(g.z, g.w)));
    return make_float4(a.x, a.y, b.x, b.y);
}

// k over 8192: the row is read twice (the second time what this thread itself wrote
// to s, or x where there is no residual).
template <typename T, int W>
__global__ void __launch_bounds__(32 * W) norm_e4m3_kernel(const NormArgs<T> p)
{
    using V = Vec4<T>;
    using raw = typename V::raw;
    __shared__ __align__(8) f32pair scratch[W];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int64_t base = row * p.k;
    f32pair2 acc = {0, 0};
    for (int b = warp; b < p.kb; b += W) {
        const int c = b * EB + lane * 4;
        if (c >= p.k) continue;
        raw xv = *reinterpret_cast<const raw *>(p.x + base + c);
        float4 s = V::widen(xv);
        if (p.residual) {
            s = stream_sum<T>(xv, *reinterpret_cast<const raw *>(p.residual + base + c), xv);
            *reinterpret_cast<raw *>(p.s + base + c) = xv;
        }
        add_squares<T>(acc, s);
    }
    const T *again = p.residual ? p.s : p.x;
    const float r = row_rms_inv<W>(acc, p.k, p.inv_k, p.eps, scratch, [&](auto f) {
        for (int b = warp; b < p.kb; b += W) {
            const int c = b * EB + lane * 4;
            if (c >= p.k) continue;
            const float4 s = V::widen(*reinterpret_cast<const raw *>(again + base + c));
            f(s.x), f(s.y), f(s.z), f(s.w);
        }
    });
    for (int b = warp; b < p.kb; b += W) {
        const int c = b * EB + lane * 4;
        const bool live = c < p.k;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            v = normalised(V::widen(*reinterpret_cast<const raw *>(again + base + c)), r,
                           V::widen(*reinterpret_cast<const raw *>(p.gamma + c)));
        }
        store_codes(v, live, p.q + base + c, p.d + row * p.kb + b, lane);
    }
}

// Rows of at most NB blocks per warp: the row stays in registers, and is read once.
template <typename T, int W, int NB>
__global__ void __launch_bounds__(32 * W) norm_row_e4m3_kernel(const NormArgs<T> p)
{
    using V = Vec4<T>;
    using raw = typename V::raw;
    __shared__ __align__(8) f32pair scratch[W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int64_t base = row * p.k;
    pdl_wait();
    pdl_trigger();
    raw v[NB], g[NB];
    f32pair2 acc = {0, 0};
    {
        raw e[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int c = (warp + W * i) * EB + lane * 4;
            v[i] = e[i] = g[i] = raw{};
            if (c >= p.k) continue;
            v[i] = *reinterpret_cast<const raw *>(p.x + base + c);
            if (p.residual) e[i] = *reinterpret_cast<const raw *>(p.residual + base + c);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int c = (warp + W * i) * EB + lane * 4;
            if (c >= p.k) continue;
            g[i] = *reinterpret_cast<const raw *>(p.gamma + c);
            if (p.residual) {
                stream_sum<T>(v[i], e[i], v[i]);
                *reinterpret_cast<raw *>(p.s + base + c) = v[i];
            }
            add_squares<T>(acc, V::widen(v[i]));
        }
    }
    const float r = row_rms_inv<W>(acc, p.k, p.inv_k, p.eps, scratch, [&](auto f) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {  // zeros where nothing is
            const float4 s = V::widen(v[i]);
            f(s.x), f(s.y), f(s.z), f(s.w);
        }
    });
    // the maxima of all blocks, then lane i divides for block i
    float4 h[NB];
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        h[i] = normalised(V::widen(v[i]), r, V::widen(g[i]));  // zeros where nothing is
        const bool live = (warp + W * i) * EB + lane * 4 < p.k;
        const float a = warp_max_nonneg(live ? max_abs4(h[i]) : 0.0f);
        if (lane == i) mine = a;
    }
    mine = e4m3_floor(mine);
    const float inv = __fdiv_rn(448.0f, mine);
    if (lane < NB && warp + W * lane < p.kb) p.d[row * p.kb + warp + W * lane] = __fdiv_rn(mine, 448.0f);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const float f = __shfl_sync(0xffffffffu, inv, i);
        const int c = (warp + W * i) * EB + lane * 4;
        if (c < p.k)
            *reinterpret_cast<uint32_t *>(p.q + base + c) = e4m3_pack4(h[i].x * f, h[i].y * f, h[i].z * f, h[i].w * f);
    }
}

template <typename T, int W, int NB>
static cudaError_t launch_row(const NormArgs<T> &p, int64_t rows, cudaStream_t st)
{
    return launch_pdl(norm_row_e4m3_kernel<T, W, NB>, dim3(static_cast<unsigned>(rows)), dim3(32 * W), 0, st, p);
}

template <typename T>
static cudaError_t launch_norm_t(const void *x, const void *residual, const void *gamma, int64_t rows, int64_t k,
                                 float eps, void *s, uint8_t *q, float *d, cudaStream_t st)
{
    NormArgs<T> p;
    p.x = static_cast<const T *>(x);
    p.residual = static_cast<const T *>(residual);
    p.gamma = static_cast<const T *>(gamma);
    p.s = static_cast<T *>(s);
    p.q = q;
    p.d = d;
    p.k = static_cast<int>(k);
    p.kb = static_cast<int>(e4m3_blocks(k));
    p.inv_k = 1.0f / static_cast<float>(k);
    p.eps = eps;
    // Four warps a row where rows fill the SMs: what a warp does once a row (the merges of
    // the compensated sums) is then shared by twice the blocks (4096x2560 bf16: 13.6 us,
    // 2.4 more with eight warps).  Eight where the row's own latency counts (1x1024: 1.5 us,
    // 0.2 more with four), and for the registers of long rows.
    const bool many = rows > 2 * num_sms();
    if (many && p.kb <= 8) return launch_row<T, 4, 2>(p, rows, st);
    if (many && p.kb <= 12) return launch_row<T, 4, 3>(p, rows, st);
    if (many && p.kb <= 20) return launch_row<T, 4, 5>(p, rows, st);
    if (many && p.kb <= 32) return launch_row<T, 4, 8>(p, rows, st);
    if (p.kb <= 8) return launch_row<T, 8, 1>(p, rows, st);
    if (p.kb <= 16) return launch_row<T, 8, 2>(p, rows, st);
    if (p.kb <= 32) return launch_row<T, 8, 4>(p, rows, st);
    if (p.kb <= 40) return launch_row<T, 8, 5>(p, rows, st);
    if (p.kb <= 64) return launch_row<T, 8, 8>(p, rows, st);
    return launch_pdl(norm_e4m3_kernel<T, 8>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, p);
}

cudaError_t launch_norm_e4m3(const void *x, const void *residual, const void *gamma, int dtype, int64_t rows, int64_t k,
                             float eps, void *s, uint8_t *q, float *d, cudaStream_t st)
{
    return dtype == QG_BF16 ? launch_norm_t<__nv_bfloat16>(x, residual, gamma, rows, k, eps, s, q, d, st)
                            : launch_norm_t<float>(x, residual, gamma, rows, k, eps, s, q, d, st);
}

cudaError_t launch_quantize_e4m3(const void *x, int dtype, int64_t rows, int64_t k, uint8_t *q, float *d,
                                 cudaStream_t st)
{
    const int64_t kb = e4m3_blocks(k), n = rows * kb;
    const int64_t per_cta = static_cast<int64_t>(QB) * (QT / 32);
    const dim3 grid(static_cast<unsigned>((n + per_cta - 1) / per_cta));
    if (dtype == QG_BF16) {
        const auto *p = static_cast<const __nv_bfloat16 *>(x);
        const auto kernel = k % EB == 0 ? quantize_e4m3_kernel<__nv_bfloat16, true> : quantize_e4m3_kernel<__nv_bfloat16, false>;
        return launch_pdl(kernel, grid, dim3(QT), 0, st, p, n, static_cast<int>(kb), static_cast<int>(k), q, d);
    }
    const auto *p = static_cast<const float *>(x);
    const auto kernel = k % EB == 0 ? quantize_e4m3_kernel<float, true> : quantize_e4m3_kernel<float, false>;
    return launch_pdl(kernel, grid, dim3(QT), 0, st, p, n, static_cast<int>(kb), static_cast<int>(k), q, d);
}

}  // namespace qg
