// Activations to e4m3 codes with one scale per row and block of 128, alone or
// behind the residual's addition and the RMSNorm.
#include "qg_e4m3.cuh"
#include "qg_norm.cuh"

namespace qg {

// x[rows][k] -> q[rows][k], d[rows][kb].  A warp holds one block per step, four
// values per lane, so a block is one load, one warp maximum and one 128-byte
// store of codes; it takes QB consecutive blocks (rows run on into one another)
// with all loads in flight before the first maximum, and lane i divides for
// block i, so the two IEEE divisions are paid once per QB blocks.
constexpr int QB = 8;
constexpr int QT = 256;

template <typename T>
__global__ void __launch_bounds__(QT) quantize_e4m3_kernel(const T *x, int64_t n_blocks, int kb, int k, uint8_t *q,
                                                           float *d)
{
    using V = Vec4<T>;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t b0 = (static_cast<int64_t>(blockIdx.x) * (QT / 32) + (threadIdx.x >> 5)) * QB;
    if (b0 >= n_blocks) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(QB), n_blocks - b0));
    const int64_t row0 = n_blocks < (int64_t(1) << 31) ? static_cast<uint32_t>(b0) / static_cast<uint32_t>(kb) : b0 / kb;
    int c = static_cast<int>(b0 - row0 * kb);        // block in its row
    int64_t at = row0 * k + static_cast<int64_t>(c) * EB;  // its first value

    typename V::raw v[QB];
    int64_t pos[QB];
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const int left = k - c * EB;  // values from here to the row's end
        pos[i] = i < n && lane * 4 < left ? at + lane * 4 : -1;
        v[i] = typename V::raw{};
        if (pos[i] >= 0) v[i] = *reinterpret_cast<const typename V::raw *>(x + pos[i]);
        at += min(left, EB);
        if (++c == kb) c = 0;
    }
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const float a = warp_max_nonneg(max_abs4(V::widen(v[i])));
        if (lane == i) mine = a;
    }
    mine = e4m3_floor(mine);
    const float inv = __fdiv_rn(448.0f, mine);
    if (lane < n) d[b0 + lane] = __fdiv_rn(mine, 448.0f);
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const float f = __shfl_sync(0xffffffffu, inv, i);
        const float4 w = V::widen(v[i]);
        if (pos[i] >= 0)
            *reinterpret_cast<uint32_t *>(q + pos[i]) = e4m3_pack4(w.x * f, w.y * f, w.z * f, w.w * f);
    }
}

// s = x + residual (rounded once to the stream's type), r = 1/sqrt(mean(s^2) + eps)
// as in f64 rounded once to f32, v = (s * r) * gamma (two f32 products), then the
// codes of v.  One CTA per row; block b of the row belongs to warp b mod W.
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

__device__ __forceinline__ void add_squares(f32pair &acc, float4 v)
{
    pair_add_square(acc, v.x);
    pair_add_square(acc, v.y);
    pair_add_square(acc, v.z);
    pair_add_square(acc, v.w);
}

// r for the CTA's row: every warp merges the W warps' sums itself (one barrier).
template <int W>
__device__ __forceinline__ float row_rms_inv(f32pair acc, int k, float inv_k, float eps, f32pair *scratch)
{
    acc = warp_pair_sum(acc);
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
    return rms_inv_from_pair(v, k, inv_k, eps);
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

// Any k: the row is read twice (the second time what this thread itself wrote to
// s, or x where there is no residual).
template <typename T, int W>
__global__ void __launch_bounds__(32 * W) norm_e4m3_kernel(const NormArgs<T> p)
{
    using V = Vec4<T>;
    using raw = typename V::raw;
    __shared__ f32pair scratch[W];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int64_t base = row * p.k;
    f32pair acc = {0.0f, 0.0f};
    for (int b = warp; b < p.kb; b += W) {
        const int c = b * EB + lane * 4;
        if (c >= p.k) continue;
        raw xv = *reinterpret_cast<const raw *>(p.x + base + c);
        float4 s = V::widen(xv);
        if (p.residual) {
            s = stream_sum<T>(xv, *reinterpret_cast<const raw *>(p.residual + base + c), xv);
            *reinterpret_cast<raw *>(p.s + base + c) = xv;
        }
        add_squares(acc, s);
    }
    const float r = row_rms_inv<W>(acc, p.k, p.inv_k, p.eps, scratch);
    const T *again = p.residual ? p.s : p.x;
    for (int b = warp; b < p.kb; b += W) {
        const int c = b * EB + lane * 4;
        const bool live = c < p.k;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            const float4 s = V::widen(*reinterpret_cast<const raw *>(again + base + c));
            const float4 g = V::widen(*reinterpret_cast<const raw *>(p.gamma + c));
            v.x = __fmul_rn(__fmul_rn(s.x, r), g.x);
            v.y = __fmul_rn(__fmul_rn(s.y, r), g.y);
            v.z = __fmul_rn(__fmul_rn(s.z, r), g.z);
            v.w = __fmul_rn(__fmul_rn(s.w, r), g.w);
        }
        store_codes(v, live, p.q + base + c, p.d + row * p.kb + b, lane);
    }
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
    if (dtype == QG_BF16)
        return launch_pdl(quantize_e4m3_kernel<__nv_bfloat16>, grid, dim3(QT), 0, st,
                          static_cast<const __nv_bfloat16 *>(x), n, static_cast<int>(kb), static_cast<int>(k), q, d);
    return launch_pdl(quantize_e4m3_kernel<float>, grid, dim3(QT), 0, st, static_cast<const float *>(x), n,
                      static_cast<int>(kb), static_cast<int>(k), q, d);
}

}  // namespace qg
