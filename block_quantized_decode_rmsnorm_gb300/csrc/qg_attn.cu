// Attention of one new token per sequence over the paged cache (plain form: a CTA to
// each sequence and query head, a warp to each token, one pass with a running maximum).
#include <cfloat>

#include "qg_kv.cuh"

namespace qg {

struct AttnArgs {
    KvPlanes c;
    const void *q;
    int64_t q_row, q_head;
    int q_bf16, group, q_heads;
    const int32_t *pages, *lengths;
    int64_t max_pages, window;
    float scale;
    void *out;
    int out_bf16;
    float *lse;
};

constexpr int AW = 4;

template <bool E4M3, int D>
__global__ void __launch_bounds__(32 * AW) attn_plain_kernel(AttnArgs a)
{
    constexpr int N = D / 32, NB = kv_blocks(E4M3, D), BLOCK = E4M3 ? EB : QK;
    __shared__ float part[AW][D + 2];
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, hq = blockIdx.x, h = hq / a.group, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t held = a.max_pages * a.c.page;
    const int64_t n = min(static_cast<int64_t>(max(a.lengths[b], 0)), held);
    const int64_t first = a.window > 0 ? max(n - a.window, int64_t(0)) : 0;
    float q[N], acc[N], m = -FLT_MAX, l = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t at = b * a.q_row + hq * a.q_head + lane + 32 * i;
        q[i] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[at])
                        : static_cast<const float *>(a.q)[at];
        acc[i] = 0.0f;
    }
    for (int64_t t = first + warp; t < n; t += AW) {
        const int32_t page = a.pages[b * a.max_pages + t / a.c.page];
        const bool there = page >= 0 && page < a.c.n_pages;
        const int64_t at = (static_cast<int64_t>(there ? page : 0) * a.c.heads + h) * a.c.page + t % a.c.page;
        float s = 0.0f, v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int col = lane + 32 * i;
            float kk = 0.0f;
            v[i] = 0.0f;
            if (there) {
                const uint8_t ck = a.c.kq[at * D + col], cv = a.c.vq[at * D + col];
                const int64_t blk = at * NB + col / BLOCK;
                if (E4M3) {
                    kk = __half2float(__half(__nv_cvt_fp8_to_halfraw(ck, __NV_E4M3))) * static_cast<const float *>(a.c.kd)[blk];
                    v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(cv, __NV_E4M3))) * static_cast<const float *>(a.c.vd)[blk];
                } else {
                    kk = static_cast<float>(static_cast<int8_t>(ck)) * h2f(static_cast<const uint16_t *>(a.c.kd)[blk]);
                    v[i] = static_cast<float>(static_cast<int8_t>(cv)) * h2f(static_cast<const uint16_t *>(a.c.vd)[blk]);
                }
            }
            s = fmaf(q[i], kk, s);
        }
        s = there ? warp_sum(s) * a.scale : __int_as_float(0x7fffffff);
        const float top = fmaxf(m, s), f = expf(m - top), p = expf(s - top);
        m = top;
        l = fmaf(l, f, p);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(acc[i], f, p * v[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) part[warp][lane + 32 * i] = acc[i];
    if (lane == 0) part[warp][D] = m, part[warp][D + 1] = l;
    __syncthreads();
    float top = -FLT_MAX, total = 0.0f;
    for (int w = 0; w < AW; ++w) top = fmaxf(top, part[w][D]);
    for (int w = 0; w < AW; ++w) total = fmaf(part[w][D + 1], expf(part[w][D] - top), total);
    const bool none = first >= n;
    for (int col = threadIdx.x; col < D; col += 32 * AW) {
        float o = 0.0f;
        for (int w = 0; w < AW; ++w) o = fmaf(part[w][col], expf(part[w][D] - top), o);
        o = none ? 0.0f : o / total;
        const int64_t at = (static_cast<int64_t>(b) * a.q_heads + hq) * D + col;
        if (a.out_bf16)
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(o);
        else
            static_cast<float *>(a.out)[at] = o;
    }
    if (threadIdx.x == 0 && a.lse)
        a.lse[static_cast<int64_t>(b) * a.q_heads + hq] = none ? -__int_as_float(0x7f800000) : top + logf(total);
}

int64_t attn_workspace_bytes(int64_t, int64_t, int64_t) { return 16; }

namespace {
template <bool E4M3>
cudaError_t plain(const AttnArgs &a, dim3 grid, cudaStream_t st)
{
    switch (a.c.dim) {
    case 64: return launch_pdl(attn_plain_kernel<E4M3, 64>, grid, dim3(32 * AW), 0, st, a);
    case 96: return launch_pdl(attn_plain_kernel<E4M3, 96>, grid, dim3(32 * AW), 0, st, a);
    case 128: return launch_pdl(attn_plain_kernel<E4M3, 128>, grid, dim3(32 * AW), 0, st, a);
    case 192: return launch_pdl(attn_plain_kernel<E4M3, 192>, grid, dim3(32 * AW), 0, st, a);
    default: return launch_pdl(attn_plain_kernel<E4M3, 256>, grid, dim3(32 * AW), 0, st, a);
    }
}
}  // namespace

cudaError_t launch_attn_decode(const KvPlanes &c, const void *q, int64_t q_row, int64_t q_head, int q_dtype,
                               int64_t batch, int64_t q_heads, const int32_t *pages, int64_t max_pages,
                               const int32_t *lengths, float scale, int64_t window, void *out, int out_dtype,
                               float *lse, void *, cudaStream_t st)
{
    const AttnArgs a = {c, q, q_row, q_head, q_dtype == QG_BF16, static_cast<int>(q_heads / c.heads),
                        static_cast<int>(q_heads), pages, lengths, max_pages, window, scale, out,
                        out_dtype == QG_BF16, lse};
    for (int64_t b = 0; b < batch; b += 32768) {
        AttnArgs part = a;
        const int64_t n = batch - b < 32768 ? batch - b : 32768;
        part.q = static_cast<const char *>(q) + b * q_row * (a.q_bf16 ? 2 : 4);
        part.pages = pages + b * max_pages;
        part.lengths = lengths + b;
        part.out = static_cast<char *>(out) + b * q_heads * c.dim * (a.out_bf16 ? 2 : 4);
        part.lse = lse ? lse + b * q_heads : nullptr;
        const dim3 grid(static_cast<unsigned>(q_heads), static_cast<unsigned>(n));
        if (cudaError_t e = c.e4m3 ? plain<true>(part, grid, st) : plain<false>(part, grid, st); e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qg
